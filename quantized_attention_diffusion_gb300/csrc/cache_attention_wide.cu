// cache_attention_wide.cu -- the attention over the KV cache for many query
// rows to a key/value head (a shared prefix, a chunk of new tokens), on the
// tcgen05 tensor cores (sm_103a).
//
// The formulas are cache_attention.cu's with one exponential a score: p = 2^(x - R)
// serves the sum L, in fp32, and, times the key's scale of V and rounded to fp16, the
// second product.  R is some 6 below the largest x + log2 sv so far (weights down to
// 2^-19 of the largest keep all their bits), but at most 60 from the
// largest x; where V's scales are farther, a row's weights take a factor f = 2^-D more
// (1 otherwise) and its accumulator stands relative to R + D.  R and D are whole
// numbers.  V's codes are exact in fp16.  (A p below 2^-126 is 0: no weight that counts has
// one while V's scales are below 2^100 and within 2^150 of one another.)
//
// A CTA owns 256 query rows of one unit and walks its key tiles of 128.  Its two
// halves are two row tiles of 128, or, where a unit has at most 128 rows, the even
// and the odd key tiles of the same rows, joined at the end: either way one half's
// softmax runs while the tensor cores work for the other.
//
//   warps 0-3    read K's codes from global memory, convert them to fp16 (exact)
//                and store them swizzled, two stages; keys behind the last are
//                stored as zeros
//   warps 4-7    the same for V's codes, with the largest of their scales
//   warps 8-11   softmax of half 0, one thread a row
//   warps 12-15  the same for half 1
//   warps 16-19  one thread each issues S_0 = Q_0 K^T, S_1 = Q_1 K^T, O_0 += P_0 V,
//                O_1 += P_1 V; what it has to know of a tile stands beside the stage
//
// TMEM (512 columns): two buffers of 64 scores for each half, [0,64) and [64,128)
// of half 0, [128,192) and [192,256) of half 1, then O0 [256,384) O1 [384,512).
// The scores of a half's next 64 keys are formed while its softmax has the last
// 64 in hand.  The weights (fp16, two to a column) take the first 32 columns of
// their scores' buffer, each 32 over columns that have been read before, and are
// the second product's A operand from there; V is its B operand with the keys as
// the outer index, as the cache has it.
//
// What bounds it is the issue of the softmax's and the conversion's instructions (61% of
// the slots in 4 bits, the tensor cores active for 38% of the time beside it): a warp's 64
// scores take 1650 of a buffer's 1950 clocks.  2 x 1000 tokens x 16 heads over up to 9000
// keys: 173 us in 8 bits, 146 us in 4, 0.39 and 0.46 of the measured bf16 rate (per 8000
// keys more, 108 us in 4 bits, 0.64 of it; the rest is the start, the parts and their
// merge); 24 x 5 tokens x 16 heads behind a prefix of 32760, all in all: 70 and 69 us.
// Until its jumps were few (what is rare told to the compiler, the usual path in a line)
// the 8-bit chunk took 207 us: each jump waits for its instructions, since five kinds of
// warps share their cache.
//
// A 4-bit cache's scales are powers of two: where those of a warp's 32 keys are near one
// another, one of them stands for all and the values take the rest, exactly, so that the
// softmax needs no scale a key (Even, below).
//
// A row's references move where 32 weights may pass 2^15 in sum, by a whole number:
// then the thread scales the row's sum, its accumulator and the weights of this
// buffer that it has stored already by a power of two, which is exact, and forms
// the 32 again.
#include <type_traits>
#include <cuda_fp16.h>

#include "cache_attention.cuh"

namespace sage::cache {

namespace {

constexpr int kThreads = 20 * 32;
// Registers of the five warpgroups: a launch of 640 threads has 96 each; with these
// nothing spills.
constexpr int kRegsConvert = 88, kRegsSoftmax = 120, kRegsIssue = 64;
static_assert(2 * kRegsConvert + 2 * kRegsSoftmax + kRegsIssue <= 5 * 96, "more registers than the launch has");
static_assert(kRegsConvert <= 96 && kRegsIssue <= 96 && kRegsSoftmax >= 96, "a share given up cannot grow, one taken cannot shrink");
constexpr uint32_t kHalf = 128 * 128;                   // 128 rows of 64 16-bit values
constexpr uint32_t kTileBytes = 2 * kHalf;
constexpr uint32_t kSmemQ = 0;                          // two row tiles
constexpr uint32_t kSmemK = 2 * kTileBytes;             // two stages
constexpr uint32_t kSmemV = 4 * kTileBytes;             // two stages
constexpr uint32_t kSmemBytes = 6 * kTileBytes + 1024;  // and room to align to 1024
constexpr int kScaleSlots = 4;                          // of ks and vs: up to three tiles ahead of the softmax
constexpr float kFar = 32768.0f;                        // 2^15: most of 32 weights' sum (fp16: 65504)
constexpr float kAbove = 6.0f;                          // a reference that moves goes so far below the largest weight:
                                                        // 32 of that are a sixteenth of kFar
constexpr float kFarSum = 0x1p70f, kTiny = 0x1p-55f;    // most of 32 p's sum, and kFar / kFarSum
constexpr uint32_t kFoldV = 4;                          // V's scales of 32 keys that one of them stands for: within 2^4
constexpr float kNear = 4096.0f;                        // most of |R| in weigh_even
constexpr float kSmall = 0x1p-70f;                      // least of L times V's scale there
constexpr float kLarge = 0x1p60f;                       // most of a row's factor and of K's scale there: their product is finite
constexpr float kReach = 60.0f, kReachV = 140.0f;       // of R, and of R + D, below the largest score

constexpr int kSub = 64;                                // keys of a score buffer
__host__ __device__ constexpr uint32_t col_s(int t, int b) { return 128u * t + 64u * b; }
__host__ __device__ constexpr uint32_t col_o(int t) { return 256u + 128u * t; }

// What the issuing threads know of a stage's tile.
constexpr int kTileOf = 3;        // 0, 1 or 2: the segment's first tile, its second, a later one
constexpr int kTileOdd = 4;       // an odd tile of its segment
constexpr int kTileByRows = 8;    // the halves are row tiles
constexpr int kTileMore = 16;     // the segment has more than one tile
constexpr int kTileEnd = 32;      // no tile: the CTA has no more

struct Barriers {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], scales[kScaleSlots];
  uint64_t q_full[3], half_full, half_read, drain[4];     // of Q tile 0, of 1, and of 0 for half 1
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];   // [half][buffer]
};

template <int N>
__device__ __forceinline__ void fewer_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void more_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// 16 bytes at chunk c (0..15) of row r of a tile: two halves of 64 values, rows of
// 128 bytes, 128-byte swizzle.
__device__ __forceinline__ uint32_t tile_offset(int r, int c) {
  return (c >> 3) * kHalf + (r >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// 16 bytes that are read once: no line of L1 for them.
__device__ __forceinline__ uint4 load_once(const uint8_t* src) {
  uint4 w;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(src));
  return w;
}

// Four E4M3 codes -> two pairs of fp16, exactly.
__device__ __forceinline__ void v_codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

// 16 codes of a row as they are in global memory, and their fp16 values.
template <int kBits>
struct Codes;
template <>
struct Codes<8> {
  uint4 w;
  __device__ void load(const uint8_t* codes, const uint8_t*) { w = load_once(codes); }
  template <bool kIsV>
  __device__ void values(uint32_t (&o)[8], uint32_t) const {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (kIsV)
        v_codes_f16(u[i], o[2 * i], o[2 * i + 1]);
      else
        k_codes_f16(u[i], o[2 * i], o[2 * i + 1]);
    }
  }
};
// One block: its codes times its scale, 6 significant bits, exact in fp16, and times
// `fold` (two fp16, a power of two down to 2^-14 or 0), exact as well.
template <>
struct Codes<4> {
  uint2 w;
  uint32_t block;
  __device__ void load(const uint8_t* codes, const uint8_t* blocks) {
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(w.x), "=r"(w.y) : "l"(codes));
    asm volatile("ld.global.nc.L1::no_allocate.u8 %0, [%1];" : "=r"(block) : "l"(blocks));
  }
  template <bool>
  __device__ void values(uint32_t (&o)[8], uint32_t fold) const {
    uint32_t s2;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2) : "h"(static_cast<uint16_t>(block * 0x0101u)));
    s2 = mul_f16x2(s2, fold);
    const uint32_t u[2] = {w.x, w.y};
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t h[4];
      e2m1x8_f16(u[i], h);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[4 * i + j] = mul_f16x2(h[j], s2);
    }
  }
};

__device__ __forceinline__ float2 unpack_bf16(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ void store32(void* dst, uint32_t a, uint32_t b, uint32_t c, uint32_t d, uint32_t e, uint32_t f,
                                        uint32_t g, uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(a), "r"(b), "r"(c), "r"(d),
               "r"(e), "r"(f), "r"(g), "r"(h)
               : "memory");
}

// What a thread knows of its row.
struct Row {
  float rk;                  // its factor
  float R, D, f;             // the reference of L, the accumulator's relative to it, f = 2^-D
  float2 l;                  // L in two parts
};

// 2^n for a whole n of at most 127, 0 below the range.
__device__ __forceinline__ float power_of_two(float n) {
  return n < -126.0f ? 0.0f : __int_as_float((127 + static_cast<int>(n)) << 23);
}

// The rare move of a row's references to its largest score and weight so far, in
// the 32 scores at tS of which it sees `left`; -> whether they moved, and the
// accumulator's factor.
__device__ __forceinline__ bool move_references(uint32_t tS, const float* kx, const float* vx, int left, bool far, Row& z,
                                                float& alpha) {
  float xm = -INFINITY, ym = -INFINITY;                    // ym: relative to xm
#pragma unroll 1
  for (int c = 0; c < 32; c += 4) {
    uint32_t a[4];
    tmem_ld4(tS + c, a);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      larger(xm, ym, c + i < left ? __fmul_rn(__uint_as_float(a[i]) * kx[c + i], z.rk) : -INFINITY, lg2_approx(vx[c + i]));
  }
  const float top = ceilf(xm);
  float R = z.R, D = z.D;
  if (far && fabsf(top) < INFINITY) {                      // a row's result is its own alone
    const float below = fmaxf(ym - (top - xm), -kReachV) - kAbove;      // of the accumulator's reference, from top
    R = fmaxf(R, top + fminf(fmaxf(ceilf(below), -kReach), kReach));
    D = fmaxf(D + (z.R - R), ceilf(below) + (top - R));
  }
  const bool moved = R != z.R || D != z.D;
  const float less = power_of_two(z.R - R);
  alpha = power_of_two((z.R - R) + (z.D - D));
  z.l.x *= less;
  z.l.y *= less;
  z.R = R;
  z.D = D;
  z.f = power_of_two(-D);
  return moved;
}

// The accumulator times alpha, of this thread's row (if it holds anything yet), and
// the buffer's first 32 weights if they are there.  All lanes of a warp together.
__device__ __forceinline__ void rescale(uint32_t tO, uint32_t tP, bool has_o, bool has_p, float alpha) {
  if (has_o) {
#pragma unroll 1
    for (int k = 0; k < 32; ++k) {
      uint32_t o[4];
      tmem_ld4(tO + 4 * k, o);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
      tmem_st4(tO + 4 * k, o);
    }
  }
  tmem_st_wait();
  if (has_p) {
#pragma unroll 1
    for (int k = 0; k < 4; ++k) {
      uint32_t w[4];
      tmem_ld4(tP + 4 * k, w);
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        w[i] = pack_f16(x.x * alpha, x.y * alpha);
      }
      tmem_st4(tP + 4 * k, w);
    }
  }
  tmem_st_wait();
}

// 32 of a row's scores (TMEM columns tS ..) to weights, and the sum of the p's.
// kx, vx: the keys' scales (K's times softmax_scale * log2 e); top: at least V's
// largest; left: keys of these that the row sees.  kSlow: not all, or a scale is not
// finite, or a row's f is not 1.  -> whether the references have to move.
template <bool kSlow>
__device__ __forceinline__ bool weigh(uint32_t tS, const float* kx, const float* vx, float top, int left, const Row& z,
                                      uint32_t (&w)[16], float2& sum) {
  uint32_t a[32];
  tmem_ld32(tS, a);
  tmem_ld_wait();
  sum = make_float2(0.0f, 0.0f);
  float2 sumw = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 k4 = reinterpret_cast<const float4*>(kx)[i], v4 = reinterpret_cast<const float4*>(vx)[i];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int at = 4 * i + 2 * e;
      const float2 k2 = e == 0 ? make_float2(k4.x, k4.y) : make_float2(k4.z, k4.w);
      const float2 v2 = e == 0 ? make_float2(v4.x, v4.y) : make_float2(v4.z, v4.w);
      const float2 y = fmul2v(make_float2(__uint_as_float(a[at]), __uint_as_float(a[at + 1])), k2);
      float2 x = ffma2_bc(y.x, y.y, z.rk, -z.R);           // rk is a power of two: y * rk is exact
      if constexpr (kSlow) {
        if (at >= left) x.x = -INFINITY;
        if (at + 1 >= left) x.y = -INFINITY;
      }
      const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
      sum = fadd2v(sum, p);
      float2 q = fmul2v(p, v2);
      if constexpr (kSlow) {                               // a scale that is not finite stays behind the limit
        q = fmul2v(q, make_float2(z.f, z.f));              // last: f may be 2^86, and a scale times it infinite
        if (at >= left) q.x = 0.0f;
        if (at + 1 >= left) q.y = 0.0f;
        sumw = fadd2v(sumw, q);
      }
      w[at / 2] = pack_f16(q.x, q.y);
    }
  }
  const float total = sum.x + sum.y;
  return kSlow ? total > kFarSum || !(sumw.x + sumw.y <= kFar) : total * top > kFar;
}

// Of a 4-bit cache's tile: for its keys 16 i + 4 g + 0 .. 3, the one scale of K (times
// softmax_scale * log2 e) and of V that stand for all of them, the rows' own being in the
// values; negative where the rows' scales were too far apart for that.
struct Even {
  float4 k, v;
  __device__ float least_k() const { return fminf(fminf(k.x, k.y), fminf(k.z, k.w)); }
  __device__ float least_v() const { return fminf(fminf(v.x, v.y), fminf(v.z, v.w)); }
};

// weigh of a buffer's 64 scores where those are positive, the row sees all of the keys and R is
// near: weights 2^(x + log2 v - R) at once, and L's p from their sums, since the scales are
// powers of two.  The product in x is not rounded by itself, as weigh and R have it, and log2 v
// joins R first: of an R up to kNear the first is 2^-12 of log2 at the most and the second
// exact, and rows farther out take weigh.  So do rows whose L times the smallest v is below
// kSmall: a weight below 2^-126 is 0, and the p that L then lacks is less than 2^-126 / v,
// 2^-56 of L (2^30 keys: 2^-26).  Five instructions for two scores where the arrays of scales take eight
// and a load; the next 16 scores are loaded meanwhile.  -> scores whose weights are
// stored: 64, or fewer where the references have to move first.
__device__ __forceinline__ int weigh_even(uint32_t tS, const Even& ev, Row& z) {
  uint32_t next[16];
  tmem_ld16(tS, next);
  const float k[4] = {ev.k.x * z.rk, ev.k.y * z.rk, ev.k.z * z.rk, ev.k.w * z.rk};
  const float v[4] = {ev.v.x, ev.v.y, ev.v.z, ev.v.w};
  float b[4], back[4];                       // log2 v - R, 1 / v
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    b[g] = static_cast<float>(static_cast<int>(__float_as_uint(v[g]) >> 23) - 127) - z.R;
    back[g] = __uint_as_float((254u << 23) - __float_as_uint(v[g]));
  }
#pragma unroll
  for (int c = 0; c < kSub; c += 32) {
    float2 q[4];
    uint32_t w[16];
#pragma unroll
    for (int h = 0; h < 32; h += 16) {
      uint32_t a[16];
      tmem_ld_wait16(next);
#pragma unroll
      for (int i = 0; i < 16; ++i) a[i] = next[i];
      if (c + h + 16 < kSub) tmem_ld16(tS + c + h + 16, next);
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        const int g = i >> 2;
        const float2 x = ffma2_bc(__uint_as_float(a[i]), __uint_as_float(a[i + 1]), k[g], b[g]);
        const float2 y = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        q[g] = h == 0 && (i & 2) == 0 ? y : fadd2v(q[g], y);
        w[(h + i) / 2] = pack_f16(y.x, y.y);
      }
    }
    float2 sum = make_float2(0.0f, 0.0f);
    float all = 0.0f;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      all += q[g].x + q[g].y;
      sum.x += q[g].x * back[g];
      sum.y += q[g].y * back[g];
    }
    if (unlikely(__any_sync(0xFFFFFFFFu, all > kFar || sum.x + sum.y > kFarSum))) {
      tmem_ld_wait16(next);
      return c;
    }
    z.l = fadd2v(z.l, sum);
    tmem_st16(tS + c / 2, w);
  }
  return kSub;
}

template <bool kPrefix, int kBits>
__global__ void __launch_bounds__(kThreads, 1) cache_attn_wide_kernel(const __grid_constant__ Params p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  __shared__ Barriers bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  __shared__ int s_len[kMaxBatch];
  __shared__ long long s_off[kPrefix ? 2 : kMaxBatch + 1];
  __shared__ __align__(16) float s_ks[kScaleSlots][kWideTok], s_vs[kScaleSlots][kWideTok];
  __shared__ __align__(16) float s_top[kScaleSlots][4];   // of a V warp's keys: the largest scale, or infinity
  __shared__ __align__(16) float s_even[2][kScaleSlots][4];   // 4 bits: Even's k and v
  __shared__ int s_info[2][2];                            // [K, V][stage]
  __shared__ volatile long long s_end, s_per;
  __shared__ float4 s_half[128];                          // R, L and D of half 1's rows

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_v = &abort_flag;
  asm volatile("griddepcontrol.launch_dependents;");

  const Walk<kWideRows, kWideTok, kWideCost, kPrefix> walk{p, s_len, s_off};
  walk.plan(s_len, s_off);
  if (threadIdx.x == 32) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bars.k_full[s], 128);
      mbar_init(&bars.k_empty[s], 2);
      mbar_init(&bars.v_full[s], 128);
      mbar_init(&bars.v_empty[s], 2);
      for (int b = 0; b < 2; ++b) {
        mbar_init(&bars.s_full[s][b], 1);
        mbar_init(&bars.p_full[s][b], 128);
        mbar_init(&bars.pv_done[s][b], 1);
      }
    }
    for (int s = 0; s < 3; ++s) mbar_init(&bars.q_full[s], 128);
    for (int s = 0; s < kScaleSlots; ++s) mbar_init(&bars.scales[s], 256);
    mbar_init(&bars.half_full, 128);
    mbar_init(&bars.half_read, 128);
    for (int s = 0; s < 4; ++s) mbar_init(&bars.drain[s], 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == 16) {
    tmem_alloc(&tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  const long long total = s_off[walk.seqs()] * p.cache.H;
  const long long per = div_floor(total + gridDim.x - 1, gridDim.x);
  const long long f0 = blockIdx.x * per, f1 = min(total, f0 + per);
  if (threadIdx.x == 8 * 32) {                          // kept here for walk.tell, to save registers
    s_end = f1;
    s_per = per;
  }
  if (!p.keep && threadIdx.x == 0) p.desc[blockIdx.x].w = 0;
  if (f0 < f1) {
    Place x = walk.locate(f0, static_cast<int>(f1 - f0));
    auto wait = [&](uint64_t* bar, uint32_t parity) { return mbar_wait_inline(bar, parity & 1u, abort_v, p.err, p.timeout_ns); };

    if (warp < 8) {
      fewer_registers<kRegsConvert>();
      // ----------------------------------------------------------- convert --
      // Step i of a tile takes its keys 16 i .. 16 i + 15, which lie in one page.
      // Lane bits: 0-1 and 3 the 16 codes of a row, 2 and 4 the row of four: the
      // eight lanes of a 16-byte store fall into distinct banks.  A tile's codes
      // are loaded while the one before is converted, its pages one tile earlier.
      const bool is_v = warp >= 4;
      const int tid = threadIdx.x & 127;
      const int sub = 4 * (warp & 3) + ((lane >> 2) & 1) + 2 * (lane >> 4);   // key of a step
      const int q16 = (lane & 3) + ((lane >> 3) & 1) * 4;                     // 16 codes of a key
      // The key whose scale it loads; of V, and in 4 bits, one that its warp converts.
      const int scale_key = is_v || kBits == 4 ? 16 * (lane >> 2) + 4 * (warp & 3) + (lane & 3) : tid;
      const int ps = p.cache.page_shift;
      constexpr int kRow = kHeadDim * kBits / 8;                              // bytes of a key's codes
      const uint8_t* codes = (is_v ? p.cache.v_codes : p.cache.k_codes) + q16 * (kRow / 8);
      const uint8_t* blocks = kBits == 8 ? nullptr : (is_v ? p.cache.v_block : p.cache.k_block) + q16;
      const float* scales = is_v ? p.cache.v_scale : p.cache.k_scale;
      uint8_t* dst = smem + (is_v ? kSmemV : kSmemK) + tile_offset(sub, 2 * q16);
      const uint32_t odd = tile_offset(sub, 2 * q16 + 1) - tile_offset(sub, 2 * q16);   // 16 or -16: wraps
      uint64_t* full = is_v ? bars.v_full : bars.k_full;
      uint64_t* empty = is_v ? bars.v_empty : bars.k_empty;
      bool bad = false;
      // The tile whose codes are loaded next: its keys' page (lane i: of step i), head and bounds.
      int page = -1, head = 0, t0 = 0, hi = 0;
      int tile = x.t0, info = 0, info_next = 0;
      bool more = true, loaded = false;   // tiles to ask for; codes that wait to be converted
      auto ask = [&]() {
        page = -1;
        more = x.left > 0;
        if (!more) return;
        const int j = tile - x.t0;
        info_next = min(j, 2) | ((j & 1) != 0 ? kTileOdd : 0) | (p.rows - x.rt * kWideRows > 128 ? kTileByRows : 0) |
                    (x.t1 - x.t0 > 1 ? kTileMore : 0);
        head = x.h;
        t0 = tile * kWideTok;
        hi = walk.keys(x.b, x.rt);
        const int key = t0 + 16 * lane;
        if (lane < 8 && key < hi) {
          page = __ldg(p.table.pages + (kPrefix ? 0 : x.b * p.table.stride) + (key >> ps));
        }
        if (++tile == x.t1) {
          walk.next(x);
          tile = x.t0;
        }
      };
      Codes<kBits> w[8];
      float scale = 0.0f, even_k = 0.0f;
      const uint32_t fold_within = (is_v ? kFoldV : 14u) << 23;
      auto load = [&]() {
        loaded = more;
        info = info_next;
        if (!more) return;
        const bool gone = page < 0 || page >= p.cache.num_pages;
        const bool mine = lane < 8 && t0 + 16 * lane < hi;
        bad |= gone && mine;
        if (gone) page = -1;
        // The rows of a step follow those of the step before within a page.
        if (unlikely(__any_sync(0xFFFFFFFFu, gone && mine) || t0 + kWideTok > hi)) {   // some keys are not there: zeros
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int pg = __shfl_sync(0xFFFFFFFFu, page, i), t = t0 + 16 * i;
            const int64_t row = ((pg * p.cache.H + head) << ps) + (t & ((1 << ps) - 1)) + sub;
            w[i] = Codes<kBits>{};
            if (pg >= 0 && t + sub < hi) w[i].load(codes + row * kRow, blocks + row * 8);
          }
        } else {
          const uint8_t *row = codes, *block = blocks;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            if (i == 0 || ((16 * i) & ((1 << ps) - 1)) == 0) {               // warp-uniform
              const int pg = __shfl_sync(0xFFFFFFFFu, page, i);
              const int64_t at = ((pg * p.cache.H + head) << ps) + (i == 0 ? t0 & ((1 << ps) - 1) : 0) + sub - 16 * i;
              row = codes + at * kRow;
              if constexpr (kBits == 4) block = blocks + at * 8;
            }
            w[i].load(row + i * 16 * kRow, block + i * 16 * 8);
          }
        }
        const int pg = __shfl_sync(0xFFFFFFFFu, page, scale_key >> 4), t = t0 + scale_key;
        scale = 0.0f;
        if (pg >= 0 && t < hi) scale = __ldg(scales + (((pg * p.cache.H + head) << ps) + (t & ((1 << ps) - 1))));
      };
      ask();
      load();
      ask();
      int it = 0;
      for (; loaded; ++it) {
        const int s = it & 1, round = it >> 1;
        // In 4 bits a warp's 32 keys get the largest of their scales, and the values the
        // rest, where that is a power of two for all of them, of K down to 2^-14, of V to
        // 2^-kFoldV: a weight that counts in a reference with more than its key's own scale leaves
        // as many bits fewer to the others (rows of zeros in V would count with any).  K's may
        // not be so large that it could not be multiplied by a row's factor first.
        uint32_t ratio = 0x3C003C00u;
        if constexpr (kBits == 4) {
          const uint32_t bits = __float_as_uint(scale);
          const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, bits), least = __reduce_min_sync(0xFFFFFFFFu, bits);
          const bool even = top < 0x7F800000u && least != 0u && top - least <= fold_within && !__any_sync(0xFFFFFFFFu, (bits & 0x7FFFFFu) != 0u);
          if (even) {
            ratio = ((15u << 10) - ((top - bits) >> 13)) * 0x10001u;
            scale = __uint_as_float(top);
          }
          if (is_v && lane == 0) s_even[1][it % kScaleSlots][warp & 3] = even ? scale : -1.0f;
          if (!is_v) even_k = even && scale * p.c_scale <= kLarge ? scale * p.c_scale : -1.0f;
        }
        // V's scales may be written before its stage is free: the tile that last
        // used the slot has been multiplied.
        if (is_v) {
          s_vs[it % kScaleSlots][scale_key] = scale;
          // Magnitudes compare as integers, infinities and NaN above all others.
          const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(scale) & 0x7FFFFFFFu);
          if (lane == 0) s_top[it % kScaleSlots][warp & 3] = __uint_as_float(min(top, 0x7F800000u));
          mbar_arrive(&bars.scales[it % kScaleSlots]);
        }
        if (unlikely(round > 0 && !__all_sync(0xFFFFFFFFu, wait(&empty[s], round - 1)))) break;
        uint8_t* to = dst + s * kTileBytes;
        if (!is_v) {
          s_ks[it % kScaleSlots][scale_key] = scale * p.c_scale;
          if (kBits == 4 && lane == 0) s_even[0][it % kScaleSlots][warp & 3] = even_k;
          mbar_arrive(&bars.scales[it % kScaleSlots]);
        }
        auto convert = [&](auto v) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t o[8];
            // Step i's row of this lane: its scale is with lane 4 i + sub % 4 of the warp.
            const uint32_t fold = kBits == 4 ? __shfl_sync(0xFFFFFFFFu, ratio, 4 * i + (sub & 3)) : 0u;
            w[i].template values<decltype(v)::value>(o, fold);
            *reinterpret_cast<uint4*>(to + i * 2048) = make_uint4(o[0], o[1], o[2], o[3]);
            *reinterpret_cast<uint4*>(to + i * 2048 + static_cast<int>(odd)) = make_uint4(o[4], o[5], o[6], o[7]);
          }
        };
        if (kBits == 8 && is_v)
          convert(std::true_type());
        else
          convert(std::false_type());
        if (tid == 0) s_info[is_v][s] = info;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        mbar_arrive(&full[s]);
        load();
        ask();
      }
      if (!loaded && (it < 2 || __all_sync(0xFFFFFFFFu, wait(&empty[it & 1], (it >> 1) - 1)))) {
        if (tid == 0) s_info[is_v][it & 1] = kTileEnd;
        mbar_arrive(&full[it & 1]);
      }
      if (bad) atomicExch(p.err, SAGE_DEVERR_BAD_PAGE);
    } else if (warp < 16) {
      more_registers<kRegsSoftmax>();
      // ------------------------------------------------- softmax, epilogue --
      const int t = (warp - 8) >> 2;                       // half
      const int quarter = warp & 3;                        // TMEM lanes of this warp
      const int trow = quarter * 32 + lane;
      const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
      const uint32_t tO = tmem + lanes + col_o(t);
      float* exchange = reinterpret_cast<float*>(smem + kSmemQ + kTileBytes) + trow;   // [channel][row], 64 channels
      int it = 0;                                          // key tiles of this CTA
      uint32_t done = 0, joined = 0;                       // score buffers (an even number) and exchanges of this half
      bool ok = true;
      while (x.left > 0 && ok) {
        const int hi = walk.keys(x.b, x.rt);
        const int n = x.t1 - x.t0;
        const int rows = min(kWideRows, p.rows - x.rt * kWideRows);
        const bool whole = walk.whole(x), by_rows = rows > 128;
        if (by_rows || t < n) {
          const int r = (by_rows ? t * 128 : 0) + trow, rr = x.rt * kWideRows + r;
          const bool valid = r < rows;
          const int lim = valid ? min(hi, walk.limit(x.b, rr)) : hi;
          const int lo = __reduce_min_sync(0xFFFFFFFFu, lim);
          // The warp's query rows, two at a time, 8 channels a lane: fp16 times a power
          // of two.  Thread `lane` keeps its row's factor.
          Row z;
          z.rk = 0.0f;
          {
            const bool store = by_rows || t == 0;
            const int pair = lane >> 4, chunk = lane & 15;
            const uint64_t own = valid ? reinterpret_cast<uint64_t>(walk.query(x, rr)) : 0;
            uint8_t* sQ = smem + kSmemQ + (by_rows ? t * kTileBytes : 0);
            uint4 w[16];                     // all on their way at once
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t src = __shfl_sync(0xFFFFFFFFu, own, 2 * i + pair);
              w[i] = make_uint4(0u, 0u, 0u, 0u);
              if (src != 0) w[i] = __ldg(reinterpret_cast<const uint4*>(src) + chunk);
            }
            // The largest magnitudes of 16 rows over 16 lanes: each step halves the rows that a
            // lane has in hand, until lane `chunk` has row 2 chunk + pair.
            uint32_t two[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              two[i] = max_u16x2(max_u16x2(w[i].x & 0x7FFF7FFFu, w[i].y & 0x7FFF7FFFu), max_u16x2(w[i].z & 0x7FFF7FFFu, w[i].w & 0x7FFF7FFFu));
#pragma unroll
            for (int d = 8; d > 0; d >>= 1) {
              const bool high = (lane & d) != 0;
#pragma unroll
              for (int i = 0; i < d; ++i) {
                const uint32_t give = high ? two[i] : two[i + d], keep = high ? two[i + d] : two[i];
                two[i] = max_u16x2(keep, __shfl_xor_sync(0xFFFFFFFFu, give, d));
              }
            }
            const uint32_t ex = row_exponent(max(two[0] & 0xFFFFu, two[0] >> 16));
            z.rk = __uint_as_float((254u - __shfl_sync(0xFFFFFFFFu, ex, ((lane & 1) << 4) | (lane >> 1))) << 23);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float up = __uint_as_float(__shfl_sync(0xFFFFFFFFu, ex, (lane & 16) | i) << 23);
              if (store) {
                const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
                uint32_t out[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                  const float2 a = unpack_bf16(u[k]);
                  out[k] = pack_f16(a.x * up, a.y * up);
                }
                *reinterpret_cast<uint4*>(sQ + tile_offset(quarter * 32 + 2 * i + pair, chunk)) = make_uint4(out[0], out[1], out[2], out[3]);
              }
            }
            if (store) {
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              mbar_arrive(&bars.q_full[t]);
              if (!by_rows && n > 1) mbar_arrive(&bars.q_full[2]);
            }
          }

          z.R = kLowest;
          z.D = 0.0f;
          z.f = 1.0f;
          z.l = make_float2(0.0f, 0.0f);
          int v = 0;                                       // of this half's nv score buffers
          const int nv = 2 * (by_rows ? n : (n - t + 1) / 2);
          auto before = [&]() {                            // the product of buffer v - 1 has ended
            const bool r2 = __all_sync(0xFFFFFFFFu, wait(&bars.pv_done[t][(v - 1) & 1], (done + v - 1) >> 1));
            tc_fence_after();
            return r2;
          };
          for (v = 0; v < nv; ++v) {
            const int j = by_rows ? v >> 1 : (v & ~1) + t, slot = (it + j) % kScaleSlots, sub = (v & 1) * kSub;
            // In this order: a half passes over tiles that are not its own, and only the
            // scores say that the slot's phase before this tile's has ended.  A tile's second
            // buffer finds the scales that its first has waited for.
            ok = wait(&bars.s_full[t][v & 1], (done + v) >> 1) && ((v & 1) != 0 || wait(&bars.scales[slot], (it + j) / kScaleSlots));
            if (unlikely(!(ok = __all_sync(0xFFFFFFFFu, ok)))) break;
            tc_fence_after();
            const uint32_t tS = tmem + lanes + col_s(t, 0) + sub;
            const int key0 = (x.t0 + j) * kWideTok + sub;
            const float4 top4 = *reinterpret_cast<const float4*>(s_top[slot]);
            const float top = fmaxf(fmaxf(fmaxf(top4.x, top4.y), fmaxf(top4.z, top4.w)), kTiny);
            Even ev;
            if constexpr (kBits == 4) {
              ev.k = *reinterpret_cast<const float4*>(s_even[0][slot]);
              ev.v = *reinterpret_cast<const float4*>(s_even[1][slot]);
            }
            // What is usual stands in a line and what is rare out of the way: with five kinds
            // of warps at work a jump waits some 100 cycles for its instructions.
            const float *kx = s_ks[slot] + sub, *vx = s_vs[slot] + sub;
            int c = 0;                                     // scores that are done
            const bool all_seen = key0 + kSub <= lo && top < INFINITY;
            bool usual = z.f == 1.0f;
            if constexpr (kBits == 4)
              usual = usual & (ev.least_k() > 0.0f) & (fabsf(z.R) <= kNear) & (z.rk <= kLarge) & ((z.l.x + z.l.y) * ev.least_v() >= kSmall);
            if (likely(all_seen && __all_sync(0xFFFFFFFFu, usual))) {
              if constexpr (kBits == 4) {
                c = weigh_even(tS, ev, z);
              } else {
#pragma unroll
                for (int i = 0; i < kSub; i += 32) {
                  uint32_t w[16];
                  float2 sum;
                  if (unlikely(__any_sync(0xFFFFFFFFu, weigh<false>(tS + i, kx + i, vx + i, top, 32, z, w, sum)))) break;
                  z.l = fadd2v(z.l, sum);
                  tmem_st16(tS + i / 2, w);
                  c = i + 32;
                }
              }
            }
#pragma unroll 1
            for (; c < kSub && ok; c += 32) {
              const int left = lim - key0 - c;
              uint32_t w[16];
              float2 sum;
              while (true) {
                bool far;
                if (!all_seen || __any_sync(0xFFFFFFFFu, z.f != 1.0f))   // warp-uniform
                  far = weigh<true>(tS + c, kx + c, vx + c, top, left, z, w, sum);
                else
                  far = weigh<false>(tS + c, kx + c, vx + c, top, left, z, w, sum);
                if (!__any_sync(0xFFFFFFFFu, far)) break;
                float alpha;
                if (!__any_sync(0xFFFFFFFFu, move_references(tS + c, kx + c, vx + c, left, far, z, alpha))) break;   // in range as it is
                if (v > 0) ok = before();
                if (!ok) break;
                rescale(tO, tS, v > 0, c > 0, alpha);
              }
              z.l = fadd2v(z.l, sum);
              tmem_st16(tS + c / 2, w);
            }
            if (unlikely(!ok)) break;
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&bars.p_full[t][v & 1]);
          }
          ok = ok && before();
          if (!ok) break;
          done += nv;
          float L = z.l.x + z.l.y;
          const bool join = !by_rows && n > 1;
          if (join && t == 1) {
            // Half 1 hands over its rows' R, L, D and sums, 64 channels at a time.
            s_half[trow] = make_float4(z.R, L, z.D, 0.0f);
            for (int k = 0; k < 2 && ok; ++k) {
#pragma unroll 1
              for (int c = 0; c < 2; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + 64 * k + 32 * c, o);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) exchange[(32 * c + i) * 128] = __uint_as_float(o[i]);
              }
              mbar_arrive(&bars.half_full);
              ok = __all_sync(0xFFFFFFFFu, wait(&bars.half_read, joined++));
            }
          } else {
            float a0 = 1.0f, a1 = 0.0f;
            const float inv_none = whole && !p.keep ? 1.0f : 0.0f;   // written out, or to the workspace
            const int64_t at = static_cast<int64_t>(walk.slot(x)) * p.slot_rows + r;
            const int tok = rr / p.G, hq = x.h * p.G + rr % p.G;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
              if (join && (c & 1) == 0) {
                ok = __all_sync(0xFFFFFFFFu, wait(&bars.half_full, joined));
                if (!ok) break;
                if (c == 0) {
                  const float4 other = s_half[trow];
                  const float to = fmaxf(z.R, other.x), r0 = z.R - to, r1 = other.x - to;
                  const float top = fmaxf(r0 + z.D, r1 + other.z);
                  L = L * ex2_approx(r0) + other.y * ex2_approx(r1);
                  a0 = ex2_approx(r0 + (z.D - top));
                  a1 = ex2_approx(r1 + (other.z - top));
                  z.R = to;
                  z.D = top;
                }
              }
              const float half = scale2(z.D), inv = L == 0.0f ? 0.0f : half / L;
              uint32_t u[32];
              tmem_ld32(tO + 32 * c, u);
              tmem_ld_wait();
              float o[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                o[i] = __uint_as_float(u[i]);
                if (join) o[i] = o[i] * a0 + exchange[(32 * (c & 1) + i) * 128] * a1;
              }
              if (join && (c & 1) == 1) {
                mbar_arrive(&bars.half_read);
                ++joined;
              }
              if (valid && inv_none != 0.0f) {
                uint16_t* dst = p.out + ((static_cast<int64_t>(x.b) * p.Sq + tok) * p.Hq + hq) * kHeadDim + 32 * c;
#pragma unroll
                for (int i = 0; i < 32; i += 16)
                  store32(dst + i, pack_bf16(o[i] * half * inv, o[i + 1] * half * inv), pack_bf16(o[i + 2] * half * inv, o[i + 3] * half * inv),
                          pack_bf16(o[i + 4] * half * inv, o[i + 5] * half * inv), pack_bf16(o[i + 6] * half * inv, o[i + 7] * half * inv),
                          pack_bf16(o[i + 8] * half * inv, o[i + 9] * half * inv), pack_bf16(o[i + 10] * half * inv, o[i + 11] * half * inv),
                          pack_bf16(o[i + 12] * half * inv, o[i + 13] * half * inv), pack_bf16(o[i + 14] * half * inv, o[i + 15] * half * inv));
              } else if (valid) {
                float* dst = p.part_o + at * kHeadDim + 32 * c;
                const uint32_t* v = reinterpret_cast<const uint32_t*>(o);
#pragma unroll
                for (int i = 0; i < 32; i += 8)
                  store32(dst + i, v[i], v[i + 1], v[i + 2], v[i + 3], v[i + 4], v[i + 5], v[i + 6], v[i + 7]);
              }
            }
            if (valid && inv_none != 0.0f) {
              if (p.lse != nullptr)
                p.lse[(static_cast<int64_t>(x.b) * p.Hq + hq) * p.Sq + tok] = L == 0.0f ? -INFINITY : (z.R + log2f(L)) * kLn2;
            } else if (valid) {
              p.part_ml[at] = make_float4(z.R, L, z.D, 0.0f);
            }
          }
          tc_fence_before();                               // O may be written again
        }
        if (warp == 8 && lane == 0) walk.tell(x, s_end, s_per);
        it += n;
        walk.next(x);
      }
      // After a wait that gave up: the merge kernel reads every unit's entry.
      if (warp == 8 && lane == 0) {
        for (; x.left > 0; walk.next(x)) walk.tell(x, s_end, s_per);
      }
    } else {
      fewer_registers<kRegsIssue>();
      if (lane == 0) {
        // ------------------------------------------------------------ issue --
        // One thread for each product of each half, so that none waits for
        // another's operands.  Buffer v of half t: 64 keys, v & 1 of key tile v / 2,
        // or of key tile 2 (v / 2) + t.
        const int t = warp & 1;
        const bool is_pv = warp >= 18;
        constexpr uint32_t kIdescQK = make_idesc_f32acc(128, kSub, 0, 0);                  // F16 x F16
        constexpr uint32_t kIdescPV = make_idesc_f32acc(128, 128, 0, 0) | (1u << 16);      // F16 x F16, B's outer index summed
        const uint32_t q_lo = sw128_desc_lo(smem_addr(smem + kSmemQ));
        const uint32_t k_lo = sw128_desc_lo(smem_addr(smem + kSmemK));
        // V: 64-channel halves kHalf bytes apart, groups of eight keys 1024.
        const uint32_t v_lo = sw128_desc_lo(smem_addr(smem + kSmemV)) | ((kHalf >> 4) << 16);
        uint64_t* full = is_pv ? bars.v_full : bars.k_full;
        uint64_t* empty = is_pv ? bars.v_empty : bars.k_empty;
        const int* info = s_info[is_pv];
        uint32_t done = 0, seen = 0, seen_odd = 0;         // score buffers of this half; its Q tiles, by rows and not
#pragma unroll 1
        for (int g = 0;; ++g) {
          const int s = g & 1;
          if (!wait(&full[s], g >> 1)) break;
          const int tile = *const_cast<const volatile int*>(&info[s]);
          if ((tile & kTileEnd) != 0) break;
          // The scales of the tile two before have been there for long; with them, since
          // scales come in order, the last phase of this tile's slot has ended, and a
          // softmax that has the scores waits for the right one.  (A wait for a parity
          // tells a phase from the next one alone.)  These threads see every tile, and
          // no slot is used again before they have freed a stage behind it.
          if (!is_pv && g >= 2 && !wait(&bars.scales[(g - 2) % kScaleSlots], (g - 2) / kScaleSlots)) break;
          const bool by_rows = (tile & kTileByRows) != 0;
          // Each of Q's barriers is waited for by one thread in every one of its phases,
          // so that it is never two phases ahead of that thread.
          if (!is_pv && (tile & kTileOf) == 0) {
            bool ok = true;
            if (t == 0)
              ok = wait(&bars.q_full[0], seen++);
            else if (by_rows)
              ok = wait(&bars.q_full[1], seen++);
            else if ((tile & kTileMore) != 0)
              ok = wait(&bars.q_full[2], seen_odd++);
            if (!ok) break;
          }
          if (!by_rows && ((tile & kTileOdd) != 0) != (t == 1)) {   // the other half's tile
            // A run of segments of one tile frees K's stages without half 1: its
            // softmax must not fall behind the scales.
            if (!is_pv && (tile & kTileMore) == 0 && done > 0 && !wait(&bars.pv_done[t][(done - 1) & 1], (done - 1) >> 1)) break;
            mbar_arrive(&empty[s]);
            continue;
          }
          const bool fresh = (tile & kTileOf) == 0 || (!by_rows && (tile & kTileOf) == 1);   // this half's first
          bool ok = true;
#pragma unroll 1
          for (int sub = 0; sub < 2; ++sub, ++done) {
            const uint32_t buf = tmem + col_s(t, 0) + sub * kSub;
            if (is_pv) {
              if (!(ok = wait(&bars.p_full[t][sub], done >> 1))) break;
              tc_fence_after();
              const uint32_t b0 = v_lo + s * (kTileBytes >> 4) + sub * (kSub * 128 >> 4);
#pragma unroll
              for (int k = 0; k < kSub / 16; ++k)
                mma_f16_ts(tmem + col_o(t), buf + 8 * k, b0 + k * (2048 >> 4), kSw128DescHi, kIdescPV, !fresh || sub > 0 || k > 0);
              mma_commit(&bars.pv_done[t][sub]);
            } else {
              // The buffer's last weights have been used.
              if (done >= 2 && !(ok = wait(&bars.pv_done[t][sub], (done - 2) >> 1))) break;
              tc_fence_after();
              const uint32_t a0 = q_lo + (by_rows ? t : 0) * (kTileBytes >> 4);
              const uint32_t b0 = k_lo + s * (kTileBytes >> 4) + sub * (kSub * 128 >> 4);
#pragma unroll
              for (int k = 0; k < 8; ++k) {
                const uint32_t off = ((k >> 2) * kHalf + (k & 3) * 32) >> 4;
                mma_f16_ss(buf, a0 + off, b0 + off, kIdescQK, k > 0);
              }
              mma_commit(&bars.s_full[t][sub]);
            }
          }
          if (!ok) break;
          mma_commit(&empty[s]);
        }
        // Every product has to end before TMEM can be released.
        mma_commit(&bars.drain[warp - 16]);
        int local_abort = 0;
        (void)mbar_wait_inline(&bars.drain[warp - 16], 0, &local_abort, p.err, p.timeout_ns);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 16) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  // The merge kernel waits for this grid alone: this grid has to end after the
  // one before it, beside which it may have run.
  if constexpr (kPrefix) asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

cudaError_t launch_wide(const Params& p, bool prefix, bool beside, unsigned ctas, cudaStream_t stream) {
  auto go = [&](auto kernel) {
    static std::atomic<uint64_t> allowed[2 * 2];       // for each kernel
    cudaError_t e = allow_smem(kernel, kSmemBytes, allowed[(p.cache.bits == 8 ? 0 : 2) + prefix]);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = stream;
    // beside: the launch before is this call's, and nothing of it is needed.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  };
  if (p.cache.bits == 8) return prefix ? go(cache_attn_wide_kernel<true, 8>) : go(cache_attn_wide_kernel<false, 8>);
  return prefix ? go(cache_attn_wide_kernel<true, 4>) : go(cache_attn_wide_kernel<false, 4>);
}

}  // namespace sage::cache
