// cache_attention.cu -- attention of a sequence's newest tokens over the
// paged quantised cache, and over a prefix that all sequences share (sm_103a).
//
// Per query row i (one query head of one new token), over the cached keys j it
// sees, with kc, vc the codes and sk, sv the scales of key j's row:
//
//   x_j = (q_i . kc_j) * softmax_scale * log2 e * sk_j
//   L   = sum 2^(x_j - m),   lse = ln 2 * (m + log2 L)
//   out = sum 2^(x_j - m) sv_j vc_j / L      (0, and lse = -inf, if no key is seen)
//
// for any reference m near the largest x_j.  The query heads that share a
// key/value head are rows of one tile, so the cache is read once for all of
// them.  A row's weights of V have a reference of their own, m + d, some 8 below the
// largest x_j + log2 sv_j: the products are formed from 2^((x_j - m) + (log2 sv_j - d)),
// below 2^15 whatever the scales of V are, in fp16.  The largest weight is 2^8 or more,
// so that every weight down to 2^-22 of it is rounded by 2^-11 of itself at most, and
// those below by 2^-33 of the largest (bf16's step is eight times as wide; with the
// largest weight at 1, 65536 equal weights of 2^-18.7 lose 1% of their sum).  Then
// out = 2^d / L * sum.  Scores come into the weights by their differences alone, as in
// L: where they are so large that log2 sv is nothing to them, both still agree.
//
// Three kernels share the work.  cache_attn_kernel (up to 16 rows to a key/value head)
// is bound by HBM, 264 bytes a key: one token of 65536 keys x 24 heads 71.7 us, 5.8 TB/s,
// 0.85 of the measured copy rate; 48 ragged sequences of up to 16384 keys x 8 heads
// 116.9 us, 0.87.  What is left is the start of each CTA's ring and the merge launch.
// cache_attn_cluster_kernel takes what is too small for that, cache_attention_wide.cu
// more rows.
//
// Q enters as fp16 times a power of two that puts the row's largest magnitude
// in [2^14, 2^15), and K's integer codes are exact in fp16, so that the
// products of Q and K are exact but for values 2^-28 below the row's largest.
//
// Of a cache in 4 bits kc and vc are code times block scale, E2M1 x E4M3, six significant
// bits between 2^-10 and 2688: exact in fp16 too, at one product for two values.  With 152 bytes a
// key the instructions are the bound, 350 for 16 keys of a warp, of which conversion and
// scaling are 130: while warps attend 0.93 of the issue slots are taken (0.60 over the whole
// launch: a tile is 2250 clocks of that and 480 of waiting for the next).  One token of 65536
// keys x 24 heads 53.7 us, 4.5 TB/s, 48 ragged sequences 99.4 us, 0.68 of the copy rate.
// Without the arithmetic the same copies take 42 us.
#include <algorithm>
#include <climits>
#include <cmath>
#include <type_traits>
#include <cuda_runtime.h>

#include "cache_attention.cuh"

namespace sage {

using namespace cache;

namespace {

// Keys per tile.  In 4 bits a warp's work on 16 of them is done twice before the next
// wait (65536 keys x 24 heads: 62 us with 64, 54 with 128).
__host__ __device__ constexpr int tok_of(int bits) { return bits == 8 ? 64 : 128; }
// Of a unit, in tiles (of 64 keys, 1, 4 and 6: the same within 1%).
__host__ __device__ constexpr int cost_of(int bits) { return bits == 8 ? 2 : 1; }
constexpr int kConsumers = 4;                             // warps that compute, a quarter of a tile's keys each
constexpr int kThreads = (kConsumers + 1) * 32;           // and one that copies
// A tile as it stands in shared memory, of a cache of kBits.
template <int kBits>
struct Tile {
  static constexpr int kTok = tok_of(kBits);
  static constexpr uint32_t kRow = kHeadDim * kBits / 8;            // bytes of a row's codes
  static constexpr uint32_t kOffV = kTok * kRow;
  static constexpr uint32_t kOffKs = 2 * kTok * kRow;
  static constexpr uint32_t kOffVs = kOffKs + kTok * 4;
  static constexpr uint32_t kOffKb = kOffVs + kTok * 4;             // 4 bits: block scales, eight a row
  static constexpr uint32_t kOffVb = kOffKb + kTok * 8;
  static constexpr uint32_t kBytes = kBits == 8 ? kOffKb : kOffVb + kTok * 8;
};
constexpr uint32_t kMergeBytes = kConsumers * 8 * kHeadDim * 4;
constexpr int kClusterKeys = 1024;                        // most keys of an SM slot, in clusters
constexpr int kMaxCtas = 3 * kSms;                        // CTAs of a launch: three on each SM
// As many as the registers of NT times 8 query rows allow without spilling much
// (65536 keys x 24 heads, one row: three 74 us, two 79).
__host__ __device__ constexpr int ctas_per_sm(int nt) { return nt == 1 ? 3 : 2; }
// Tiles in flight: 9 or 8 on an SM, 135 KB or more; in 4 bits 6 or 8, 114 KB or more.
__host__ __device__ constexpr int stages_of(int nt, int bits) { return bits == 8 ? (nt == 1 ? 3 : 4) : (nt == 1 ? 2 : 4); }
template <int kBits>
constexpr uint32_t smem_of(int nt) { return stages_of(nt, kBits) * Tile<kBits>::kBytes + kMergeBytes + 8 * nt * kHeadDim * 2; }
constexpr float kFar = 32768.0f, kFarLog2 = 15.0f;        // most of a weight (fp16: 65504)
constexpr float kAbove = 8.0f;                            // a weights' reference that moves goes so far below the largest
constexpr float kLeast = -160.0f;                         // of d: scales of V are 0 or 2^-149 at least

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two E4M3 codes in the low or high half of a word -> a pair of fp16.
__device__ __forceinline__ uint32_t v_codes_f16_lo(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
  return r;
}
__device__ __forceinline__ uint32_t v_codes_f16_hi(uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, h;\n\t}" : "=r"(r) : "r"(w));
  return r;
}

// Untiled copy global -> shared, completion counted on `bar` in bytes.  Both
// addresses and the size are multiples of 16.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(src), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ void consumer_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kConsumers * 32) : "memory"); }

// Transpose of an 8 x 8 matrix of 16-bit values, two to a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// A tile's run of keys is copied in parts by as many lanes: K, V and, in 8 bits, their
// scales.  A bulk copy costs an SM some 60 ns however small it is (65536 keys x 24 heads
// in 4 bits, copies alone: six a tile 58 us, four 49, two 38), so that the scales of 4
// bits, 1.5 of 9.5 KB, go by 16 bytes a lane instead (copy_scales).
template <int kBits>
constexpr int kPartBits = kBits == 8 ? 2 : 1;
template <int kBits>
constexpr uint32_t kBulkBytes = Tile<kBits>::kRow * 2 + (kBits == 8 ? 8 : 0);   // of a key
template <int kBits>
constexpr uint32_t kFullCount = kBits == 8 ? 1 : 33;     // arrivals that make a tile full
template <int kBits>
__device__ __forceinline__ void copy_part(const CacheView& cache, int part, uint32_t st, uint32_t bar, int64_t row, int o, int run) {
  using T = Tile<kBits>;
  if (part == 0)
    bulk_load(st + o * T::kRow, cache.k_codes + row * T::kRow, run * T::kRow, bar);
  else if (part == 1)
    bulk_load(st + T::kOffV + o * T::kRow, cache.v_codes + row * T::kRow, run * T::kRow, bar);
  else if (part == 2)
    bulk_load(st + T::kOffKs + o * 4, cache.k_scale + row, run * 4, bar);
  else
    bulk_load(st + T::kOffVs + o * 4, cache.v_scale + row, run * 4, bar);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// The block scales and scales of the 4-bit tile of keys first .. first + 127, those before
// hi; every lane counts for `bar` when its copies have landed.  `page`: of run i of the
// tile in lane 2i.  The whole warp together.
__device__ __forceinline__ void copy_scales(const CacheView& cache, uint32_t st, uint32_t bar, int page, int h, int first, int hi) {
  using T = Tile<4>;
  const int lane = threadIdx.x & 31, ps = cache.page_shift, shift = min(7, ps), mask = (1 << ps) - 1;
  auto row_of = [&](int key) {
    const int pg = __shfl_sync(0xFFFFFFFFu, page, (key >> shift) << 1);
    return static_cast<uint32_t>(((pg * cache.H + h) << ps) + ((first + key) & mask));    // below 2^31, as all rows are
  };
#pragma unroll
  for (int i = 0; i < 2; ++i) {              // two keys a lane
    const int key = 64 * i + 2 * lane;
    const uint64_t row = row_of(key);
    if (first + key < hi) {
      copy16(st + T::kOffKb + key * 8, cache.k_block + row * 8);
      copy16(st + T::kOffVb + key * 8, cache.v_block + row * 8);
    }
  }
  const int key = 4 * lane;                  // four
  const uint64_t row = row_of(key);
  if (first + key < hi) {
    copy16(st + T::kOffKs + key * 4, cache.k_scale + row);
    copy16(st + T::kOffVs + key * 4, cache.v_scale + row);
  }
  asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar) : "memory");
}

// What a warp holds of a unit's query rows.  Lane (r, c): queries 2c and 2c + 1 of
// each eight in the arrays with [2], column r (a query) of the products' B in q.
template <int NT>
struct QueryRows {
  uint32_t q[NT][8][2];
  float rk[NT][2];           // the row's factor
  int lim[NT][2];            // keys that the row sees
  float o[NT][8][4];         // channels 16r + 2j + e / 2, queries 2c + e % 2
  float m[NT][2], d[NT][2], l[NT][2];
};

// Row r of K's products is key keyrow(r) of 16: in 4 bits keys 2 and 3 change places, and
// 6 and 7, so that the lanes of a load of V, 64 bytes a key, meet in fewer banks.
template <int kBits>
__device__ __forceinline__ int keyrow(int r) { return kBits == 8 ? r : r ^ ((r >> 1) & 1); }

// Scores of 16 keys, whose rows begin at row `at` of the tile at st, before any
// factor: sc[a][e] is key keyrow(r) + 8 (e / 2), query 2c + e % 2.
template <int NT>
__device__ __forceinline__ void scores8(const QueryRows<NT>& z, const uint8_t* st, int at, int r, int c, float (&sc)[NT][4]) {
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[a][e] = 0.0f;
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const uint8_t* kp = st + (at + r) * kHeadDim + c * 32 + half * 16;
    const uint4 k0 = *reinterpret_cast<const uint4*>(kp);
    const uint4 k1 = *reinterpret_cast<const uint4*>(kp + 8 * kHeadDim);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      uint32_t ka[4];
      k_codes_f16(reinterpret_cast<const uint32_t*>(&k0)[i], ka[0], ka[2]);
      k_codes_f16(reinterpret_cast<const uint32_t*>(&k1)[i], ka[1], ka[3]);
#pragma unroll
      for (int a = 0; a < NT; ++a) mma_f16(sc[a], ka, z.q[a][half * 4 + i][0], z.q[a][half * 4 + i][1]);
    }
  }
}

// The same from 4 bits: a lane's 32 channels of a key are 16 bytes and two blocks.  The
// products of each block add up by themselves, two chains half as long.
template <int NT>
__device__ __forceinline__ void scores4(const QueryRows<NT>& z, const uint8_t* st, int at, int r, int c, float (&sc)[NT][4]) {
  using T = Tile<4>;
  float more[NT][4];
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[a][e] = more[a][e] = 0.0f;
  uint4 kw[2];
  uint32_t sb[2][2];
#pragma unroll
  for (int n = 0; n < 2; ++n) {
    const int key = at + keyrow<4>(r) + 8 * n;
    kw[n] = *reinterpret_cast<const uint4*>(st + key * T::kRow + c * 16);
    uint32_t two;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(two) : "h"(*reinterpret_cast<const uint16_t*>(st + T::kOffKb + key * 8 + 2 * c)));
    sb[n][0] = __byte_perm(two, two, 0x1010);
    sb[n][1] = __byte_perm(two, two, 0x3232);
  }
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const int i = (w >> 1) | (w & 1) << 1;         // words 0, 2, 1, 3: products 2i and 2i + 1
    uint32_t h0[4], h1[4];
    e2m1x8_f16(reinterpret_cast<const uint32_t*>(&kw[0])[i], h0);
    e2m1x8_f16(reinterpret_cast<const uint32_t*>(&kw[1])[i], h1);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h0[j] = mul_f16x2(h0[j], sb[0][i >> 1]);
      h1[j] = mul_f16x2(h1[j], sb[1][i >> 1]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t ka[4] = {h0[2 * j], h1[2 * j], h0[2 * j + 1], h1[2 * j + 1]};
#pragma unroll
      for (int a = 0; a < NT; ++a) mma_f16(i < 2 ? sc[a] : more[a], ka, z.q[a][2 * i + j][0], z.q[a][2 * i + j][1]);
    }
  }
#pragma unroll
  for (int a = 0; a < NT; ++a)
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[a][e] += more[a][e];
}

// O^T += V^T P^T of 16 keys; some: some of them are keys that no row sees.
template <int NT>
__device__ __forceinline__ void values8(QueryRows<NT>& z, const uint8_t* st, int at, int t0, int hi, int r, int c,
                                        const uint32_t (&pb)[NT][2]) {
  uint4 vw[4];
  const uint8_t* vp = st + Tile<8>::kOffV + (at + 2 * c) * kHeadDim + r * 16;
#pragma unroll
  for (int k = 0; k < 4; ++k)         // keys 2c, 2c + 1, 2c + 8, 2c + 9
    vw[k] = *reinterpret_cast<const uint4*>(vp + ((k >> 1) * 8 + (k & 1)) * kHeadDim);
  if (t0 + 16 > hi) {                 // codes behind the last key may be anything, NaN too
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (t0 + 2 * c + (k >> 1) * 8 + (k & 1) >= hi) vw[k] = make_uint4(0u, 0u, 0u, 0u);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t w0 = reinterpret_cast<const uint32_t*>(&vw[0])[i], w1 = reinterpret_cast<const uint32_t*>(&vw[1])[i];
    const uint32_t w2 = reinterpret_cast<const uint32_t*>(&vw[2])[i], w3 = reinterpret_cast<const uint32_t*>(&vw[3])[i];
    const uint32_t a01 = __byte_perm(w0, w1, 0x5140), b01 = __byte_perm(w0, w1, 0x7362);
    const uint32_t a23 = __byte_perm(w2, w3, 0x5140), b23 = __byte_perm(w2, w3, 0x7362);
    const uint32_t va[4] = {v_codes_f16_lo(a01), v_codes_f16_hi(a01), v_codes_f16_lo(a23), v_codes_f16_hi(a23)};
    const uint32_t vb[4] = {v_codes_f16_lo(b01), v_codes_f16_hi(b01), v_codes_f16_lo(b23), v_codes_f16_hi(b23)};
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      mma_f16(z.o[a][2 * i], va, pb[a][0], pb[a][1]);
      mma_f16(z.o[a][2 * i + 1], vb, pb[a][0], pb[a][1]);
    }
  }
}

// The same from 4 bits: a lane's 16 channels of a key are eight bytes and one block.
// Bytes of the codes of keys A and B, even channels in one word and odd ones in
// another, are the pairs that the products take; so are the scales.
template <int NT>
__device__ __forceinline__ void values4(QueryRows<NT>& z, const uint8_t* st, int at, int t0, int hi, int r, int c,
                                        const uint32_t (&pb)[NT][2]) {
  using T = Tile<4>;
  uint2 vw[4];
  uint32_t sv[4];
  const uint8_t* vp = st + T::kOffV + at * T::kRow + r * 8;
  const uint8_t* vb = st + T::kOffVb + at * 8 + r;
#pragma unroll
  for (int k = 0; k < 4; ++k) {       // the keys of rows 2c, 2c + 1, 2c + 8, 2c + 9 of K's products
    const int key = (k >> 1) * 8 + keyrow<4>(2 * c + (k & 1));
    vw[k] = *reinterpret_cast<const uint2*>(vp + key * T::kRow);
    sv[k] = vb[key * 8];
  }
  if (t0 + 16 > hi) {                 // scales behind the last key may be anything, NaN too; codes are finite
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (t0 + (k >> 1) * 8 + keyrow<4>(2 * c + (k & 1)) >= hi) sv[k] = 0u;
  }
  uint32_t s2[2];
#pragma unroll
  for (int k = 0; k < 2; ++k)
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(s2[k]) : "h"(static_cast<uint16_t>(sv[2 * k] | sv[2 * k + 1] << 8)));
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t even[2][4], odds[2][4];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t w0 = i == 0 ? vw[2 * k].x : vw[2 * k].y, w1 = i == 0 ? vw[2 * k + 1].x : vw[2 * k + 1].y;
      e2m1x8_f16((w0 & 0x0F0F0F0Fu) | ((w1 << 4) & 0xF0F0F0F0u), even[k]);
      e2m1x8_f16(((w0 >> 4) & 0x0F0F0F0Fu) | (w1 & 0xF0F0F0F0u), odds[k]);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t va[4] = {mul_f16x2(even[0][j], s2[0]), mul_f16x2(odds[0][j], s2[0]), mul_f16x2(even[1][j], s2[1]),
                              mul_f16x2(odds[1][j], s2[1])};
#pragma unroll
      for (int a = 0; a < NT; ++a) mma_f16(z.o[a][4 * i + j], va, pb[a][0], pb[a][1]);
    }
  }
}

// 16 kN keys, t0 and on, which stand at row `at` and on of the tile at st.  hi: keys
// that some row sees; lo: keys that all see.
template <int NT, int kBits, int kN>
__device__ __forceinline__ void attend(QueryRows<NT>& z, const uint8_t* st, float c_scale, int t0, int at, int r, int c, int hi,
                                       int lo) {
  using T = Tile<kBits>;
  float sc[kN][NT][4], lw[kN][NT][4], lv[kN][2];
  const int key = keyrow<kBits>(r);
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    if constexpr (kBits == 8)
      scores8<NT>(z, st, at + 16 * n, r, c, sc[n]);
    else
      scores4<NT>(z, st, at + 16 * n, r, c, sc[n]);
  }
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    float ks[2];                        // of keys `key` and key + 8; K's times softmax_scale * log2 e
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      ks[k] = *reinterpret_cast<const float*>(st + T::kOffKs + (at + 16 * n + k * 8 + key) * 4) * c_scale;
      lv[n][k] = lg2_approx(*reinterpret_cast<const float*>(st + T::kOffVs + (at + 16 * n + k * 8 + key) * 4));
    }
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        sc[n][a][e] = __fmul_rn(sc[n][a][e] * z.rk[a][e & 1], ks[e >> 1]);     // rk is a power of two: rounded once
        lw[n][a][e] = lv[n][e >> 1] - z.d[a][e & 1];
      }
    if (t0 + 16 * n + 16 > lo) {              // some row does not see all of these keys
#pragma unroll
      for (int a = 0; a < NT; ++a)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (t0 + 16 * n + key + 8 * (e >> 1) >= z.lim[a][e & 1]) {
            sc[n][a][e] = -INFINITY;
            lw[n][a][e] = 0.0f;         // the scale may be anything
          }
    }
  }
  bool over = false;
  float pl[kN][NT][4], pw[kN][NT][4];
#pragma unroll
  for (int n = 0; n < kN; ++n)
#pragma unroll
    for (int a = 0; a < NT; ++a)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float t = sc[n][a][e] - z.m[a][e & 1];
        pl[n][a][e] = ex2_approx(t);
        pw[n][a][e] = ex2_approx(t + lw[n][a][e]);
        over |= fmaxf(pl[n][a][e], pw[n][a][e]) > kFar;
      }
  // The references m and m + d need not be the maxima, only near them: they move
  // where a weight passes 2^15, which after the first keys is rare, and
  // otherwise no value crosses lanes.
  if (__any_sync(0xFFFFFFFFu, over)) {
#pragma unroll
    for (int a = 0; a < NT; ++a) {
      float alpha[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float mx = z.m[a][e];
#pragma unroll
        for (int n = 0; n < kN; ++n) mx = fmaxf(mx, fmaxf(sc[n][a][e], sc[n][a][e + 2]));
        float wx = -INFINITY;           // a masked key's is -inf or NaN
#pragma unroll
        for (int n = 0; n < kN; ++n) wx = fmaxf(wx, fmaxf((sc[n][a][e] - mx) + lv[n][0], (sc[n][a][e + 2] - mx) + lv[n][1]));
#pragma unroll
        for (int d = 4; d < 32; d <<= 1)
          larger(mx, wx, __shfl_xor_sync(0xFFFFFFFFu, mx, d), __shfl_xor_sync(0xFFFFFFFFu, wx, d));
        const float up = mx - z.m[a][e];
        float dn = z.d[a][e];
        if (up > kFarLog2 || up + (wx - dn) > kFarLog2)
          dn = fmaxf(fmaxf(wx - kAbove, dn - up), kLeast);
        else
          mx = z.m[a][e];             // a row's result is its own alone
        z.l[a][e] *= ex2_approx(z.m[a][e] - mx);
        alpha[e] = ex2_approx((z.m[a][e] - mx) + (z.d[a][e] - dn));
        z.m[a][e] = mx;
        z.d[a][e] = dn;
#pragma unroll
        for (int n = 0; n < kN; ++n)
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            const float t = sc[n][a][e + k] - mx;
            pl[n][a][e + k] = ex2_approx(t);
            pw[n][a][e + k] = t == -INFINITY ? 0.0f : ex2_approx(t + (lv[n][k >> 1] - dn));
          }
      }
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) z.o[a][j][e] *= alpha[e & 1];
    }
  }
#pragma unroll
  for (int n = 0; n < kN; ++n) {
    uint32_t pb[NT][2];
#pragma unroll
    for (int a = 0; a < NT; ++a) {
#pragma unroll
      for (int e = 0; e < 4; ++e) z.l[a][e & 1] += pl[n][a][e];
      // (key r, queries 2c, 2c + 1) -> (query r, keys 2c, 2c + 1)
      pb[a][0] = transpose8(pack_f16(pw[n][a][0], pw[n][a][1]));
      pb[a][1] = transpose8(pack_f16(pw[n][a][2], pw[n][a][3]));
    }
    if constexpr (kBits == 8)
      values8<NT>(z, st, at + 16 * n, t0 + 16 * n, hi, r, c, pb);
    else
      values4<NT>(z, st, at + 16 * n, t0 + 16 * n, hi, r, c, pb);
  }
}

// A warp's quarter of a tile.  With 16 rows its registers do for 16 keys at a time.
template <int NT, int kBits>
__device__ __forceinline__ void attend_quarter(QueryRows<NT>& z, const uint8_t* st, float c_scale, int t0, int at, int r, int c,
                                               int hi, int lo) {
  constexpr int kN = tok_of(kBits) / (16 * kConsumers), kStep = NT == 1 ? kN : 1;
#pragma unroll
  for (int n = 0; n < kN; n += kStep)
    if (t0 + 16 * n < hi) attend<NT, kBits, kStep>(z, st, c_scale, t0 + 16 * n, at + 16 * n, r, c, hi, lo);
}

// The unit's query rows (bf16 in shared memory) as a warp holds them, nothing attended
// to yet.
template <int NT>
__device__ __forceinline__ void load_queries(QueryRows<NT>& z, const uint8_t* queries, int rows, int r, int c) {
#pragma unroll
  for (int a = 0; a < NT; ++a) {
    uint4 raw[4];              // row r of these eight, a quarter of its channels
#pragma unroll
    for (int i = 0; i < 4; ++i)
      raw[i] = a * 8 + r < rows ? *reinterpret_cast<const uint4*>(queries + (a * 8 + r) * kHeadDim * 2 + c * 64 + i * 16)
                                : make_uint4(0u, 0u, 0u, 0u);
    const uint32_t* u = reinterpret_cast<const uint32_t*>(raw);
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < 16; ++i) top = max(top, max(u[i] & 0x7FFFu, (u[i] >> 16) & 0x7FFFu));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t ex = row_exponent(top);
    const float up = __uint_as_float(ex << 23);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      z.q[a][i >> 1][i & 1] = pack_f16(__uint_as_float(u[i] << 16) * up, __uint_as_float(u[i] & 0xFFFF0000u) * up);
    const float back = __uint_as_float((254u - ex) << 23);
#pragma unroll
    for (int e = 0; e < 2; ++e) z.rk[a][e] = __shfl_sync(0xFFFFFFFFu, back, (2 * c + e) * 4);
#pragma unroll
    for (int j = 0; j < 8; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) z.o[a][j][e] = 0.0f;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      z.m[a][e] = kLowest;
      z.d[a][e] = z.l[a][e] = 0.0f;
    }
  }
}

// What the warps' join takes in shared memory, one set a CTA.
struct JoinStats {
  float m[kConsumers][8], d[kConsumers][8], l[kConsumers][8];
};

// The four warps' parts of rows 8a .. 8a + 7, joined: this thread gets channels
// 8 (thread % 16) .. of row 8a + thread / 16 relative to m + d, and the row's m, L, d.
// `merge`: 8 rows of each warp.
template <int NT>
__device__ __forceinline__ float4 join_warps(QueryRows<NT>& z, int a, int rows, JoinStats& s, float4* merge, float4 (&sum)[2]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
#pragma unroll
    for (int d = 4; d < 32; d <<= 1) z.l[a][e] += __shfl_xor_sync(0xFFFFFFFFu, z.l[a][e], d);
    if (r == 0) {
      s.m[warp][2 * c + e] = z.m[a][e];
      s.d[warp][2 * c + e] = z.d[a][e];
      s.l[warp][2 * c + e] = z.l[a][e];
    }
  }
  consumer_sync();
  const int row = threadIdx.x >> 4, g = threadIdx.x & 15;
  // The largest m of a row, and the largest reference relative to it.
  auto refs = [&](int row, float& m, float& d) {
    m = s.m[0][row];
    d = s.d[0][row];
#pragma unroll
    for (int k = 1; k < kConsumers; ++k) larger(m, d, s.m[k][row], s.d[k][row]);
  };
  float m, d, L = 0.0f;
  refs(row, m, d);
#pragma unroll
  for (int k = 0; k < kConsumers; ++k) L += s.l[k][row] * ex2_approx(s.m[k][row] - m);
  // float4 i of channels 16r .. 16r + 15 stands at 4r + (i ^ c): the eight lanes of
  // a store fall into distinct banks.
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    if (a * 8 + 2 * c + e < rows) {
      float mr, dr;
      refs(2 * c + e, mr, dr);
      const float w = ex2_approx((z.m[a][e] - mr) + (z.d[a][e] - dr));
#pragma unroll
      for (int i = 0; i < 4; ++i)
        merge[(warp * 8 + 2 * c + e) * 32 + 4 * r + (i ^ c)] =
            make_float4(z.o[a][2 * i][e] * w, z.o[a][2 * i][e + 2] * w, z.o[a][2 * i + 1][e] * w, z.o[a][2 * i + 1][e + 2] * w);
    }
  }
  consumer_sync();
  sum[0] = sum[1] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (a * 8 + row < rows) {
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int at = g * 2 + e, idx = row * 32 + (at & ~3) + ((at & 3) ^ (row >> 1));
      sum[e] = merge[idx];
#pragma unroll
      for (int k = 1; k < kConsumers; ++k) {
        const float4 y = merge[k * 8 * 32 + idx];
        sum[e].x += y.x;
        sum[e].y += y.y;
        sum[e].z += y.z;
        sum[e].w += y.w;
      }
    }
  }
  return make_float4(m, L, d, 0.0f);
}

template <int NT, bool kPrefix, int kBits>
__global__ void __launch_bounds__(kThreads, ctas_per_sm(NT)) cache_attn_kernel(const Params p) {
  constexpr int R = 8 * NT, kStages = stages_of(NT, kBits);
  constexpr uint32_t kStageBytes = Tile<kBits>::kBytes;
  constexpr int kTok = tok_of(kBits), kCost = cost_of(kBits);
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kStages], empty[kStages], q_full, q_empty;
  __shared__ int abort_flag;
  __shared__ int s_len[kMaxBatch];
  __shared__ long long s_off[kPrefix ? 2 : kMaxBatch + 1];
  __shared__ JoinStats stats;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_v = &abort_flag;
  // The merge kernel (or the other part's launch) may be scheduled as soon as
  // there is room; it waits for this grid before it reads anything from it.
  asm volatile("griddepcontrol.launch_dependents;");

  const Walk<R, kTok, kCost, kPrefix> walk{p, s_len, s_off};
  walk.plan(s_len, s_off);
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], kFullCount<kBits>);
      mbar_init(&empty[s], kConsumers);
    }
    mbar_init(&q_full, 1);
    mbar_init(&q_empty, kConsumers);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();

  const long long total = s_off[walk.seqs()] * p.cache.H;
  const long long per = div_floor(total + gridDim.x - 1, gridDim.x);
  const long long f0 = blockIdx.x * per, f1 = min(total, f0 + per);
  if (!p.keep && threadIdx.x == 0) p.desc[blockIdx.x].w = 0;
  if (f0 < f1) {
    Place x = walk.locate(f0, static_cast<int>(f1 - f0));
    const uint32_t smem0 = smem_addr(smem);
    if (warp == kConsumers) {
      // ------------------------------------------------------------ copies --
      // A tile is 1, 2 or 4 runs of keys that lie together in a page; lane
      // 4i + k (in 4 bits 2i + k) copies part k of run i.  Every lane holds a
      // page number of the unit's table, reloaded for the next 32 pages.
      const int ps = p.cache.page_shift;
      const int run = min(kTok, 1 << ps), runs = kTok / run;
      const int my_run = lane >> kPartBits<kBits>, part = lane & ((1 << kPartBits<kBits>) - 1);
      int it = 0;
      bool bad = false, ok = true;
      uint32_t seg = 0;
      auto pages_of = [&](const Place& at, int first) {    // entry first + lane of the unit's row of the table
        const int32_t* row = p.table.pages + (kPrefix ? 0 : at.b * p.table.stride);
        return first + lane < p.table.width ? __ldg(row + first + lane) : -1;
      };
      int ahead = x.left > 0 ? pages_of(x, (x.t0 * kTok) >> ps) : -1;
      while (x.left > 0 && ok) {
        const int hi = walk.keys(x.b, x.rt);
        int base = (x.t0 * kTok) >> ps, cur = ahead, nxt = -1;
        if ((((x.t1 - 1) * kTok) >> ps) - base >= 32) nxt = pages_of(x, base + 32);
        Place after = x;                 // the next segment's pages are on their way during this one
        walk.next(after);
        if (after.left > 0) ahead = pages_of(after, (after.t0 * kTok) >> ps);
        // The unit's queries, once all warps have read the last unit's.
        const int rows = min(R, p.rows - x.rt * R);
        if (seg > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(&q_empty, (seg - 1) & 1, abort_v, p.err, p.timeout_ns))) break;
        if (lane == 0) mbar_arrive_expect_tx(&q_full, rows * kHeadDim * 2);
        __syncwarp();
        if (lane < rows)
          bulk_load(smem0 + kStages * kStageBytes + kMergeBytes + lane * kHeadDim * 2, walk.query(x, x.rt * R + lane),
                    kHeadDim * 2, smem_addr(&q_full));
        ++seg;
        for (int t = x.t0; t < x.t1; ++t, ++it) {
          const int t0 = t * kTok + my_run * run;
          if (((t * kTok) >> ps) - base >= 32) {
            base += 32;
            cur = nxt;
            nxt = pages_of(x, base + 32);
          }
          // The tile's pages are base .. base + 31: run <= page and a tile
          // begins at a multiple of 64 keys.
          int page = __shfl_sync(0xFFFFFFFFu, cur, ((t0 >> ps) - base) & 31);
          const bool live = my_run < runs && t0 < hi;
          if (live && (page < 0 || page >= p.cache.num_pages)) {
            bad = true;
            page = 0;        // a page that exists: the result is void, the read is not out of bounds
          }
          const int s = it % kStages, round = it / kStages;
          if (round > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], (round - 1) & 1, abort_v, p.err, p.timeout_ns))) {
            ok = false;
            break;
          }
          const int n_live = (min(kTok, hi - t * kTok) + run - 1) / run;   // <= 0 for a unit without keys
          if (lane == 0) mbar_arrive_expect_tx(&full[s], max(0, n_live) * run * kBulkBytes<kBits>);
          __syncwarp();
          if (live) {
            const int64_t r = ((static_cast<int64_t>(page) * p.cache.H + x.h) << ps) + (t0 & ((1 << ps) - 1));
            const uint32_t bar = smem_addr(&full[s]), st = smem0 + s * kStageBytes;
            const int o = my_run * run;
            copy_part<kBits>(p.cache, part, st, bar, r, o, run);
          }
          if constexpr (kBits == 4) copy_scales(p.cache, smem0 + s * kStageBytes, smem_addr(&full[s]), page, x.h, t * kTok, hi);
        }
        x = after;
      }
      if (bad) atomicExch(p.err, SAGE_DEVERR_BAD_PAGE);
      if (*abort_v) {   // let the copies in flight land before the CTA can exit
        for (int j = max(0, it - kStages); j < it; ++j) {
          int local_abort = 0;
          (void)mbar_wait(&full[j % kStages], (j / kStages) & 1, &local_abort, p.err, p.timeout_ns);
        }
        int local_abort = 0;
        if (seg > 0) (void)mbar_wait(&q_full, (seg - 1) & 1, &local_abort, p.err, p.timeout_ns);
      }
    } else {
      // ----------------------------------------------------------- compute --
      // Keys are the rows of the m16n8k16 products' A and queries the columns of
      // B, so that up to 8 queries cost 8 columns: S^T = K Q^T, then O^T = V^T
      // P^T.  Lane (r, c) = (lane / 4, lane % 4) holds rows r and r + 8 of A and of
      // the accumulator, column r of B, columns 2c and 2c + 1 of the
      // accumulator, and the summed indices 2c, 2c + 1, 2c + 8, 2c + 9.  The
      // order of a summed index is free as long as A and B agree, and so is that
      // of V's channels: in product i of K Q^T those are channels 32c + 4i .. + 3,
      // so that a lane's share of a key is 32 bytes that lie together, and rows r
      // and r + 8 of product j of V^T P^T are channels 16r + 2j and 16r + 2j + 1,
      // 16 bytes that lie together.
      const int r = lane >> 2, c = lane & 3;
      float4* merge = reinterpret_cast<float4*>(smem + kStages * kStageBytes);
      int it = 0;
      bool ok = true;
      const uint8_t* queries = smem + kStages * kStageBytes + kMergeBytes;
      for (uint32_t seg = 0; x.left > 0; ++seg) {
        const int hi = walk.keys(x.b, x.rt);
        const int rows = min(R, p.rows - x.rt * R);   // of this tile
        QueryRows<NT> z;
        int lo = INT_MAX;            // keys that every row sees
        ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(&q_full, seg & 1, abort_v, p.err, p.timeout_ns));
        load_queries<NT>(z, queries, rows, r, c);
#pragma unroll
        for (int a = 0; a < NT; ++a)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = x.rt * R + a * 8 + 2 * c + e;
            z.lim[a][e] = row < p.rows ? min(hi, walk.limit(x.b, row)) : hi;
            lo = min(lo, z.lim[a][e]);
          }
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_empty);
        lo = __reduce_min_sync(0xFFFFFFFFu, lo);

        for (int t = x.t0; t < x.t1; ++t, ++it) {
          const int s = it % kStages;
          ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(&full[s], (it / kStages) & 1, abort_v, p.err, p.timeout_ns));
          const int at = warp * (kTok / kConsumers);   // this warp's first key
          if (ok) attend_quarter<NT, kBits>(z, smem + s * kStageBytes, p.c_scale, t * kTok + at, at, r, c, hi, lo);
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[s]);
        }

        // The four warps' parts of the segment, 8 rows at a time.  A warp whose
        // wait gave up takes part in the barriers and writes nothing.
        const bool whole = walk.whole(x);
#pragma unroll
        for (int a = 0; a < NT; ++a) {
          if (a * 8 >= rows) break;
          float4 sum[2];
          const float4 mld = join_warps<NT>(z, a, rows, stats, merge, sum);
          const float m = mld.x, L = mld.y, d = mld.z;
          const int row = threadIdx.x >> 4, g = threadIdx.x & 15;   // 8 channels of a row a thread
          const int rr = x.rt * R + a * 8 + row;
          if (a * 8 + row < rows && !abort_flag) {
            if (whole && !p.keep) {
              const int t = rr / p.G, hq = x.h * p.G + rr % p.G;
              const float half = scale2(d), inv = L == 0.0f ? 0.0f : half / L;
              const uint4 w = make_uint4(pack_bf16(sum[0].x * half * inv, sum[0].y * half * inv),
                                         pack_bf16(sum[0].z * half * inv, sum[0].w * half * inv),
                                         pack_bf16(sum[1].x * half * inv, sum[1].y * half * inv),
                                         pack_bf16(sum[1].z * half * inv, sum[1].w * half * inv));
              *reinterpret_cast<uint4*>(p.out + ((static_cast<int64_t>(x.b) * p.Sq + t) * p.Hq + hq) * kHeadDim + g * 8) = w;
              if (p.lse != nullptr && g == 0)
                p.lse[(static_cast<int64_t>(x.b) * p.Hq + hq) * p.Sq + t] = L == 0.0f ? -INFINITY : (m + log2f(L)) * kLn2;
            } else {
              const int64_t at = static_cast<int64_t>(walk.slot(x)) * p.slot_rows + a * 8 + row;
              float4* dst = reinterpret_cast<float4*>(p.part_o + at * kHeadDim) + g * 2;
              dst[0] = sum[0];
              dst[1] = sum[1];
              if (g == 0) p.part_ml[at] = make_float4(m, L, d, 0.0f);
            }
          }
        }
        if (threadIdx.x == 0) walk.tell(x, f1, per);
        walk.next(x);
      }
    }
  }
  // The merge kernel waits for this grid alone: this grid has to end after the
  // one before it, beside which it may have run.
  if constexpr (kPrefix) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ---------------------------------------------------------------- cluster --

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// Every thread of the cluster; shared memory written before is seen by all after.
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// The address of this CTA's shared-memory `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ float4 load_cluster4(uint32_t addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
  return v;
}
// A row's parts, one (m, L, d) a lane, beside its m, d and L so far: the references
// move to the largest of all, and L with them; -> the factor of the sums so far, and
// each lane's L and factor in part.y and part.z.  The whole warp together.
__device__ __forceinline__ float take_in(float4& part, float& m, float& d, float& L) {
  float mx = m, dx = d;
  larger(mx, dx, part.x, part.z);
#pragma unroll
  for (int i = 16; i > 0; i >>= 1)
    larger(mx, dx, __shfl_xor_sync(0xFFFFFFFFu, mx, i), __shfl_xor_sync(0xFFFFFFFFu, dx, i));
  const float to = part.x - mx;
  L *= ex2_approx(m - mx);
  const float less = ex2_approx((m - mx) + (d - dx));
  part.y *= ex2_approx(to);
  part.z = ex2_approx(to + (part.z - dx));
  m = mx;
  d = dx;
  return less;
}

// The parts of a prefix's launch: closed form, since every unit has as many tiles.
struct PrefixParts {
  const float* o;
  const float4* ml;
  int R, slot_rows, n, cost, ctas;   // rows of a tile and of a slot, a unit's tiles and cost, CTAs
  long long per;                     // steps of a CTA
};

// The parts that hold row `pr` of the prefix's rows, key/value head h of H.
struct RowParts {
  int n, slot, row;
  __device__ RowParts(const PrefixParts& p, int pr, int h, int H) {
    row = pr % p.R;
    const int u = pr / p.R * H + h;
    const long long f = static_cast<long long>(u) * (p.n + p.cost) + p.cost;   // its first tile's step
    slot = static_cast<int>(div_floor(f, p.per));
    n = static_cast<int>(div_floor(f + p.n - 1, p.per)) - slot + 1;
    slot = n == 1 ? 2 * p.ctas + u : 2 * slot;
  }
  // Where part j stands among the slots' rows.
  __device__ int64_t at(const PrefixParts& p, int j) const {
    return static_cast<int64_t>(n == 1 ? slot : j == 0 ? slot + 1 : slot + 2 * j) * p.slot_rows + row;
  }
};

// What the cluster kernel finds before a sequence's own keys.
enum Before { kNothing, kPrefixTiles, kPrefixParts };

// Few units of short sequences: a cluster of up to eight CTAs takes a unit, its CTAs
// the key tiles in turn (the prefix's, if there is one, before the sequence's own), and
// they join their parts through one another's shared memory: one launch and no
// workspace where the kernel above takes two, or three behind a prefix.  A short prefix is
// then read once for each sequence, from L2; behind a longer one, multiplied for all
// sequences in a launch before (kPrefixParts), the join takes that launch's parts in
// and no merge kernel follows.  What bounds it is one chain of
// latencies: the length, the pages, the copies, the products, the join.
//
// kPerSm: CTAs on an SM, three, or four with a few registers spilled where that saves a
// second round of them (4 bits behind a prefix of 16384, 4 rows: 64 sequences x 8 heads 46
// us, of three on an SM 53; 56 sequences, one round either way, 46.8 and 43.9).
template <int ctas, Before kBefore, int kBits, int kPerSm>
__global__ void __cluster_dims__(ctas, 1, 1) __launch_bounds__(kThreads, kPerSm)
    cache_attn_cluster_kernel(const Params p, const int32_t* prefix_pages, const PrefixParts parts) {
  constexpr bool kPrefix = kBefore == kPrefixTiles;
  constexpr int R = 8, kStages = stages_of(1, kBits), kTok = tok_of(kBits);
  constexpr uint32_t kStageBytes = Tile<kBits>::kBytes;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ uint64_t full[kStages], empty[kStages], q_full;
  __shared__ int abort_flag;
  __shared__ JoinStats stats;
  __shared__ float4 s_ml[R];
  static_assert(R * kHeadDim * 4 <= kStages * kStageBytes, "a unit's part in the place of the tiles");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  volatile int* abort_v = &abort_flag;
  const int rank = static_cast<int>(cluster_rank());
  const int unit = blockIdx.x / ctas, h = unit % p.cache.H;
  const int rt = unit / p.cache.H % p.row_tiles, b = unit / p.cache.H / p.row_tiles;
  const int np = kPrefix ? (p.prefix_len + kTok - 1) / kTok : 0;      // tiles of the prefix
  const int len_raw = __ldg(p.lens + b);
  if (threadIdx.x == 32) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], kFullCount<kBits>);
      mbar_init(&empty[s], kConsumers);
    }
    mbar_init(&q_full, 1);
    abort_flag = 0;
    fence_mbarrier_init();
  }
  __syncthreads();
  const int row0 = rt * R, rows = min(R, p.rows - row0);
  // The parts are joined where the tiles were, behind the place of this CTA's result.
  constexpr uint32_t kMergeAt = kBits == 8 ? kStages * kStageBytes : R * kHeadDim * 4, kQueriesAt = kStages * kStageBytes + (kBits == 8 ? kMergeBytes : 0);
  static_assert(kBits == 8 || kMergeAt + kMergeBytes <= kStages * kStageBytes, "room for the parts");
  float4* merge = reinterpret_cast<float4*>(smem + kMergeAt);
  const uint8_t* queries = smem + kQueriesAt;
  const uint32_t smem0 = smem_addr(smem);

  if (warp == kConsumers) {
    // -------------------------------------------------------------- copies --
    const int ps = p.cache.page_shift;
    const int run = min(kTok, 1 << ps), runs = kTok / run;
    const int my_run = lane >> kPartBits<kBits>, part = lane & ((1 << kPartBits<kBits>) - 1);       // as in the kernel above
    if (lane == 0) mbar_arrive_expect_tx(&q_full, rows * kHeadDim * 2);
    __syncwarp();
    if (lane < rows)
      bulk_load(smem0 + kQueriesAt + lane * kHeadDim * 2,
                p.q + b * p.q_sb + ((row0 + lane) / p.G) * p.q_ss + (h * p.G + (row0 + lane) % p.G) * kHeadDim, kHeadDim * 2, smem_addr(&q_full));
    // The page of this lane's run of tile t, wherever the sequence ends: on its way
    // before its length is known.
    auto page_of = [&](int t) {
      const bool pre = kPrefix && t < np;
      const int at = ((pre ? t : t - np) * kTok + my_run * run) >> ps;
      const int width = pre ? ((p.prefix_len - 1) >> ps) + 1 : p.table.width;
      const int32_t* row = pre ? prefix_pages : p.table.pages + b * p.table.stride;
      return my_run < runs && at < width ? __ldg(row + at) : -1;
    };
    int next = page_of(rank);
    const int len = held(len_raw, p), n = np + (len + kTok - 1) / kTok;
    int it = 0;
    bool bad = false;
    for (int t = rank; t < n; t += ctas, ++it) {
      int page = next;
      if (t + ctas < n) next = page_of(t + ctas);
      const bool pre = kPrefix && t < np;
      const int first = (pre ? t : t - np) * kTok, hi = pre ? p.prefix_len : len;
      const int t0 = first + my_run * run;
      const bool live = my_run < runs && t0 < hi;
      if (live && (page < 0 || page >= p.cache.num_pages)) {
        bad = true;
        page = 0;        // a page that exists: the result is void, the read is not out of bounds
      }
      const int s = it % kStages, round = it / kStages;
      if (round > 0 && !__all_sync(0xFFFFFFFFu, mbar_wait(&empty[s], (round - 1) & 1, abort_v, p.err, p.timeout_ns))) break;
      const int n_live = (min(kTok, hi - first) + run - 1) / run;
      if (lane == 0) mbar_arrive_expect_tx(&full[s], n_live * run * kBulkBytes<kBits>);
      __syncwarp();
      if (live) {
        const int64_t r = ((static_cast<int64_t>(page) * p.cache.H + h) << ps) + (t0 & ((1 << ps) - 1));
        const uint32_t bar = smem_addr(&full[s]), st = smem0 + s * kStageBytes;
        const int o = my_run * run;
        copy_part<kBits>(p.cache, part, st, bar, r, o, run);
      }
      if constexpr (kBits == 4) copy_scales(p.cache, smem0 + s * kStageBytes, smem_addr(&full[s]), page, h, first, hi);
    }
    if (bad) atomicExch(p.err, SAGE_DEVERR_BAD_PAGE);
    if (*abort_v) {   // let the copies in flight land before the CTA can exit
      for (int j = max(0, it - kStages); j < it; ++j) {
        int local_abort = 0;
        (void)mbar_wait(&full[j % kStages], (j / kStages) & 1, &local_abort, p.err, p.timeout_ns);
      }
      int local_abort = 0;
      (void)mbar_wait(&q_full, 0, &local_abort, p.err, p.timeout_ns);
    }
  } else {
    // ------------------------------------------------------------- compute --
    const int r = lane >> 2, c = lane & 3;
    QueryRows<1> z;
    bool ok = __all_sync(0xFFFFFFFFu, mbar_wait(&q_full, 0, abort_v, p.err, p.timeout_ns));
    load_queries<1>(z, queries, rows, r, c);
    const int len = max(0, min(p.room, len_raw)), n = np + (len + kTok - 1) / kTok;
    int hi = 0, lo = 0;
    // What the rows see of the prefix, or of the sequence's own keys.
    auto part_of = [&](bool pre) {
      hi = lo = pre ? p.prefix_len : len;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int row = 2 * c + e;
        int seen = hi;
        if (p.causal && row < rows) seen = max(0, min(hi, (pre ? p.prefix_len : 0) + len - p.Sq + (row0 + row) / p.G + 1));
        z.lim[0][e] = seen;
        lo = min(lo, seen);
      }
      lo = __reduce_min_sync(0xFFFFFFFFu, lo);
    };
    bool pre = kPrefix && rank < np;
    part_of(pre);
    int it = 0;
    for (int t = rank; t < n; t += ctas, ++it) {
      if (kPrefix && pre && t >= np) {
        pre = false;
        part_of(false);
      }
      const int s = it % kStages;
      ok = ok && __all_sync(0xFFFFFFFFu, mbar_wait(&full[s], (it / kStages) & 1, abort_v, p.err, p.timeout_ns));
      const int at = warp * (kTok / kConsumers);
      if (ok) attend_quarter<1, kBits>(z, smem + s * kStageBytes, p.c_scale, (pre ? t : t - np) * kTok + at, at, r, c, hi, lo);
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }
    // This CTA's part goes where the tiles were: all warps are behind them after
    // the first barrier of join_warps.
    float4 sum[2];
    const float4 mld = join_warps<1>(z, 0, rows, stats, merge, sum);
    const int row = threadIdx.x >> 4, g = threadIdx.x & 15;
    float4* dst = reinterpret_cast<float4*>(smem + row * kHeadDim * 4) + g * 2;
    dst[0] = sum[0];
    dst[1] = sum[1];
    if (g == 0) s_ml[row] = mld;
  }
  __syncwarp();
  cluster_sync_all();
  if constexpr (kBefore == kPrefixParts) asm volatile("griddepcontrol.wait;" ::: "memory");
  if (warp < kConsumers) {
    // A warp a row, four channels a lane.
    for (int row = rank * kConsumers + warp; row < rows; row += ctas * kConsumers) {
      float m = kLowest, d = kLowest, L = 0.0f;
      float4 ml[ctas], part[ctas], acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < ctas; ++k) {
        ml[k] = load_cluster4(in_cta(smem_addr(&s_ml[row]), k));
        part[k] = load_cluster4(in_cta(smem0 + row * kHeadDim * 4 + lane * 16, k));
        m = fmaxf(m, ml[k].x);
      }
#pragma unroll
      for (int k = 0; k < ctas; ++k) d = fmaxf(d, (ml[k].x - m) + ml[k].z);
#pragma unroll
      for (int k = 0; k < ctas; ++k) {
        L += ml[k].y * ex2_approx(ml[k].x - m);
        const float w = ex2_approx((ml[k].x - m) + (ml[k].z - d));
        acc = make_float4(acc.x + part[k].x * w, acc.y + part[k].y * w, acc.z + part[k].z * w, acc.w + part[k].w * w);
      }
      if constexpr (kBefore == kPrefixParts) {
        const RowParts of(parts, b * p.rows + row0 + row, h, p.cache.H);
        for (int k0 = 0; k0 < of.n; k0 += 32) {
          float4 mine = make_float4(kLowest, 0.0f, 0.0f, 0.0f);
          if (k0 + lane < of.n) mine = parts.ml[of.at(parts, k0 + lane)];
          const float less = take_in(mine, m, d, L);
          acc = make_float4(acc.x * less, acc.y * less, acc.z * less, acc.w * less);
          float lw = mine.y;
          const float w = mine.z;
#pragma unroll
          for (int d = 16; d > 0; d >>= 1) lw += __shfl_xor_sync(0xFFFFFFFFu, lw, d);
          L += lw;
          const int end = min(32, of.n - k0);
          for (int k = 0; k < end; k += 8) {                   // eight parts in flight
            float4 y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i)
              y[i] = reinterpret_cast<const float4*>(parts.o + of.at(parts, k0 + min(k + i, end - 1)) * kHeadDim)[lane];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float wk = k + i < end ? __shfl_sync(0xFFFFFFFFu, w, (k + i) & 31) : 0.0f;
              if (k + i < end) acc = make_float4(acc.x + y[i].x * wk, acc.y + y[i].y * wk, acc.z + y[i].z * wk, acc.w + y[i].w * wk);
            }
          }
        }
      }
      const int t = (row0 + row) / p.G, hq = h * p.G + (row0 + row) % p.G;
      const float half = scale2(d), inv = L == 0.0f ? 0.0f : half / L;
      const uint2 w = make_uint2(pack_bf16(acc.x * half * inv, acc.y * half * inv), pack_bf16(acc.z * half * inv, acc.w * half * inv));
      *reinterpret_cast<uint2*>(p.out + ((static_cast<int64_t>(b) * p.Sq + t) * p.Hq + hq) * kHeadDim + lane * 4) = w;
      if (p.lse != nullptr && lane == 0)
        p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.Sq + t] = L == 0.0f ? -INFINITY : (m + log2f(L)) * kLn2;
    }
  }
  __syncwarp();
  cluster_sync_all();            // no CTA ends while another reads from it
}

// ------------------------------------------------------------------ merge --

struct MergeParams {
  const float* part_o;
  const float4* part_ml;
  const int4* desc;          // one key/value part alone
  const int2* info;          // a prefix and the sequences
  int ctas, R, slot_rows, rows, row_tiles, H;
  PrefixParts pre;           // o null: none
  uint16_t* out;
  float* lse;
  int Sq, G, Hq;
  int split;                 // warps of a row: a power of two
};

constexpr int kMergeWarps = 8;

// A CTA takes kMergeWarps / p.split rows of a unit, `split` warps each: a warp goes
// through the row's parts, 32 at a time with one part's m, L and d a lane, adds
// those of its turn in order, and the warps' results are joined in order.
__global__ void __launch_bounds__(kMergeWarps * 32) cache_merge_kernel(const MergeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  __shared__ float s_l[kMergeWarps];
  __shared__ float4 s_o[kMergeWarps][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int b, rt, h, first, n, own = -1;
  if (p.info == nullptr) {
    const int4 d = p.desc[blockIdx.x];
    if (d.w < 2) return;
    b = d.x;
    rt = d.y;
    h = d.z;
    first = blockIdx.x;
    n = d.w;
  } else {
    const int2 d = p.info[blockIdx.x];
    h = blockIdx.x % p.H;
    rt = blockIdx.x / p.H % p.row_tiles;
    b = blockIdx.x / p.H / p.row_tiles;
    first = d.x;
    n = d.y == 0 ? 1 : d.y;
    if (d.y == 0) own = 2 * p.ctas + blockIdx.x;
  }
  const int turn = warp % p.split;
  const int row = (blockIdx.y * kMergeWarps + warp) / p.split, rr = rt * p.R + row;
  const bool live = row < p.R && rr < p.rows;
  float m = kLowest, d = kLowest, L = 0.0f;
  float4 acc = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (live) {
    const bool behind = p.pre.o != nullptr;
    const RowParts of(p.pre, b * p.rows + rr, h, p.H);       // row b * rows + rr of the prefix's launch
    const int total = n + (behind ? of.n : 0);
    auto place = [&](int k, const float*& o, const float4*& ml) {
      if (k < n) {
        const int slot = own >= 0 ? own : (k == 0 ? 2 * first + 1 : 2 * (first + k));
        const int64_t at = static_cast<int64_t>(slot) * p.slot_rows + row;
        o = p.part_o + at * kHeadDim;
        ml = p.part_ml + at;
      } else {
        const int64_t at = of.at(p.pre, k - n);
        o = p.pre.o + at * kHeadDim;
        ml = p.pre.ml + at;
      }
    };
    for (int k0 = 0; k0 < total; k0 += 32) {
      float4 mine = make_float4(kLowest, 0.0f, 0.0f, 0.0f);
      const float* o;
      const float4* ml;
      if (k0 + lane < total) {
        place(k0 + lane, o, ml);
        mine = *ml;
      }
      const float less = take_in(mine, m, d, L);
      acc = make_float4(acc.x * less, acc.y * less, acc.z * less, acc.w * less);
      const float lw = mine.y, w = mine.z;
      const int end = min(32, total - k0);
      for (int k = turn; k < end; k += 4 * p.split) {        // four parts in flight
        float4 y[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          place(k0 + min(k + i * p.split, end - 1), o, ml);
          y[i] = reinterpret_cast<const float4*>(o)[lane];
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = k + i * p.split;
          const float wk = __shfl_sync(0xFFFFFFFFu, w, at & 31), lk = __shfl_sync(0xFFFFFFFFu, lw, at & 31);
          if (at >= end) break;
          L += lk;
          acc.x += y[i].x * wk;
          acc.y += y[i].y * wk;
          acc.z += y[i].z * wk;
          acc.w += y[i].w * wk;
        }
      }
    }
  }
  if (p.split > 1) {                                         // m and d are the same for all warps of a row
    s_o[warp][lane] = acc;
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    if (turn != 0) return;
    for (int k = 1; k < p.split; ++k) {
      const float4 y = s_o[warp + k][lane];
      L += s_l[warp + k];
      acc.x += y.x;
      acc.y += y.y;
      acc.z += y.z;
      acc.w += y.w;
    }
  }
  if (!live) return;
  const int t = rr / p.G, hq = h * p.G + rr % p.G;
  const float half = scale2(d);
  const float inv = L == 0.0f ? 0.0f : half / L;
  uint2 w;
  w.x = pack_bf16(acc.x * half * inv, acc.y * half * inv);
  w.y = pack_bf16(acc.z * half * inv, acc.w * half * inv);
  *reinterpret_cast<uint2*>(p.out + ((static_cast<int64_t>(b) * p.Sq + t) * p.Hq + hq) * kHeadDim + lane * 4) = w;
  if (p.lse != nullptr && lane == 0)
    p.lse[(static_cast<int64_t>(b) * p.Hq + hq) * p.Sq + t] = L == 0.0f ? -INFINITY : (m + log2f(L)) * kLn2;
}

// The same where a unit has many rows and few parts: a warp takes kMergeRows rows side by
// side, so that their loads are in flight together, and the sums are those of one warp a
// row above, in the same order (2 x 1000 tokens, 16 / 4 heads over 8000 keys, 32000 rows in
// two parts or three, the whole call: 196 us, with the kernel above 206).
constexpr int kMergeRows = 4;
__global__ void __launch_bounds__(kMergeWarps * 32, 3) cache_merge_rows_kernel(const MergeParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int4 unit = p.desc[blockIdx.x];
  const int n = unit.w;
  const int row0 = (blockIdx.y * kMergeWarps + warp) * kMergeRows;
  if (n < 2 || row0 >= min(p.R, p.rows - unit.y * p.R)) return;      // warp-uniform
  auto at = [&](int k, int i) {                                      // row row0 + i of part k, where there is one
    const int slot = k == 0 ? 2 * static_cast<int>(blockIdx.x) + 1 : 2 * (static_cast<int>(blockIdx.x) + k);
    return static_cast<int64_t>(slot) * p.slot_rows + min(row0 + i, p.slot_rows - 1);
  };
  float m[kMergeRows], d[kMergeRows], L[kMergeRows];
  float4 acc[kMergeRows];
#pragma unroll
  for (int i = 0; i < kMergeRows; ++i) {
    m[i] = d[i] = kLowest;
    L[i] = 0.0f;
    acc[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  for (int k0 = 0; k0 < n; k0 += 32) {
    float4 mine[kMergeRows];
#pragma unroll
    for (int i = 0; i < kMergeRows; ++i) {
      mine[i] = make_float4(kLowest, 0.0f, 0.0f, 0.0f);
      if (k0 + lane < n) mine[i] = p.part_ml[at(k0 + lane, i)];
    }
#pragma unroll
    for (int i = 0; i < kMergeRows; ++i) {
      const float less = take_in(mine[i], m[i], d[i], L[i]);
      acc[i] = make_float4(acc[i].x * less, acc[i].y * less, acc[i].z * less, acc[i].w * less);
    }
    const int end = min(32, n - k0);
    for (int k = 0; k < end; k += 2) {
      float4 y[2][kMergeRows];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i)
          y[j][i] = reinterpret_cast<const float4*>(p.part_o + at(k0 + min(k + j, end - 1), i) * kHeadDim)[lane];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (k + j >= end) break;
#pragma unroll
        for (int i = 0; i < kMergeRows; ++i) {
          const float w = __shfl_sync(0xFFFFFFFFu, mine[i].z, k + j);
          L[i] += __shfl_sync(0xFFFFFFFFu, mine[i].y, k + j);
          acc[i].x += y[j][i].x * w;
          acc[i].y += y[j][i].y * w;
          acc[i].z += y[j][i].z * w;
          acc[i].w += y[j][i].w * w;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kMergeRows; ++i) {
    const int rr = unit.y * p.R + row0 + i;
    if (row0 + i >= p.R || rr >= p.rows) break;
    const int t = rr / p.G, hq = unit.z * p.G + rr % p.G;
    const float half = scale2(d[i]), inv = L[i] == 0.0f ? 0.0f : half / L[i];
    const uint2 w = make_uint2(pack_bf16(acc[i].x * half * inv, acc[i].y * half * inv), pack_bf16(acc[i].z * half * inv, acc[i].w * half * inv));
    *reinterpret_cast<uint2*>(p.out + ((static_cast<int64_t>(unit.x) * p.Sq + t) * p.Hq + hq) * kHeadDim + lane * 4) = w;
    if (p.lse != nullptr && lane == 0)
      p.lse[(static_cast<int64_t>(unit.x) * p.Hq + hq) * p.Sq + t] = L[i] == 0.0f ? -INFINITY : (m[i] + log2f(L[i])) * kLn2;
  }
}

// ------------------------------------------------------------------- host --

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// 8 or 16 query rows a tile where they are all, else the wide kernel's 256: the keys
// are read and converted once for all rows of a tile.  32 sequences of 16384 keys, 8
// key/value heads, us, 8 bits / 4 bits: 16 rows 224 / 202, as two tiles of eight 328 / 245,
// in the wide kernel 381 / 395; 24 rows in the wide kernel 382 / 396, as three tiles of
// eight 484 / 362, as two of 16 428 / 384; 32 rows 383 / 396, as two of 16 429 / 385; 64 rows
// 383 / 397, as four of 16 840 / 747.  (17 to 32 rows in 4 bits would be up to 9% sooner done
// in small tiles; one rule serves both caches.)
int rows_per_tile(int rows) { return rows <= 8 ? 8 : rows <= 16 ? 16 : kWideRows; }
int max_ctas(int R) { return kSms * (R == kWideRows ? 1 : ctas_per_sm(R / 8)); }
int keys_per_tile(int R, int bits) { return R == kWideRows ? kWideTok : tok_of(bits); }
int unit_cost(int R, int bits) { return R == kWideRows ? kWideCost : cost_of(bits); }

// One launch's part of the workspace.
struct Layout {
  int rows, R, slot_rows, row_tiles, units, slots;
  size_t o, ml, desc, info, end;
};

// keep: every unit may also need a slot of its own.
Layout layout(int rows, int B, int H, bool keep, size_t at) {
  Layout w;
  w.rows = rows;
  w.R = rows_per_tile(rows);
  w.row_tiles = (rows + w.R - 1) / w.R;
  w.units = B * w.row_tiles * H;
  w.slot_rows = std::min(w.R, rows);
  w.slots = 2 * max_ctas(w.R) + (keep ? w.units : 0);
  w.o = at;
  w.ml = w.o + align256(static_cast<size_t>(w.slots) * w.slot_rows * kHeadDim * sizeof(float));
  w.desc = w.ml + align256(static_cast<size_t>(w.slots) * w.slot_rows * sizeof(float4));
  w.info = w.desc + align256(kMaxCtas * sizeof(int4));
  w.end = w.info + (keep ? align256(static_cast<size_t>(w.units) * sizeof(int2)) : 0);
  return w;
}

template <typename T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + off);
}

// beside: the launch before is this call's, and nothing of it is needed.
cudaError_t launch_part(const Params& p, int R, bool prefix, bool beside, unsigned ctas, cudaStream_t stream) {
  if (R == kWideRows) return launch_wide(p, prefix, beside, ctas, stream);
  const bool in8 = p.cache.bits == 8;
  const uint32_t smem = in8 ? smem_of<8>(R / 8) : smem_of<4>(R / 8);
  auto go = [&](auto kernel) {
    static std::atomic<uint64_t> allowed[2 * 2 * 2];   // for each kernel
    cudaError_t e = allow_smem(kernel, smem, allowed[(in8 ? 0 : 4) + (prefix ? 2 : 0) + R / 16]);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = beside ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p);
  };
  auto of = [&](auto bits) {
    constexpr int kBits = decltype(bits)::value;
    if (prefix)
      return R == 8 ? go(cache_attn_kernel<1, true, kBits>) : go(cache_attn_kernel<2, true, kBits>);
    return R == 8 ? go(cache_attn_kernel<1, false, kBits>) : go(cache_attn_kernel<2, false, kBits>);
  };
  return in8 ? of(std::integral_constant<int, 8>()) : of(std::integral_constant<int, 4>());
}

unsigned ctas_for(long long tiles, int R) {
  return static_cast<unsigned>(std::min<long long>(max_ctas(R), std::max(1ll, tiles)));
}

// CTAs of a unit's cluster where one launch of clusters does it all, or 0: where no SM
// slot (three on each SM) has more than 16 tiles to do, one CTA after another, and, for
// more than 32 rows, which the wide kernel takes together, no more than two CTAs.
// Both sides, us (clusters, the kernels above or the wide one), 8 key/value heads of
// full sequences: 4 rows: 1 of 1024 keys 8.3, 12.4; 1 of 8192 18.6, 16.5; 12 of 4096
// 23.8, 27.3; 48 of 1024 23.9, 29.4; 100 of 512 28.8, 34.0; 48 of 2048 40.0, 45.6 (half full
// 34.9, 32.9).  32 rows: 1 of 1024 10.4, 19.1; 4 of 2048 20.6, 25.8; 64 of 128 37.0, 47.2.
// 64 rows: 4 of 1024 20.6, 24.7; 12 of 512 28.8, 29.3; 24 of 256 (four CTAs) 36.1, 32.8.
// 256 rows, 2 heads: 1 of 4096 20.6, 43.4; 24 of 256 (four CTAs) 37.0, 28.9.  Behind a prefix of
// 1024, 4 rows: 6 sequences, 2 heads 8.7, 18.6; 24, 8 heads, 16.5, 27.7, of 4096 41.1, 32.9.
int cluster_ctas(const CacheAttnArgs& a, int prefix_len) {
  const int64_t rows = static_cast<int64_t>(a.Sq) * (a.Hq / a.cache.H);
  const int64_t units = a.B * ((rows + 7) / 8) * a.cache.H;   // of eight rows
  const int64_t room = std::min<int64_t>(kMaxCacheLen, static_cast<int64_t>(a.table.width) << a.cache.page_shift);
  const int tok = tok_of(a.cache.bits), most_tiles = kClusterKeys / tok;
  const int64_t tiles = (room + tok - 1) / tok + (prefix_len + tok - 1) / tok;
  const int most = max_ctas(8);
  int ctas = 8;
  while (ctas > 1 && (units * ctas > most || tiles <= ctas / 2)) ctas /= 2;
  const int64_t waves = (units * ctas + most - 1) / most;
  if (waves > (rows <= 32 ? most_tiles : 2)) return 0;
  return waves * ((tiles + ctas - 1) / ctas) <= most_tiles ? ctas : 0;
}

// The same for the sequences' own keys behind a prefix that has a launch of its own,
// whose parts the clusters join: where no row has more than 48 of those, which one warp
// goes through (the merge kernel has up to eight on a row), and there are at most two
// CTAs to an SM slot.  Both sides, us, of 64 .. 512 keys behind 16384, 4 rows, 8 heads:
// 8 sequences 34.0, 40.1 .. 35.3, 39.9; 64 53.5, 56.4 .. 68.4, 66.9.  24 x 5 rows, 16 heads
// behind 32768 76, 81 .. 81, 89; 128 (five CTAs) 305, 296.  2 heads, 8 rows (76 parts a
// row) behind 8192: 8 sequences 33.4, 26.8.
int joining_ctas(const CacheAttnArgs& a) {
  const int rows = a.Sq * (a.Hq / a.cache.H);
  if (a.B > kMaxBatch || static_cast<int64_t>(a.B) * ((rows + 7) / 8) * a.cache.H > 2 * max_ctas(8)) return 0;
  const int all = a.B * rows, R = rows_per_tile(all), units = (all + R - 1) / R * a.cache.H;
  return max_ctas(R) / units + 1 <= 48 ? cluster_ctas(a, 0) : 0;
}

cudaError_t launch_clusters(const CacheAttnArgs& a, int ctas, const PrefixParts* parts, cudaStream_t stream) {
  Params p = {};
  p.cache = a.cache;
  p.table = a.table;
  p.lens = a.lens;
  p.q = a.q;
  p.q_sb = a.q_sb;
  p.q_ss = a.q_ss;
  p.out = a.out;
  p.lse = a.lse;
  p.B = a.B;
  p.Sq = a.Sq;
  p.G = a.Hq / a.cache.H;
  p.Hq = a.Hq;
  p.causal = a.causal;
  p.prefix_len = a.prefix_len;
  p.room = static_cast<int>(std::min<int64_t>(kMaxCacheLen, static_cast<int64_t>(a.table.width) << a.cache.page_shift));
  p.rows = a.Sq * p.G;
  p.row_tiles = (p.rows + 7) / 8;
  p.c_scale = a.softmax_scale * kLog2e;
  p.timeout_ns = a.timeout_ns;
  p.err = a.err;
  auto go = [&](auto size, auto bits) {
    constexpr int kCtas = decltype(size)::value, kBits = decltype(bits)::value;
    constexpr uint32_t smem = smem_of<kBits>(1) - (kBits == 8 ? 0 : kMergeBytes);
    static std::atomic<uint64_t> allowed[4];           // for each kernel
    const int which = parts != nullptr ? kPrefixParts : a.prefix_len > 0 ? kPrefixTiles : kNothing;
    constexpr int kPerSm = ctas_per_sm(1);
    auto kernel = which == kPrefixParts   ? cache_attn_cluster_kernel<kCtas, kPrefixParts, kBits, kPerSm>
                  : which == kPrefixTiles ? cache_attn_cluster_kernel<kCtas, kPrefixTiles, kBits, kPerSm>
                                          : cache_attn_cluster_kernel<kCtas, kNothing, kBits, kPerSm>;
    int kind = which;
    if constexpr (kCtas == 1 && kBits == 4) {
      const int64_t all = static_cast<int64_t>(a.B) * p.row_tiles * a.cache.H;
      const auto rounds = [&](int per_sm) { return (all + per_sm * kSms - 1) / (per_sm * kSms); };
      if (which == kPrefixParts && rounds(kPerSm + 1) < rounds(kPerSm)) {
        kernel = cache_attn_cluster_kernel<1, kPrefixParts, 4, kPerSm + 1>;
        kind = 3;
      }
    }
    const cudaError_t e = allow_smem(kernel, smem, allowed[kind]);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(a.B) * p.row_tiles * a.cache.H * kCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    // Behind the prefix's launch, whose parts are waited for before the join.
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = which == kPrefixParts ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, p, a.prefix_pages, parts != nullptr ? *parts : PrefixParts{});
  };
  auto of = [&](auto bits) {
    return ctas == 8   ? go(std::integral_constant<int, 8>(), bits)
           : ctas == 4 ? go(std::integral_constant<int, 4>(), bits)
           : ctas == 2 ? go(std::integral_constant<int, 2>(), bits)
                       : go(std::integral_constant<int, 1>(), bits);
  };
  return a.cache.bits == 8 ? of(std::integral_constant<int, 8>()) : of(std::integral_constant<int, 4>());
}

}  // namespace

size_t cache_attn_workspace_bytes(int B, int Sq, int Hq, int Hkv, int prefix_len) {
  const int b = std::min(B, kMaxBatch), rows = Sq * (Hq / Hkv);
  const bool both = prefix_len > 0;
  Layout w = layout(rows, b, Hkv, both, 0);
  if (both) w = layout(b * rows, 1, Hkv, true, w.end);
  return w.end;
}

bool cache_attn_fits(int B, int Sq, int Hq, int Hkv, int page_size, int table_width, int prefix_len) {
  const auto fits = [](int64_t keys, int64_t rows, int64_t seqs, int64_t H) {
    const int R = rows_per_tile(static_cast<int>(rows));
    const int64_t tiles = (keys + keys_per_tile(R, 8) - 1) / keys_per_tile(R, 8) + unit_cost(R, 8);   // of a unit, at most 2^25; fewer in 4 bits
    const int64_t units = seqs * ((rows + R - 1) / R) * H;                                   // at most 2^31
    return tiles * units / max_ctas(R) < INT_MAX;
  };
  const int64_t b = std::min(B, kMaxBatch), rows = static_cast<int64_t>(Sq) * (Hq / Hkv);
  return fits(std::min<int64_t>(kMaxCacheLen, static_cast<int64_t>(table_width) * page_size), rows, b, Hkv) &&
         (prefix_len == 0 || fits(prefix_len, b * rows, 1, Hkv));
}

bool cache_attn_needs_workspace(const CacheAttnArgs& a) { return cluster_ctas(a, a.prefix_len) == 0; }

cudaError_t launch_cache_attention(const CacheAttnArgs& a, cudaStream_t stream) {
  if (const int ctas = cluster_ctas(a, a.prefix_len); ctas > 0) return launch_clusters(a, ctas, nullptr, stream);
  const int H = a.cache.H, G = a.Hq / H, bits = a.cache.bits;
  const bool both = a.prefix_len > 0;
  const int join_ctas = both ? joining_ctas(a) : 0;
  for (int b0 = 0; b0 < a.B; b0 += kMaxBatch) {
    const int B = std::min(kMaxBatch, a.B - b0);
    const Layout w = layout(a.Sq * G, B, H, both, 0);
    Params p = {};
    p.cache = a.cache;
    p.table = a.table;
    p.table.pages += b0 * a.table.stride;
    p.lens = a.lens + b0;
    p.q = a.q + b0 * a.q_sb;
    p.q_sb = a.q_sb;
    p.q_ss = a.q_ss;
    p.out = a.out + static_cast<int64_t>(b0) * a.Sq * a.Hq * kHeadDim;
    p.lse = a.lse == nullptr ? nullptr : a.lse + static_cast<int64_t>(b0) * a.Sq * a.Hq;
    p.B = B;
    p.Sq = a.Sq;
    p.G = G;
    p.Hq = a.Hq;
    p.causal = a.causal;
    p.prefix_len = a.prefix_len;
    p.rows = w.rows;
    p.row_tiles = w.row_tiles;
    p.c_scale = a.softmax_scale * kLog2e;
    p.keep = both;
    p.slot_rows = w.slot_rows;
    p.part_o = at<float>(a.workspace, w.o);
    p.part_ml = at<float4>(a.workspace, w.ml);
    p.desc = at<int4>(a.workspace, w.desc);
    p.info = both ? at<int2>(a.workspace, w.info) : nullptr;
    p.timeout_ns = a.timeout_ns;
    p.err = a.err;
    p.room = static_cast<int>(std::min<int64_t>(kMaxCacheLen, static_cast<int64_t>(a.table.width) << a.cache.page_shift));
    // The lengths are on the device: as many CTAs as the table has room for.
    const unsigned ctas = ctas_for(std::min<long long>(kMaxCtas, (static_cast<long long>(p.room) + keys_per_tile(w.R, bits) - 1) / keys_per_tile(w.R, bits) + unit_cost(w.R, bits)) * w.units, w.R);
    cudaError_t e = join_ctas > 0 ? cudaSuccess : launch_part(p, w.R, false, false, ctas, stream);
    if (e != cudaSuccess) return e;

    MergeParams mp = {};
    mp.pre.R = 1;                                          // no division by zero where there is none
    mp.pre.per = 1;
    mp.part_o = p.part_o;
    mp.part_ml = p.part_ml;
    mp.desc = p.desc;
    mp.info = p.info;
    mp.ctas = ctas;
    mp.R = w.R;
    mp.slot_rows = w.slot_rows;
    mp.rows = w.rows;
    mp.row_tiles = w.row_tiles;
    mp.H = H;
    mp.out = p.out;
    mp.lse = p.lse;
    mp.Sq = a.Sq;
    mp.G = G;
    mp.Hq = a.Hq;
    int pre_units = 0;
    if (both) {
      const Layout u = layout(B * a.Sq * G, 1, H, true, w.end);
      p.table.pages = a.prefix_pages;
      p.table.width = (a.prefix_len + (1 << a.cache.page_shift) - 1) >> a.cache.page_shift;
      p.table.stride = 0;
      p.rows = u.rows;
      p.row_tiles = u.row_tiles;
      p.slot_rows = u.slot_rows;
      p.part_o = at<float>(a.workspace, u.o);
      p.part_ml = at<float4>(a.workspace, u.ml);
      p.desc = at<int4>(a.workspace, u.desc);
      p.info = at<int2>(a.workspace, u.info);
      const int n = (a.prefix_len + keys_per_tile(u.R, bits) - 1) / keys_per_tile(u.R, bits);
      const long long steps = static_cast<long long>(n + unit_cost(u.R, bits)) * u.units;
      const unsigned pc = ctas_for(steps, u.R);
      e = launch_part(p, u.R, true, join_ctas == 0, pc, stream);
      if (e != cudaSuccess) return e;
      mp.pre.o = p.part_o;
      mp.pre.ml = p.part_ml;
      mp.pre.R = u.R;
      mp.pre.slot_rows = u.slot_rows;
      mp.pre.n = n;
      mp.pre.cost = unit_cost(u.R, bits);
      mp.pre.per = (steps + pc - 1) / pc;
      mp.pre.ctas = pc;
      if (join_ctas > 0) return launch_clusters(a, join_ctas, &mp.pre, stream);
      pre_units = u.units;
    }
    // Warps of a row: so many that each adds about eight parts, and that few rows
    // leave none idle.
    const int tile_rows = std::min(w.R, w.rows);
    const long long parts = ctas / w.units + 1 + (both ? mp.pre.ctas / std::max(1, pre_units) + 1 : 0);
    mp.split = 1;
    while (mp.split < kMergeWarps && (mp.split * 8 < parts || mp.split * 2 * tile_rows <= kMergeWarps)) mp.split *= 2;
    cudaLaunchConfig_t cfg = {};
    const bool by_rows = !both && mp.split == 1 && w.R == kWideRows;
    cfg.gridDim = dim3(both ? w.units : ctas, (tile_rows * mp.split + kMergeWarps - 1) / kMergeWarps);
    if (by_rows) cfg.gridDim.y = (tile_rows + kMergeWarps * kMergeRows - 1) / (kMergeWarps * kMergeRows);
    cfg.blockDim = dim3(kMergeWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, by_rows ? cache_merge_rows_kernel : cache_merge_kernel, mp);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace sage
