// cache_attention.cuh -- what the kernels of the attention over the KV cache
// share: their arguments, the way a launch's work is cut up, and the forms of
// the codes.
#pragma once

#include <climits>
#include <cstdint>
#include <cuda_runtime.h>

#include "sage_internal.cuh"
#include "sm103_ptx.cuh"

namespace sage::cache {

constexpr int kSms = 152;
constexpr int kMaxBatch = 256;                            // sequences of one launch
constexpr float kLowest = -3.4028234663852886e38f;        // the lowest fp32: a reference below every score
constexpr float kLog2e = 1.44269502162933349609375f;      // fp32(log2 e)
constexpr float kLn2 = 0.693147182464599609375f;          // fp32(ln 2)

struct Params {
  CacheView cache;
  PageTable table;           // of the sequences, or of the prefix (one row)
  const int32_t* lens;       // [B] of this launch
  const uint16_t* q;
  int64_t q_sb, q_ss;
  uint16_t* out;
  float* lse;
  int B, Sq, G, Hq;          // G query heads share a key/value head
  int causal, prefix_len;
  int room;                  // longest sequence the sequences' table can hold
  int rows, row_tiles;       // query rows of one unit's key/value head, and tiles of them
  float c_scale;             // softmax_scale * log2 e
  int keep;                  // 1: every result goes to the workspace (merged with another launch's)
  int slot_rows;             // rows of a slot: a full tile's, or all there are
  float* part_o;             // [slot][slot_rows][128]: sums relative to m + d
  float4* part_ml;           // [slot][slot_rows]: m, L, d
  int4* desc;                // [CTA]: the unit that begins in this CTA and ends in a later one
  int2* info;                // [unit], with keep: first CTA and CTAs of the unit (0: its own slot)
  uint64_t timeout_ns;
  int* err;
};

// The square root of 2^e: a product with 2^e is taken in two steps, so that
// nothing in between overflows or vanishes.
__device__ __forceinline__ float scale2(float e) { return ex2_approx(0.5f * e); }

// a / b for a >= 0, b > 0: in 32 bits where they do.
__device__ __forceinline__ long long div_floor(long long a, long long b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// A launch's work is a row of steps: for each sequence, each tile of query rows
// and each key/value head (a unit) Cost steps, which stand for what a unit takes
// however short it is, and one for each of its tiles of keys, in order.  CTA c has
// steps [c * per, (c + 1) * per), whatever units they belong to, so that unequal
// lengths leave no SM idle.  The tiles of a unit that a CTA has are a segment: a
// unit of one segment is written out at once, segments of a unit that CTAs share
// go to the workspace (slot 2c + 1 for the unit that begins in CTA c and ends
// later, slot 2c for one that began earlier) and the merge kernel joins them in
// the order of the CTAs.
struct Place {
  int b, rt, h, n;           // a unit and its tiles
  int skip, left;            // its steps that earlier CTAs have, and steps of this CTA from there on
  int t0, t1;                // tiles of the segment
};

// A sequence's length, cut to what its table has room for: an error, except that
// kMaxCacheLen or more asks for just that.
__device__ __forceinline__ int held(int len, const Params& p) {
  if (len > p.room && len < kMaxCacheLen) atomicExch(p.err, SAGE_DEVERR_BAD_PAGE);
  return max(0, min(p.room, len));
}

// R query rows and Tok keys a tile.
template <int R, int Tok, int Cost, bool kPrefix>
struct Walk {
  const Params& p;
  const int* s_len;
  const long long* s_off;

  // Keys that query row rr of sequence b may see, in this launch's keys.
  __device__ int limit(int b, int rr) const {
    if constexpr (kPrefix) {
      if (!p.causal) return p.prefix_len;
      const int per_seq = p.Sq * p.G, seq = rr / per_seq, t = rr % per_seq / p.G;
      return max(0, p.prefix_len + min(0, s_len[seq] - p.Sq + t + 1));   // the sum of both lengths may be 2^31
    } else {
      const int len = s_len[b];
      return p.causal ? max(0, min(len, len - p.Sq + rr / p.G + 1)) : len;
    }
  }
  // Keys that some row of the unit may see.
  __device__ int keys(int b, int rt) const {
    if constexpr (kPrefix) return p.prefix_len;
    return limit(b, min(p.rows, (rt + 1) * R) - 1);
  }
  __device__ int tiles(int b, int rt) const { return max(1, (keys(b, rt) + Tok - 1) / Tok); }
  __device__ int seqs() const { return kPrefix ? 1 : p.B; }

  // The first segment of the CTA that has the steps [f, f + left); x.left is 0
  // if it has none, which is so too after `next` behind the last.
  __device__ Place locate(long long f, int left) const {
    Place x;
    int lo = 0, hi = seqs();
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (s_off[mid] * p.cache.H <= f)
        lo = mid;
      else
        hi = mid;
    }
    long long rem = f - s_off[lo] * p.cache.H;
    x.b = lo;
    x.rt = 0;
    x.n = tiles(lo, 0);
    if constexpr (kPrefix) {             // all row tiles see the same keys
      const long long each = static_cast<long long>(x.n + Cost) * p.cache.H;
      x.rt = static_cast<int>(div_floor(rem, each));
      rem -= x.rt * each;
    }
    while (rem >= static_cast<long long>(x.n + Cost) * p.cache.H) {
      rem -= static_cast<long long>(x.n + Cost) * p.cache.H;
      x.n = tiles(lo, ++x.rt);
    }
    x.h = static_cast<int>(div_floor(rem, x.n + Cost));
    x.skip = static_cast<int>(rem - static_cast<long long>(x.h) * (x.n + Cost));
    x.left = left;
    if (!cut(x)) next(x);
    return x;
  }
  // The segment's tiles; false if it has none.
  __device__ bool cut(Place& x) const {
    x.t0 = max(0, x.skip - Cost);
    x.t1 = min(x.n, x.skip + x.left - Cost);
    return x.t1 > x.t0;
  }
  __device__ void next(Place& x) const {
    do {
      x.left -= min(x.left, x.n + Cost - x.skip);
      x.skip = 0;
      if (x.left == 0) return;
      if (++x.h == p.cache.H) {
        x.h = 0;
        if (++x.rt == p.row_tiles) {
          x.rt = 0;
          ++x.b;
        }
        x.n = tiles(x.b, x.rt);
      }
    } while (!cut(x));
  }
  __device__ bool whole(const Place& x) const { return x.t0 == 0 && x.t1 == x.n; }
  // The lengths of the launch's sequences, cut to what their table can hold, and
  // off[b] = steps of the sequences before b, for one key/value head.  Every thread
  // calls it; a barrier has to follow.
  __device__ void plan(int* len, long long* off) const {
    if constexpr (kPrefix) {
      for (int i = threadIdx.x; i < p.B; i += blockDim.x) len[i] = held(__ldg(p.lens + i), p);
      if (threadIdx.x == 0) {
        off[0] = 0;
        off[1] = static_cast<long long>(p.row_tiles) * (tiles(0, 0) + Cost);
      }
    } else if (threadIdx.x < 32) {
      const int lane = threadIdx.x;
      long long base = 0;
      int next = lane < p.B ? __ldg(p.lens + lane) : 0;
      for (int b0 = 0; b0 < p.B; b0 += 32) {
        const int b = b0 + lane, mine = held(next, p);
        if (b + 32 < p.B) next = __ldg(p.lens + b + 32);
        long long n = 0;
        if (b < p.B) {
          len[b] = mine;
          for (int rt = 0; rt < p.row_tiles; ++rt) n += tiles(b, rt) + Cost;   // reads what this thread has written
        }
        long long sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
          const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
          if (lane >= d) sum += up;
        }
        if (b < p.B) off[b] = base + sum - n;
        base += __shfl_sync(0xFFFFFFFFu, sum, 31);
      }
      if (lane == 0) off[p.B] = base;
    }
  }
  // Where a segment's result goes if it is not written out.
  __device__ int slot(const Place& x) const {
    if (whole(x)) return 2 * static_cast<int>(gridDim.x) + unit(x);
    return 2 * static_cast<int>(blockIdx.x) + (x.t0 > 0 ? 0 : 1);
  }
  // For the merge kernel, by one thread where a unit's tiles begin: how many CTAs
  // have some of them.  f1: the step behind this CTA's last, per: steps of a CTA.
  __device__ void tell(const Place& x, long long f1, long long per) const {
    if (x.t0 != 0) return;
    const long long last = f1 - x.left - x.skip + Cost + x.n - 1;
    const int ctas = static_cast<int>(div_floor(last, per)) - static_cast<int>(blockIdx.x) + 1;
    if (p.keep)
      p.info[unit(x)] = make_int2(blockIdx.x, whole(x) ? 0 : ctas);
    else if (!whole(x))
      p.desc[blockIdx.x] = make_int4(x.b, x.rt, x.h, ctas);
  }
  // The query row rr of the unit's key/value head, 128 channels.
  __device__ const uint16_t* query(const Place& x, int rr) const {
    const int per_seq = p.Sq * p.G;
    const int seq = kPrefix ? rr / per_seq : x.b, in = kPrefix ? rr % per_seq : rr;
    return p.q + seq * p.q_sb + (in / p.G) * p.q_ss + (x.h * p.G + in % p.G) * kHeadDim;
  }
  __device__ int unit(const Place& x) const { return (x.b * p.row_tiles + x.rt) * p.cache.H + x.h; }
};

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// 2^(141 - exponent of the largest of a row's magnitudes, given as bf16 bits),
// at most 2^113, as the bits of an fp32 exponent field: times it the row's
// largest lies in [2^14, 2^15).  254 less it is the field of the inverse.
__device__ __forceinline__ uint32_t row_exponent(uint32_t top) { return min(240u, 268u - (top >> 7)); }
__device__ __forceinline__ float lg2_approx(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// (m, d) becomes the larger of two scores and, relative to it, the larger of two
// references m + d.
__device__ __forceinline__ void larger(float& m, float& d, float m2, float d2) {
  const float mx = fmaxf(m, m2);
  d = fmaxf((m - mx) + d, (m2 - mx) + d2);
  m = mx;
}

// Four INT8 codes (one word) -> two pairs of fp16: code + 128 is put into the
// low bits of 1024 and 1152 taken off again, both exact.
__device__ __forceinline__ void k_codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
  hi = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
}

// The launch of the kernel for many query rows (cache_attention_wide.cu): 256
// rows and 128 keys a tile, one CTA on each SM.
constexpr int kWideRows = 256, kWideTok = 128, kWideCost = 3;
cudaError_t launch_wide(const Params& p, bool prefix, bool beside, unsigned ctas, cudaStream_t stream);

}  // namespace sage::cache
