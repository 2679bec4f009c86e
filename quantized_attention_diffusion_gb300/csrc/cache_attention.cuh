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
constexpr int kMaxBatch = 512;                            // sequences of one launch
constexpr float kLowest = -1e30f;                         // a reference below every score
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
  float* part_o;             // [slot][slot_rows][128]: sums relative to M
  float4* part_ml;           // [slot][slot_rows]: m, L, M
  int4* desc;                // [CTA]: the unit that begins in this CTA and ends in a later one
  int2* info;                // [unit], with keep: first CTA and CTAs of the unit (0: its own slot)
  uint64_t timeout_ns;
  int* err;
};

// The square root of 2^e: a product with 2^e is taken in two steps, so that
// nothing in between overflows or vanishes.
__device__ __forceinline__ float scale2(float e) { return ex2_approx(0.5f * e); }

// A launch's work is a row of key tiles: for each sequence, each tile of query
// rows and each key/value head (a unit) its tiles of keys in order.  CTA c
// takes tiles [c * per, (c + 1) * per), whatever units they belong to, so that
// unequal lengths leave no SM idle.  The part of a unit that a CTA has is a
// segment: a unit of one segment is written out at once, segments of a unit
// that CTAs share go to the workspace (slot 2c + 1 for the unit that begins
// in CTA c and ends later, slot 2c for one that began earlier) and the merge
// kernel joins them in the order of the CTAs.
struct Place {
  int b, rt, h, tile, n;     // n: tiles of the unit
};

// R query rows and Tok keys a tile.
template <int R, int Tok, bool kPrefix>
struct Walk {
  const Params& p;
  const int* s_len;
  const long long* s_off;

  // Keys that query row rr of sequence b may see, in this launch's keys.
  __device__ int limit(int b, int rr) const {
    if constexpr (kPrefix) {
      if (!p.causal) return p.prefix_len;
      const int per_seq = p.Sq * p.G, seq = rr / per_seq, t = rr % per_seq / p.G;
      return max(0, min(p.prefix_len, p.prefix_len + s_len[seq] - p.Sq + t + 1));
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

  __device__ Place locate(long long f) const {
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
    while (rem >= static_cast<long long>(x.n) * p.cache.H) {
      rem -= static_cast<long long>(x.n) * p.cache.H;
      x.n = tiles(lo, ++x.rt);
    }
    x.h = static_cast<int>(rem / x.n);
    x.tile = static_cast<int>(rem % x.n);
    return x;
  }
  __device__ void next(Place& x) const {
    x.tile = 0;
    if (++x.h < p.cache.H) return;
    x.h = 0;
    if (++x.rt == p.row_tiles) {
      x.rt = 0;
      ++x.b;
    }
    if (x.b < seqs()) x.n = tiles(x.b, x.rt);
  }
  // The lengths of the launch's sequences, cut to what their table can hold.
  __device__ void load_lengths(int* len) const {
    for (int i = threadIdx.x; i < p.B; i += blockDim.x) len[i] = max(0, min(p.room, __ldg(p.lens + i)));
  }
  // One warp: off[b] = tiles of the sequences before b, for one key/value head.
  __device__ void sum_tiles(long long* off, int lane) const {
    long long base = 0;
    for (int b0 = 0; b0 < seqs(); b0 += 32) {
      long long n = 0;
      if (b0 + lane < seqs())
        for (int rt = 0; rt < p.row_tiles; ++rt) n += tiles(b0 + lane, rt);
      long long sum = n;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long up = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += up;
      }
      if (b0 + lane < seqs()) off[b0 + lane] = base + sum - n;
      base += __shfl_sync(0xFFFFFFFFu, sum, 31);
    }
    if (lane == 0) off[seqs()] = base;
  }
  // Where a segment's result goes if it is not written out.
  __device__ int slot(const Place& x, bool whole) const {
    if (whole) return 2 * static_cast<int>(gridDim.x) + unit(x);
    return 2 * static_cast<int>(blockIdx.x) + (x.tile > 0 ? 0 : 1);
  }
  // For the merge kernel, by one thread where a unit begins: how many CTAs have a
  // part of it.  f: flat index of its first tile, per: tiles of a CTA.
  __device__ void tell(const Place& x, bool whole, long long f, long long per) const {
    if (x.tile != 0) return;
    const int ctas = static_cast<int>((f + x.n - 1) / per) - static_cast<int>(blockIdx.x) + 1;
    if (p.keep)
      p.info[unit(x)] = make_int2(blockIdx.x, whole ? 0 : ctas);
    else if (!whole)
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

// Four INT8 codes (one word) -> two pairs of fp16: code + 128 is put into the
// low bits of 1024 and 1152 taken off again, both exact.
__device__ __forceinline__ void k_codes_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  const uint32_t u = w ^ 0x80808080u;
  lo = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4140), 0x64806480u);
  hi = sub_f16x2(__byte_perm(u, 0x64646464u, 0x4342), 0x64806480u);
}

// The launch of the kernel for many query rows (cache_attention_wide.cu): 256
// rows and 128 keys a tile, one CTA on each SM.
constexpr int kWideRows = 256, kWideTok = 128;
cudaError_t launch_wide(const Params& p, bool prefix, unsigned ctas, cudaStream_t stream);

}  // namespace sage::cache
