// kv_cache.cu -- writing K and V into the paged quantised cache, and reading
// them back (sm_103a).
//
// A row is one token of one key/value head, 128 channels.  As in the
// quantisation of whole sequences (quantize.cu) K becomes INT8 and V E4M3, but
// each row has scales of its own, since tokens arrive one at a time and a block
// scale would have to requantise what is in the cache already:
//
//   sk = fl(max |k| / 127),  kc = clamp(rint(fl(k / sk)), -127, 127)
//   sv = fl(max |v| / 448),  vc = e4m3_rn(fl(v / sv))         fl: fp32, nearest even
//
// A row of zeros has scale 0 and codes 0; a row that holds an infinity or a
// NaN has a NaN scale and codes 0, so that it reads back as NaN and reaches
// nothing but what attends to it.  Reading back gives bf16(fl(code * scale)).
//
// Both kernels are bound by HBM: 512 bytes of bf16 and 264 bytes of codes and
// scales per row.  Eight lanes take a row, 16 channels each, and the four rows
// of a warp are consecutive tokens of one head, whose codes and scales lie
// together in a page; a warp does its K and then its V, so that no lane waits
// for the other formula.  The quotients go through a reciprocal and one correction,
// two at a time (2 x 32760 tokens of 16 heads: 130 us; by division 390).  That write moves
// 814 MB at 6.3 TB/s, 0.92 of the measured copy rate; 4 x 16384 tokens of 8 heads are read
// back in 62 us, 0.93 of it.  Small calls cost a launch and three loads in a row (start or
// length, page, row): 5.6 us for 8 tokens, 4.4 us for 3 x 333 read.
//
// In 4 bits (kv_rows.cuh has the formulas) a row is 76 bytes.  Reading it back is bound by
// HBM, writing by the latency of its loads: a warp asks for one step's rows, waits and
// computes with none in flight (the first of its stalls; 0.64 of the issue slots taken, DRAM at
// 47%).  4 x up to 16384 tokens of 8 heads: 38 us (0.73 of the copy rate) and 49 us (0.94).
#include <cuda_runtime.h>

#include "kv_rows.cuh"

namespace sage {

namespace {

using namespace rows;

constexpr int kWarps = 8;      // per CTA
constexpr int kRows = 4;       // tokens of one step of a warp

// Row index of token `pos` of sequence b and head h in the cache, or -1 where
// the table or the cache does not reach: the caller then skips the row.
__device__ __forceinline__ int64_t cache_row(const CacheView& c, const PageTable& t, int b, int64_t pos, int h) {
  if (pos < 0) return -1;
  const int64_t i = pos >> c.page_shift;
  if (i >= t.width) return -1;
  const int page = __ldg(t.pages + b * t.stride + i);
  if (page < 0 || page >= c.num_pages) return -1;
  return (((static_cast<int64_t>(page) * c.H + h) << c.page_shift) + (pos & ((1 << c.page_shift) - 1)));
}

// The rows of step i of a warp: head h, tokens kTokens j and on of sequence b, the
// head running fastest, then j.
struct Step {
  int b, s, h;
};
template <int kTokens>
__device__ __forceinline__ Step step_of(uint32_t i, int H, int steps_per_seq) {
  Step x;
  const uint32_t j = i / static_cast<uint32_t>(H);
  x.h = static_cast<int>(i - j * H);
  x.b = static_cast<int>(j / static_cast<uint32_t>(steps_per_seq));
  x.s = static_cast<int>(j - x.b * static_cast<uint32_t>(steps_per_seq)) * kTokens;
  return x;
}

__global__ void __launch_bounds__(kWarps * 32) kv_cache_write_kernel(const CacheWriteArgs a, uint32_t steps,
                                                                     int steps_per_seq) {
  const uint32_t i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= steps) return;                  // warp-uniform
  const int lane = threadIdx.x & 31, l = lane & 7;
  Step x = step_of<kRows>(i, a.cache.H, steps_per_seq);
  x.s += lane >> 3;
  const bool live = x.s < a.S && (a.count == nullptr || x.s < __ldg(a.count + x.b));
  uint4 k0 = make_uint4(0u, 0u, 0u, 0u), k1 = k0, v0 = k0, v1 = k0;
  if (live) {
    const uint4* k = reinterpret_cast<const uint4*>(a.k + x.b * a.k_sb + x.s * a.k_ss + x.h * kHeadDim) + l;
    const uint4* v = reinterpret_cast<const uint4*>(a.v + x.b * a.v_sb + x.s * a.v_ss + x.h * kHeadDim) + l;
    k0 = __ldcs(k);
    k1 = __ldcs(k + 8);
    v0 = __ldcs(v);
    v1 = __ldcs(v + 8);
  }
  const int64_t row = live ? cache_row(a.cache, a.table, x.b, static_cast<int64_t>(__ldg(a.start + x.b)) + x.s, x.h) : -1;
  if (live && row < 0 && l == 0) atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
  put_row<8, false>(a.cache, k0, k1, row, l, l, l + 8);
  put_row<8, true>(a.cache, v0, v1, row, l, l, l + 8);
}

// 16 channels of a row to bf16, one 32-byte store.
__device__ __forceinline__ void store_row(uint16_t* dst, const float (&x)[16], float sc) {
  uint32_t w[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = pack_bf16(x[2 * i] * sc, x[2 * i + 1] * sc);
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
               "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}

__global__ void __launch_bounds__(kWarps * 32) kv_cache_read_kernel(const CacheReadArgs a, uint32_t steps,
                                                                    int steps_per_seq) {
  const uint32_t i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= steps) return;                  // warp-uniform
  const int lane = threadIdx.x & 31, l = lane & 7;
  Step x = step_of<kRows>(i, a.cache.H, steps_per_seq);
  x.s += lane >> 3;
  if (x.s >= a.S) return;
  uint4 kc = make_uint4(0u, 0u, 0u, 0u), vc = kc;
  float ks = 0.0f, vs = 0.0f;
  if (x.s < __ldg(a.lens + x.b)) {
    const int64_t row = cache_row(a.cache, a.table, x.b, x.s, x.h);
    if (row >= 0) {
      kc = __ldcs(reinterpret_cast<const uint4*>(a.cache.k_codes + row * kHeadDim) + l);
      vc = __ldcs(reinterpret_cast<const uint4*>(a.cache.v_codes + row * kHeadDim) + l);
      ks = __ldg(a.cache.k_scale + row);
      vs = __ldg(a.cache.v_scale + row);
    } else if (l == 0) {
      atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
    }
  }
  const int64_t dst = ((static_cast<int64_t>(x.b) * a.S + x.s) * a.cache.H + x.h) * kHeadDim + l * 16;
  const uint32_t kw[4] = {kc.x, kc.y, kc.z, kc.w}, vw[4] = {vc.x, vc.y, vc.z, vc.w};
  float y[16];
  // byte + 128 in the low bits of 2^23 is exact: no integer conversion.
#pragma unroll
  for (int e = 0; e < 16; ++e)
    y[e] = __uint_as_float(__byte_perm(kw[e >> 2] ^ 0x80808080u, 0x4B000000u, 0x7440 + (e & 3))) - 8388736.0f;
  store_row(a.k + dst, y, ks);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const float2 two = e4m3x2_to_f32(vw[e >> 1] >> (16 * (e & 1)));
    y[2 * e] = two.x;
    y[2 * e + 1] = two.y;
  }
  store_row(a.v + dst, y, vs);
}

// The same into 4 bits.  Eight tokens a warp, four lanes and 32 channels each: what a
// row needs once is shared by twice as many as above (4 x up to 16384 tokens of 8 heads:
// 38 us; by eight lanes a row 45).
constexpr int kRows4 = 8;
__global__ void __launch_bounds__(kWarps * 32) kv4_cache_write_kernel(const CacheWriteArgs a, uint32_t steps,
                                                                      int steps_per_seq) {
  const uint32_t i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= steps) return;                  // warp-uniform
  const int lane = threadIdx.x & 31, l = lane & 3;
  Step x = step_of<kRows4>(i, a.cache.H, steps_per_seq);
  x.s += lane >> 2;
  const bool live = x.s < a.S && (a.count == nullptr || x.s < __ldg(a.count + x.b));
  if (!__any_sync(0xFFFFFFFFu, live)) return;
  uint4 k[4], v[4];
  const int c[4] = {l, l + 4, l + 8, l + 12};
#pragma unroll
  for (int j = 0; j < 4; ++j) k[j] = v[j] = make_uint4(0u, 0u, 0u, 0u);
  if (live) {
    const uint4* kp = reinterpret_cast<const uint4*>(a.k + x.b * a.k_sb + x.s * a.k_ss + x.h * kHeadDim);
    const uint4* vp = reinterpret_cast<const uint4*>(a.v + x.b * a.v_sb + x.s * a.v_ss + x.h * kHeadDim);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      k[j] = __ldcs(kp + c[j]);
      v[j] = __ldcs(vp + c[j]);
    }
  }
  const int64_t row = live ? cache_row(a.cache, a.table, x.b, static_cast<int64_t>(__ldg(a.start + x.b)) + x.s, x.h) : -1;
  if (live && row < 0 && l == 0) atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
  write_rows4<4>(k, a.cache.k_codes, a.cache.k_block, a.cache.k_scale, row, l, c);
  write_rows4<4>(v, a.cache.v_codes, a.cache.v_block, a.cache.v_scale, row, l, c);
}

// Reading back from 4 bits: eight bytes of codes and one block scale a lane.
__global__ void __launch_bounds__(kWarps * 32) kv4_cache_read_kernel(const CacheReadArgs a, uint32_t steps,
                                                                     int steps_per_seq) {
  const uint32_t i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= steps) return;                  // warp-uniform
  const int lane = threadIdx.x & 31, l = lane & 7;
  Step x = step_of<kRows>(i, a.cache.H, steps_per_seq);
  x.s += lane >> 3;
  if (x.s >= a.S) return;
  uint2 kc = make_uint2(0u, 0u), vc = kc;
  uint32_t kb = 0u, vb = 0u;
  float ks = 0.0f, vs = 0.0f;
  if (x.s < __ldg(a.lens + x.b)) {
    const int64_t row = cache_row(a.cache, a.table, x.b, x.s, x.h);
    if (row >= 0) {
      kc = __ldcs(reinterpret_cast<const uint2*>(a.cache.k_codes + row * 64) + l);
      vc = __ldcs(reinterpret_cast<const uint2*>(a.cache.v_codes + row * 64) + l);
      kb = __ldcs(a.cache.k_block + row * 8 + l);
      vb = __ldcs(a.cache.v_block + row * 8 + l);
      ks = __ldg(a.cache.k_scale + row);
      vs = __ldg(a.cache.v_scale + row);
    } else if (l == 0) {
      atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
    }
  }
  const int64_t dst = ((static_cast<int64_t>(x.b) * a.S + x.s) * a.cache.H + x.h) * kHeadDim + l * 16;
  auto store = [&](uint16_t* to, const uint2& c, uint32_t block, float sc) {
    float lo[8], hi[8], y[16];
    e2m1x8_to_f32(c.x, lo);
    e2m1x8_to_f32(c.y, hi);
    const float sb = e4m3x2_to_f32(block).x;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = lo[e] * sb;                     // 6 significant bits: exact
      y[8 + e] = hi[e] * sb;
    }
    store_row(to + dst, y, sc);
  };
  store(a.k, kc, kb, ks);
  store(a.v, vc, vb, vs);
}

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args, uint32_t, int), int tokens, const Args& a, cudaStream_t stream) {
  const int per_seq = (a.S + tokens - 1) / tokens;
  const uint32_t steps = static_cast<uint32_t>(a.B) * per_seq * a.cache.H;
  kernel<<<(steps + kWarps - 1) / kWarps, kWarps * 32, 0, stream>>>(a, steps, per_seq);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_cache_write(const CacheWriteArgs& a, cudaStream_t stream) {
  return a.cache.bits == 8 ? launch_rows(kv_cache_write_kernel, kRows, a, stream) : launch_rows(kv4_cache_write_kernel, kRows4, a, stream);
}

cudaError_t launch_kv_cache_read(const CacheReadArgs& a, cudaStream_t stream) {
  return launch_rows(a.cache.bits == 8 ? kv_cache_read_kernel : kv4_cache_read_kernel, kRows, a, stream);
}

}  // namespace sage
