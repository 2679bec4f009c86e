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
#include <cuda_runtime.h>

#include "qk_codes.cuh"
#include "sage_internal.cuh"
#include "sm103_ptx.cuh"

namespace sage {

namespace {

constexpr int kWarps = 8;      // per CTA
constexpr int kRows = 4;       // tokens of one step of a warp

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float2 ffma2v(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 x, y, z, w;\n\t"
      "mov.b64 x, {%2, %3};\n\tmov.b64 y, {%4, %5};\n\tmov.b64 z, {%6, %7};\n\t"
      "fma.rn.f32x2 w, x, y, z;\n\tmov.b64 {%0, %1}, w;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

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

// -fl(x / sc) of the 8 bf16 values of w, for a scale in [2^-100, 2^125]:
// Markstein's correction with the negated reciprocal nr = -fl(1 / sc), as in
// quantize.cu's V encoder.
__device__ __forceinline__ void quotients(const uint4& w, float sc, float nr, float2 (&y)[4]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  const float2 n2 = make_float2(nr, nr), s2 = make_float2(sc, sc);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
    const float2 z = fmul2v(x, n2);
    y[i] = ffma2v(ffma2v(z, s2, x), n2, z);
  }
}

// Eight codes, in channel order, of values whose row has scale sc.
template <bool kIsV>
__device__ __forceinline__ uint2 encode(const uint4& w, float sc, float nr, bool in_range) {
  uint32_t code[2] = {0u, 0u};
  if (in_range) {
    float2 y[4];
    quotients(w, sc, nr, y);
    if constexpr (kIsV) {
#pragma unroll
      for (int i = 0; i < 2; ++i)
        code[i] = cvt_e4m3x4(y[2 * i].x, y[2 * i].y, y[2 * i + 1].x, y[2 * i + 1].y) ^ 0x80808080u;
    } else {
      // 1.5 * 2^23 - y: its low byte is the two's complement of rint(-y)
      // (ties to even on either side), at most 127 in magnitude since
      // |x| <= amax = 127 sc (1 + 2^-24).
      const float2 magic = make_float2(kRoundMagic, kRoundMagic);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 a = fsub2v(magic, y[2 * i]), b = fsub2v(magic, y[2 * i + 1]);
        const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
        code[i] = __byte_perm(lo, hi, 0x5410);
      }
    }
  } else if (sc > 0.0f) {        // outside the quotient's range: by division (a scale of 0 or NaN: codes 0)
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = (i & 1) ? bf16_hi(u[i >> 1]) : bf16_lo(u[i >> 1]);
      uint32_t byte;
      if constexpr (kIsV)
        byte = cvt_e4m3x2(__fdiv_rn(x, sc), 0.0f) & 0xFFu;
      else
        byte = (__float_as_uint(code_by_division(x, sc) + kRoundMagic) - 0x4B400000u) & 0xFFu;
      code[i >> 2] |= byte << (8 * (i & 3));
    }
  }
  return make_uint2(code[0], code[1]);
}

// The rows of step i of a warp: head h, tokens 4 j .. 4 j + 3 of sequence b, the
// head running fastest, then j.
struct Step {
  int b, s, h;
};
__device__ __forceinline__ Step step_of(uint32_t i, int H, int steps_per_seq) {
  Step x;
  const uint32_t j = i / static_cast<uint32_t>(H);
  x.h = static_cast<int>(i - j * H);
  x.b = static_cast<int>(j / static_cast<uint32_t>(steps_per_seq));
  x.s = static_cast<int>(j - x.b * static_cast<uint32_t>(steps_per_seq)) * kRows;
  return x;
}

// One tensor's part of a step: w0 and w1 are channels 8 l .. + 7 and 64 + 8 l ..
// + 7 of the lane's row, l = lane % 8.
template <bool kIsV>
__device__ __forceinline__ void write_rows(const uint4& w0, const uint4& w1, uint8_t* codes, float* scales, int64_t row,
                                           int l) {
  // Magnitudes compare as integers, infinities and NaN above all others.
  uint32_t top = 0u;
  const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
  for (int e = 0; e < 8; ++e) top = max_u16x2(top, u[e] & 0x7FFF7FFFu);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  top = max(top & 0xFFFFu, top >> 16);
  const float sc = top < 0x7F80u ? __fdiv_rn(__uint_as_float(top << 16), kIsV ? 448.0f : 127.0f) : __uint_as_float(0x7FC00000u);
  const bool in_range = sc >= 0x1p-100f && sc <= 0x1p125f;
  const float nr = -__frcp_rn(sc);
  const uint2 c0 = encode<kIsV>(w0, sc, nr, in_range), c1 = encode<kIsV>(w1, sc, nr, in_range);
  if (row >= 0) {
    uint2* dst = reinterpret_cast<uint2*>(codes + row * kHeadDim) + l;
    dst[0] = c0;
    dst[8] = c1;
    if (l == 0) scales[row] = sc;
  }
}

__global__ void __launch_bounds__(kWarps * 32) kv_cache_write_kernel(const CacheWriteArgs a, uint32_t steps,
                                                                     int steps_per_seq) {
  const uint32_t i = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (i >= steps) return;                  // warp-uniform
  const int lane = threadIdx.x & 31, l = lane & 7;
  Step x = step_of(i, a.cache.H, steps_per_seq);
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
  write_rows<false>(k0, k1, a.cache.k_codes, a.cache.k_scale, row, l);
  write_rows<true>(v0, v1, a.cache.v_codes, a.cache.v_scale, row, l);
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Two E4M3 codes -> two floats, exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t two) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(static_cast<uint16_t>(two)));
  float2 r;
  asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "r"(h2));
  return r;
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
  Step x = step_of(i, a.cache.H, steps_per_seq);
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

template <typename Args>
cudaError_t launch_rows(void (*kernel)(Args, uint32_t, int), const Args& a, cudaStream_t stream) {
  const int per_seq = (a.S + kRows - 1) / kRows;
  const uint32_t steps = static_cast<uint32_t>(a.B) * per_seq * a.cache.H;
  kernel<<<(steps + kWarps - 1) / kWarps, kWarps * 32, 0, stream>>>(a, steps, per_seq);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_cache_write(const CacheWriteArgs& a, cudaStream_t stream) {
  return launch_rows(kv_cache_write_kernel, a, stream);
}

cudaError_t launch_kv_cache_read(const CacheReadArgs& a, cudaStream_t stream) {
  return launch_rows(kv_cache_read_kernel, a, stream);
}

}  // namespace sage
