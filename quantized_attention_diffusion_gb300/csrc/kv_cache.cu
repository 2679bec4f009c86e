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
// scales per row.  One warp takes a row, lanes 0-15 its K and lanes 16-31 its
// V, 8 channels (16 bytes of bf16, 8 of codes) a lane, so that a row's maximum
// is four shuffles.
#include <cuda_runtime.h>

#include "qk_codes.cuh"
#include "sage_internal.cuh"
#include "sm103_ptx.cuh"

namespace sage {

namespace {

constexpr int kWarps = 8;      // per CTA

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

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

// Codes of 8 values of a K row (bytes in channel order).
__device__ __forceinline__ uint2 encode_k(const float (&x)[8], float sc) {
  const float rcp = __frcp_rn(sc);
  float c[8];
  codes8(x, sc, rcp, sc >= 0x1p-125f && sc <= 0x1p125f, c);
  uint32_t b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = (__float_as_uint(c[i] + kRoundMagic) - 0x4B400000u) & 0xFFu;
  return make_uint2(b[0] | (b[1] << 8) | (b[2] << 16) | (b[3] << 24), b[4] | (b[5] << 8) | (b[6] << 16) | (b[7] << 24));
}

// Codes of 8 values of a V row.  The quotient is formed as in quantize.cu's
// V encoder (Markstein's correction with the negated reciprocal gives
// -fl(x / sv) for scales in [2^-100, 2^125]), outside that range by division.
__device__ __forceinline__ uint2 encode_v(const float (&x)[8], float sv) {
  float y[8];
  if (sv >= 0x1p-100f && sv <= 0x1p125f) {
    const float nr = -__frcp_rn(sv);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float z = x[i] * nr;
      y[i] = -fmaf(fmaf(z, sv, x[i]), nr, z);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = sv == 0.0f ? 0.0f : __fdiv_rn(x[i], sv);
  }
  return make_uint2(cvt_e4m3x4(y[0], y[1], y[2], y[3]), cvt_e4m3x4(y[4], y[5], y[6], y[7]));
}

// kRows rows a warp, their loads all in flight before the first is used.
template <int kRows>
__global__ void __launch_bounds__(kWarps * 32) kv_cache_write_kernel(const CacheWriteArgs a) {
  const int lane = threadIdx.x & 31;
  const bool is_v = lane >= 16;
  const int c8 = (lane & 15) * 8;
  const uint32_t total = static_cast<uint32_t>(a.B) * a.S * a.cache.H;      // < 2^31
  const uint32_t r0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows;
  if (r0 >= total) return;
  int h = static_cast<int>(r0 % a.cache.H);
  int s = static_cast<int>(r0 / a.cache.H % a.S);
  int b = static_cast<int>(r0 / a.cache.H / a.S);
  uint4 raw[kRows];
  int64_t row[kRows];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    raw[i] = make_uint4(0u, 0u, 0u, 0u);
    row[i] = -1;
    if (r0 + i < total) {
      const bool live = a.count == nullptr || s < __ldg(a.count + b);
      if (live) {
        const uint16_t* src = is_v ? a.v + b * a.v_sb + s * a.v_ss : a.k + b * a.k_sb + s * a.k_ss;
        raw[i] = __ldcs(reinterpret_cast<const uint4*>(src + h * kHeadDim + c8));
        row[i] = cache_row(a.cache, a.table, b, static_cast<int64_t>(__ldg(a.start + b)) + s, h);
        bad |= row[i] < 0;
      }
      if (++h == a.cache.H) {
        h = 0;
        if (++s == a.S) {
          s = 0;
          ++b;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    // Magnitudes compare as integers, infinities and NaN above all others.
    uint32_t top = 0u;
#pragma unroll
    for (int e = 0; e < 4; ++e) top = max(top, max(w[e] & 0x7FFFu, (w[e] >> 16) & 0x7FFFu));
#pragma unroll
    for (int off = 8; off > 0; off >>= 1) top = max(top, __shfl_xor_sync(0xFFFFFFFFu, top, off));
    const bool finite = top < 0x7F80u;
    const float sc = finite ? __fdiv_rn(__uint_as_float(top << 16), is_v ? 448.0f : 127.0f) : __uint_as_float(0x7FC00000u);
    float x[8];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = bf16_lo(w[e]);
      x[2 * e + 1] = bf16_hi(w[e]);
    }
    uint2 code = make_uint2(0u, 0u);
    if (finite) code = is_v ? encode_v(x, sc) : encode_k(x, sc);
    if (row[i] >= 0) {
      *reinterpret_cast<uint2*>((is_v ? a.cache.v_codes : a.cache.k_codes) + row[i] * kHeadDim + c8) = code;
      if (c8 == 0) (is_v ? a.cache.v_scale : a.cache.k_scale)[row[i]] = sc;
    }
  }
  if (bad && lane == 0) atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
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

template <int kRows>
__global__ void __launch_bounds__(kWarps * 32) kv_cache_read_kernel(const CacheReadArgs a) {
  const int lane = threadIdx.x & 31;
  const bool is_v = lane >= 16;
  const int c8 = (lane & 15) * 8;
  const uint32_t total = static_cast<uint32_t>(a.B) * a.S * a.cache.H;      // < 2^31
  const uint32_t r0 = (blockIdx.x * kWarps + (threadIdx.x >> 5)) * kRows;
  if (r0 >= total) return;
  int h = static_cast<int>(r0 % a.cache.H);
  int s = static_cast<int>(r0 / a.cache.H % a.S);
  int b = static_cast<int>(r0 / a.cache.H / a.S);
  uint2 code[kRows];
  float sc[kRows];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    code[i] = make_uint2(0u, 0u);
    sc[i] = 0.0f;
    if (r0 + i < total) {
      if (s < __ldg(a.lens + b)) {
        const int64_t row = cache_row(a.cache, a.table, b, s, h);
        if (row >= 0) {
          code[i] = __ldcs(reinterpret_cast<const uint2*>((is_v ? a.cache.v_codes : a.cache.k_codes) + row * kHeadDim + c8));
          sc[i] = __ldg((is_v ? a.cache.v_scale : a.cache.k_scale) + row);
        }
        bad |= row < 0;
      }
      if (++h == a.cache.H) {
        h = 0;
        if (++s == a.S) {
          s = 0;
          ++b;
        }
      }
    }
  }
  uint16_t* dst = (is_v ? a.v : a.k) + static_cast<int64_t>(r0) * kHeadDim + c8;
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    if (r0 + i >= total) break;
    const uint32_t w[2] = {code[i].x, code[i].y};
    float x[8];
    if (is_v) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 p = e4m3x2_to_f32(w[e >> 1] >> (16 * (e & 1)));
        x[2 * e] = p.x;
        x[2 * e + 1] = p.y;
      }
    } else {
      // byte + 128 in the low bits of 2^23 is exact: no integer conversion.
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t u = ((w[e >> 2] ^ 0x80808080u) >> (8 * (e & 3))) & 0xFFu;
        x[e] = __uint_as_float(0x4B000000u | u) - 8388736.0f;
      }
    }
    uint4 o;
    o.x = pack_bf16(x[0] * sc[i], x[1] * sc[i]);
    o.y = pack_bf16(x[2] * sc[i], x[3] * sc[i]);
    o.z = pack_bf16(x[4] * sc[i], x[5] * sc[i]);
    o.w = pack_bf16(x[6] * sc[i], x[7] * sc[i]);
    __stcs(reinterpret_cast<uint4*>(dst + static_cast<int64_t>(i) * kHeadDim), o);
  }
  if (bad && lane == 0) atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
}

// Four rows a warp keep enough loads in flight once every SM has its warps;
// below that one row a warp spreads the rows over more SMs.
constexpr uint32_t kManyRows = 152u * 64u * 4u;

template <typename Args>
cudaError_t launch_rows(void (*one)(Args), void (*four)(Args), const Args& a, cudaStream_t stream) {
  const uint32_t total = static_cast<uint32_t>(a.B) * a.S * a.cache.H;
  const bool many = total >= kManyRows;
  const uint32_t per_cta = kWarps * (many ? 4u : 1u);
  (many ? four : one)<<<(total + per_cta - 1) / per_cta, kWarps * 32, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_cache_write(const CacheWriteArgs& a, cudaStream_t stream) {
  return launch_rows(kv_cache_write_kernel<1>, kv_cache_write_kernel<4>, a, stream);
}

cudaError_t launch_kv_cache_read(const CacheReadArgs& a, cudaStream_t stream) {
  return launch_rows(kv_cache_read_kernel<1>, kv_cache_read_kernel<4>, a, stream);
}

}  // namespace sage
