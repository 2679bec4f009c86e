// kv_rows.cuh -- rows of the quantised KV cache (one token of one key/value head,
// 128 channels), formed by eight lanes: shared by the kernels that write them.
#pragma once

#include <cuda_runtime.h>

#include "qk_codes.cuh"
#include "sage_internal.cuh"
#include "sm103_ptx.cuh"

namespace sage::rows {

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

// One row of eight lanes put into the cache in 8 bits: w0 and w1 are channels 8 c0 ..
// + 7 and 8 c1 .. + 7 of the lane's row, l = lane % 8.  All lanes of a warp together;
// row < 0: nothing is written.
template <bool kIsV>
__device__ __forceinline__ void write_rows(const uint4& w0, const uint4& w1, uint8_t* codes, float* scales, int64_t row,
                                           int l, int c0, int c1) {
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
  const uint2 lo = encode<kIsV>(w0, sc, nr, in_range), hi = encode<kIsV>(w1, sc, nr, in_range);
  if (row >= 0) {
    uint2* dst = reinterpret_cast<uint2*>(codes + row * kHeadDim);
    dst[c0] = lo;
    dst[c1] = hi;
    if (l == 0) scales[row] = sc;
  }
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

// ------------------------------------------------------------- 4-bit rows --
//
//   scale = 2^k, the least that has max |x| <= 2688 * 2^k (2688 = 6 * 448), k >= -126
//   sb    = e4m3_rn(fl(max over 16 channels of |x| * 2^-k / 6))
//   code  = e2m1_rn(fl(x * 2^-k / sb)),  0 where sb = 0       fl: fp32, nearest even
//
// A power of two for the row loses nothing (the E4M3 scales have the same precision
// over 2^15 below the largest) and makes x * 2^-k exact.

// Eight E2M1 codes (channel 0 in the low four bits), ties to even, at most 6.
__device__ __forceinline__ uint32_t cvt_e2m1x8(const float2 (&y)[4]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(y[0].x), "f"(y[0].y), "f"(y[1].x), "f"(y[1].y), "f"(y[2].x), "f"(y[2].y), "f"(y[3].x), "f"(y[3].y));
  return r;
}

// fl(1 / sb) of a block's scale, 0 for 0: one Newton step from the hardware's
// approximation, which is within an ulp.  (Of the eight significands that E4M3 has,
// that gives the rounded value from as far as three ulp.)
__device__ __forceinline__ float inverse(float sb) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(sb));
  r = fmaf(r, fmaf(-sb, r, 1.0f), r);
  return sb > 0.0f ? r : 0.0f;
}

// The codes of the 8 bf16 values of w, times `inv` (a power of two), over sb; 0 if that
// is 0.
__device__ __forceinline__ uint32_t encode4(const uint4& w, float inv, float sb) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
  const float nr = -inverse(sb);
  const float2 n2 = make_float2(nr, nr), s2 = make_float2(sb, sb), i2 = make_float2(inv, inv);
  float2 y[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {                 // -fl(x / sb), as above
    const float2 x = fmul2v(make_float2(bf16_lo(u[i]), bf16_hi(u[i])), i2);
    const float2 z = fmul2v(x, n2);
    y[i] = ffma2v(ffma2v(z, s2, x), n2, z);
  }
  return sb > 0.0f ? cvt_e2m1x8(y) ^ 0x88888888u : 0u;
}

// fl(x / 6) for the x that count, 0 or 2^-100 .. 2688: a product with fl(1 / 6) and
// Markstein's correction (smaller ones are 0 in E4M3 either way).
__device__ __forceinline__ float sixth(float x) {
  constexpr float r = 1.0f / 6.0f;
  const float q = x * r;
  return fmaf(fmaf(q, -6.0f, x), r, q);
}

__device__ __forceinline__ uint32_t top_of(const uint4& w) {
  const uint32_t m = 0x7FFF7FFFu;
  return max_u16x2(max_u16x2(w.x & m, w.y & m), max_u16x2(w.z & m, w.w & m));
}

// write_rows for 4 bits, of rows of 16 / kN lanes: a lane has the chunks c[i] in w[i], and
// those of lanes l and l ^ 1 are one block of 16 channels.
template <int kN>
__device__ __forceinline__ void write_rows4(const uint4 (&w)[kN], uint8_t* codes, uint8_t* blocks, float* scales, int64_t row,
                                            int l, const int (&c)[kN]) {
  uint32_t t[kN], top = 0u;
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    t[i] = top_of(w[i]);
    t[i] = max_u16x2(t[i], __shfl_xor_sync(0xFFFFFFFFu, t[i], 1));
    top = max_u16x2(top, t[i]);
  }
#pragma unroll
  for (int d = 2; d < 16 / kN; d <<= 1) top = max_u16x2(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  top = max(top & 0xFFFFu, top >> 16);
  // A row of zeros or with an infinity or a NaN: blocks and codes 0.
  const bool some = top > 0u && top < 0x7F80u;
  // 2688 = (1 + 40 / 128) * 2^11
  const uint32_t field = static_cast<uint32_t>(max(1, static_cast<int>(top >> 7) - 11 + ((top & 0x7Fu) > 40u ? 1 : 0)));
  const float inv = __uint_as_float((254u - field) << 23);
  uint32_t block[kN], code[kN];
#pragma unroll
  for (int i = 0; i < kN; i += 2) {
    float x[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) x[e] = sixth(some ? __uint_as_float(max(t[i + e] << 16, t[i + e] & 0xFFFF0000u)) * inv : 0.0f);
    const uint32_t both = cvt_e4m3x2(x[0], x[1]);
    const float2 sb = e4m3x2_to_f32(both);
    block[i] = both & 0xFFu;
    block[i + 1] = both >> 8;
    code[i] = encode4(w[i], inv, sb.x);
    code[i + 1] = encode4(w[i + 1], inv, sb.y);
  }
  if (row >= 0) {
    uint32_t* dst = reinterpret_cast<uint32_t*>(codes + row * 64);
#pragma unroll
    for (int i = 0; i < kN; ++i) dst[c[i]] = code[i];
    if ((l & 1) == 0) {
#pragma unroll
      for (int i = 0; i < kN; ++i) blocks[row * 8 + (c[i] >> 1)] = static_cast<uint8_t>(block[i]);
    }
    if (l == 0) scales[row] = some ? __uint_as_float(field << 23) : top == 0u ? 0.0f : __uint_as_float(0x7FC00000u);
  }
}

// Eight codes -> eight fp32 values, in channel order.
__device__ __forceinline__ void e2m1x8_to_f32(uint32_t w, float (&y)[8]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
    y[2 * i] = f.x;
    y[2 * i + 1] = f.y;
  }
}

// K's and V's row `row` of a cache of kBits.
template <int kBits, bool kIsV>
__device__ __forceinline__ void put_row(const CacheView& c, const uint4& w0, const uint4& w1, int64_t row, int l, int c0, int c1) {
  if constexpr (kBits == 8)
    write_rows<kIsV>(w0, w1, kIsV ? c.v_codes : c.k_codes, kIsV ? c.v_scale : c.k_scale, row, l, c0, c1);
  else
    write_rows4<2>({w0, w1}, kIsV ? c.v_codes : c.k_codes, kIsV ? c.v_block : c.k_block, kIsV ? c.v_scale : c.k_scale, row, l,
                   {c0, c1});
}

}  // namespace sage::rows
