// qk_rope.cu -- RMS norms of each head of Q and K with the rotation of their
// positions in one pass, to bf16 or straight into the paged KV cache (sm_103a).
//
// A row is one token of one head, x its 128 channels, w the head norm's weights:
//
//   n   = x * w / sqrt(mean x^2 + eps)                      (n = x without a norm)
//   (y_a, y_b) = (n_a cos - n_b sin, n_a sin + n_b cos)     for each pair (a, b)
//
// with the pairs (2i, 2i + 1) or (i, i + R / 2) of the first R channels, the others
// as they are.  The angle of pair i at position p is p * f_i.  F_i = f_i / (2 pi) in
// 2^-64 stands in the table, so that p * F_i modulo 2^64 is the angle in revolutions
// with nothing lost, however far the position; its upper half goes to sine and
// cosine.  They take the weights, and the norm's factor comes last.
//
// Bound by HBM: 512 bytes a row of Q (and of K to bf16): 32760 tokens of 40 + 40 heads
// 221 us, 6.1 TB/s, 0.90 of the measured copy rate; 15000 packed tokens of 32 + 8 + 8
// heads into 8 bits 67 us, 0.74.  48 tokens take 3.6 us: a launch, the slot or the
// position, a row.  Eight lanes take a row, 16
// channels each, chosen so that a lane holds both channels of its pairs whichever
// way they are laid out: nothing crosses lanes but the norm's sum.  The sines and
// cosines of a token, times the weights, are formed once for up to 16 heads of one of
// q, k and v, eight pairs a lane, and the arithmetic goes two values at a time: one
// value at a time it took 240 instructions for four rows, and the issue slots, not HBM,
// were the bound.
#include <algorithm>
#include <type_traits>
#include <cuda_runtime.h>

#include "kv_rows.cuh"

namespace sage {

namespace {

using namespace rows;

constexpr int kWarps = 4;      // per CTA
constexpr int kTokens = 4;     // of a warp
constexpr int kAhead = 2;      // heads on their way while one is in hand
constexpr int kMaxHeads = 16;  // of a warp

// A lane's place in its rows: chunks (8 channels) c0 and c1, both channels of the
// pairs (i, i + R / 2) in the same place of both; lanes from R / 16 on hold the channels
// that are not rotated.  With R a multiple of 32 the chunks c0 of lanes l and l ^ 1
// lie together, and so do their c1, as the 4-bit rows want it.
struct Lane {
  int l, c0, c1;
  bool turns;
  __device__ Lane(int lane, int rot) {
    l = lane & 7;
    const int n = rot >> 4;
    turns = l < n;
    c0 = turns ? l : n + l;                  // 2n .. n + 7, then 8 + n .. 15: of the last 16 - 2n chunks
    c1 = turns ? n + l : 8 + l;
  }
};

// A lane's eight pairs, two at a time: (a, b) becomes (a ac - b bs, a as + b bc), the
// sines and cosines times the weights of a and b.
struct Turn {
  float2 ac[4], bs[4], as[4], bc[4];
};

// Which channels a lane's words hold: of words 0 .. 3 (chunk c0) and 4 .. 7 (c1), in the
// half layout pair 2i + e is channel 2i + e of both chunks; interleaved, pair j is
// both channels of word j.
template <bool kInterleaved>
__device__ __forceinline__ void unpack(const uint4& w0, const uint4& w1, float2 (&a)[4], float2 (&b)[4]) {
  const uint32_t u[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInterleaved) {
      a[i] = make_float2(bf16_lo(u[2 * i]), bf16_lo(u[2 * i + 1]));
      b[i] = make_float2(bf16_hi(u[2 * i]), bf16_hi(u[2 * i + 1]));
    } else {
      a[i] = make_float2(bf16_lo(u[i]), bf16_hi(u[i]));
      b[i] = make_float2(bf16_lo(u[4 + i]), bf16_hi(u[4 + i]));
    }
  }
}
template <bool kInterleaved>
__device__ __forceinline__ void pack(const float2 (&a)[4], const float2 (&b)[4], uint4& w0, uint4& w1) {
  uint32_t u[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (kInterleaved) {
      u[2 * i] = pack_bf16(a[i].x, b[i].x);
      u[2 * i + 1] = pack_bf16(a[i].y, b[i].y);
    } else {
      u[i] = pack_bf16(a[i].x, a[i].y);
      u[4 + i] = pack_bf16(b[i].x, b[i].y);
    }
  }
  w0 = make_uint4(u[0], u[1], u[2], u[3]);
  w1 = make_uint4(u[4], u[5], u[6], u[7]);
}

// The coefficients of the token at `pos` for this lane; a lane that does not turn its
// channels has their weights in ac and bc.
template <bool kInterleaved>
__device__ __forceinline__ void turn_of(const RopeView& r, const int32_t* pos, const Lane& at, const uint16_t* weight, bool live,
                                        Turn& z) {
  float2 ga[4], gb[4];
  const uint4 one = make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  const uint4* g = reinterpret_cast<const uint4*>(weight);
  unpack<kInterleaved>(weight ? __ldg(g + at.c0) : one, weight ? __ldg(g + at.c1) : one, ga, gb);
  int64_t p[kMaxAxes];
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) p[a] = a < r.axes && live ? __ldg(pos + a) : 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float s[2] = {0.0f, 0.0f}, c[2] = {1.0f, 1.0f};
    if (at.turns) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int j = 2 * i + e, pair = kInterleaved ? 4 * (j < 4 ? at.c0 : at.c1) + (j & 3) : 8 * at.c0 + j;
        const uint64_t f = __ldg(reinterpret_cast<const unsigned long long*>(r.freq) + pair);
        int64_t mine = p[0];
#pragma unroll
        for (int a = 1; a < kMaxAxes; ++a)
          if (pair >= r.ends[a - 1]) mine = p[a];
        const uint64_t angle = static_cast<uint64_t>(mine) * f;
        sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &s[e], &c[e]);
        s[e] *= r.factor;
        c[e] *= r.factor;
      }
    }
    const float2 s2 = make_float2(s[0], s[1]), c2 = make_float2(c[0], c[1]);
    z.ac[i] = fmul2v(ga[i], c2);
    z.as[i] = fmul2v(ga[i], s2);
    z.bc[i] = fmul2v(gb[i], c2);
    z.bs[i] = fmul2v(make_float2(-gb[i].x, -gb[i].y), s2);     // negated
  }
}

// One row: norm, weights and rotation.
template <bool kInterleaved>
__device__ __forceinline__ void turn_row(uint4& w0, uint4& w1, bool norm, float eps, bool turns, const Turn& z) {
  if (!norm && !turns) return;               // as they are, a NaN's bits too; without a norm no lane is waited for
  float2 a[4], b[4];
  unpack<kInterleaved>(w0, w1, a, b);
  float by = 1.0f;
  if (norm) {
    float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = ffma2v(a[i], a[i], ffma2v(b[i], b[i], sum));
    float all = sum.x + sum.y;
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) all += __shfl_xor_sync(0xFFFFFFFFu, all, d);
    by = rsqrtf(all * (1.0f / kHeadDim) + eps);
  }
  const float2 by2 = make_float2(by, by);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 x, y;
    if (turns) {
      x = ffma2v(a[i], z.ac[i], fmul2v(b[i], z.bs[i]));
      y = ffma2v(a[i], z.as[i], fmul2v(b[i], z.bc[i]));
    } else {
      x = fmul2v(a[i], z.ac[i]);
      y = fmul2v(b[i], z.bc[i]);
    }
    a[i] = fmul2v(x, by2);
    b[i] = fmul2v(y, by2);
  }
  pack<kInterleaved>(a, b, w0, w1);
}

// Heads [h0, h1) of one tensor at src, loaded kAhead ahead; `put` has each row.
template <bool kInterleaved, bool kTurn, typename Put>
__device__ __forceinline__ void run_heads(const uint16_t* src, int h0, int h1, bool live, const Lane& at, const TurnArgs& a,
                                          const Turn& z, Put put) {
  auto load = [&](int h, uint4 (&w)[2]) {
    w[0] = w[1] = make_uint4(0u, 0u, 0u, 0u);
    if (live && h < h1) {
      const uint4* row = reinterpret_cast<const uint4*>(src + h * kHeadDim);
      w[0] = __ldcs(row + at.c0);
      w[1] = __ldcs(row + at.c1);
    }
  };
  uint4 next[kAhead][2];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(h0 + i, next[i]);
  for (int h = h0; h < h1; h += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (h + i >= h1) break;
      uint4 w[2] = {next[i][0], next[i][1]};
      load(h + i + kAhead, next[i]);
      if constexpr (kTurn) turn_row<kInterleaved>(w[0], w[1], a.norm, a.eps, at.turns, z);
      put(h + i, w[0], w[1]);
    }
  }
}

// Parts of a token's heads: of q, of k, of v, each of `heads` at most.
struct Split {
  int parts[3], heads[3];
};

// kBits 0: q and k to bf16; 8 or 4: q to bf16, k and v into a cache of so many.
template <int kBits, bool kInterleaved>
__global__ void __launch_bounds__(kWarps * 32, 5) turn_kernel(const TurnArgs a, const Split split, uint32_t items) {
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= items) return;                 // warp-uniform
  const uint32_t all = split.parts[0] + split.parts[1] + split.parts[2], group = item / all;
  int part = static_cast<int>(item - group * all), which = 0;
  if (part >= split.parts[0]) {
    part -= split.parts[0];
    which = 1;
    if (part >= split.parts[1]) {
      part -= split.parts[1];
      which = 2;
    }
  }
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(group) * kTokens + (lane >> 3);
  const bool live = t < static_cast<int64_t>(a.B) * a.S;
  const int b = live ? static_cast<int>(static_cast<uint32_t>(t) / static_cast<uint32_t>(a.S)) : 0;
  const int s = live ? static_cast<int>(t - static_cast<int64_t>(b) * a.S) : 0;
  const Lane at(lane, a.rope.rot);
  const int per = which == 0 ? split.heads[0] : which == 1 ? split.heads[1] : split.heads[2];
  const int h0 = part * per, h1 = min(h0 + per, which == 0 ? a.Hq : a.Hk);

  if (kBits == 0 || which == 0) {
    const uint16_t* src = which == 0 ? a.q + b * a.q_sb + s * a.q_ss : a.k + b * a.k_sb + s * a.k_ss;
    uint16_t* out = which == 0 ? a.q_out + t * a.Hq * kHeadDim : a.k_out + t * a.Hk * kHeadDim;
    Turn z;
    turn_of<kInterleaved>(a.rope, a.positions + b * a.p_sb + s * a.p_ss, at, which == 0 ? a.q_weight : a.k_weight, live, z);
    run_heads<kInterleaved, true>(src, h0, h1, live, at, a, z, [&](int h, const uint4& w0, const uint4& w1) {
      if (!live) return;
      uint4* row = reinterpret_cast<uint4*>(out + h * kHeadDim);
      row[at.c0] = w0;
      row[at.c1] = w1;
    });
  }
  if constexpr (kBits != 0) {
    if (which == 0) return;
    int64_t row0 = -1;                       // of head 0
    const int ps = a.cache.page_shift;
    if (live) {
      const int slot = __ldg(a.slots + t), page = slot >> ps;
      if (slot >= 0 && page < a.cache.num_pages)
        row0 = ((static_cast<int64_t>(page) * a.cache.H) << ps) + (slot & ((1 << ps) - 1));
      else if (slot >= 0 && at.l == 0)
        atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
    }
    Turn z;
    if (which == 1) {
      turn_of<kInterleaved>(a.rope, a.positions + b * a.p_sb + s * a.p_ss, at, a.k_weight, live, z);
      run_heads<kInterleaved, true>(a.k + b * a.k_sb + s * a.k_ss, h0, h1, live, at, a, z, [&](int h, const uint4& w0, const uint4& w1) {
        put_row<kBits, false>(a.cache, w0, w1, row0 < 0 ? -1 : row0 + (static_cast<int64_t>(h) << ps), at.l, at.c0, at.c1);
      });
    } else {
      run_heads<kInterleaved, false>(a.v + b * a.v_sb + s * a.v_ss, h0, h1, live, at, a, z, [&](int h, const uint4& w0, const uint4& w1) {
        put_row<kBits, true>(a.cache, w0, w1, row0 < 0 ? -1 : row0 + (static_cast<int64_t>(h) << ps), at.l, at.c0, at.c1);
      });
    }
  }
}

}  // namespace

cudaError_t launch_turn(const TurnArgs& a, cudaStream_t stream) {
  const int bits = a.slots == nullptr ? 0 : a.cache.bits;
  const int H[3] = {a.Hq, a.Hk, bits == 0 ? 0 : a.Hk};
  const int64_t groups = (static_cast<int64_t>(a.B) * a.S + kTokens - 1) / kTokens;
  // Parts of up to 16 heads, so that there are few sines, or of fewer while all warps are
  // resident at once (20 on an SM; 2 x 333 tokens of 24 + 24 heads: parts of four 4.8 us, of
  // two, in two waves, 6.1).
  const auto parts_of = [&](int per, int i) { return H[i] / per + (H[i] % per != 0 ? 1 : 0); };
  const auto warps = [&](int per) { return groups * (static_cast<int64_t>(parts_of(per, 0)) + parts_of(per, 1) + parts_of(per, 2)); };
  int per = kMaxHeads;
  while (per > 1 && warps(per / 2) <= 152 * 20) per /= 2;
  Split split = {};
  for (int i = 0; i < 3; ++i) split.parts[i] = parts_of(per, i);
  for (int i = 0; i < 3; ++i) split.heads[i] = split.parts[i] == 0 ? 0 : H[i] / split.parts[i] + (H[i] % split.parts[i] != 0 ? 1 : 0);
  const uint32_t items = static_cast<uint32_t>(warps(per));
  const unsigned ctas = (items + kWarps - 1) / kWarps;
  auto go = [&](auto kernel) {
    kernel<<<ctas, kWarps * 32, 0, stream>>>(a, split, items);
    return cudaGetLastError();
  };
  if (a.rope.interleaved) return bits == 0 ? go(turn_kernel<0, true>) : bits == 8 ? go(turn_kernel<8, true>) : go(turn_kernel<4, true>);
  return bits == 0 ? go(turn_kernel<0, false>) : bits == 8 ? go(turn_kernel<8, false>) : go(turn_kernel<4, false>);
}

}  // namespace sage
