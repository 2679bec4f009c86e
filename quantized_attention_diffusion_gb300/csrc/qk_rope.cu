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
// cosine.  x * w is exact in fp32 (both bf16); the norm's factor comes last.
//
// Bound by HBM: 512 bytes a row of Q (and of K to bf16).  Eight lanes take a row, 16
// channels each, chosen so that a lane holds both channels of its pairs whichever
// way they are laid out: nothing crosses lanes but the norm's sum.  The sines and
// cosines of a token are formed once for up to 16 heads of it, eight pairs a lane.
#include <algorithm>
#include <type_traits>
#include <cuda_runtime.h>

#include "kv_rows.cuh"

namespace sage {

namespace {

using namespace rows;

constexpr int kWarps = 4;      // per CTA
constexpr int kTokens = 4;     // of a warp
constexpr int kAhead = 2;      // heads in flight
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

struct Turn {
  float cs[8], sn[8];
};

// The rotation of token t's pairs that this lane holds.
__device__ __forceinline__ void turn_of(const RopeView& r, const int32_t* pos, const Lane& at, Turn& z) {
  int64_t p[kMaxAxes];
#pragma unroll
  for (int a = 0; a < kMaxAxes; ++a) p[a] = a < r.axes ? __ldg(pos + a) : 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int pair = r.interleaved ? 4 * (j < 4 ? at.c0 : at.c1) + (j & 3) : 8 * at.c0 + j;
    const uint64_t f = __ldg(reinterpret_cast<const unsigned long long*>(r.freq) + pair);
    int64_t mine = p[0];
#pragma unroll
    for (int a = 1; a < kMaxAxes; ++a)
      if (pair >= r.ends[a - 1]) mine = p[a];
    const uint64_t angle = static_cast<uint64_t>(mine) * f;
    float s, c;
    sincospif(static_cast<float>(static_cast<int32_t>(angle >> 32)) * 0x1p-31f, &s, &c);
    z.cs[j] = c * r.factor;
    z.sn[j] = s * r.factor;
  }
}

__device__ __forceinline__ void unpack(const uint4& w, float (&x)[8]) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = bf16_lo(u[i]);
    x[2 * i + 1] = bf16_hi(u[i]);
  }
}
__device__ __forceinline__ uint4 pack(const float (&x)[8], float by) {
  return make_uint4(pack_bf16(x[0] * by, x[1] * by), pack_bf16(x[2] * by, x[3] * by), pack_bf16(x[4] * by, x[5] * by),
                    pack_bf16(x[6] * by, x[7] * by));
}

// One row: norm, weights g0 and g1 of the lane's chunks, rotation.
__device__ __forceinline__ void turn_row(uint4& w0, uint4& w1, const TurnArgs& a, bool weigh, const uint4& g0, const uint4& g1,
                                         const Lane& at, const Turn& z) {
  float x[8], y[8];
  unpack(w0, x);
  unpack(w1, y);
  float by = 1.0f;
  if (a.norm) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum = fmaf(x[i], x[i], fmaf(y[i], y[i], sum));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
    by = rsqrtf(sum * (1.0f / kHeadDim) + a.eps);
    if (weigh) {
      float g[8];
      unpack(g0, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= g[i];
      unpack(g1, g);
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= g[i];
    }
  }
  if (at.turns) {
    if (a.rope.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float u = x[2 * i], v = y[2 * i];
        x[2 * i] = fmaf(u, z.cs[i], -(x[2 * i + 1] * z.sn[i]));
        x[2 * i + 1] = fmaf(u, z.sn[i], x[2 * i + 1] * z.cs[i]);
        y[2 * i] = fmaf(v, z.cs[4 + i], -(y[2 * i + 1] * z.sn[4 + i]));
        y[2 * i + 1] = fmaf(v, z.sn[4 + i], y[2 * i + 1] * z.cs[4 + i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float u = x[i];
        x[i] = fmaf(u, z.cs[i], -(y[i] * z.sn[i]));
        y[i] = fmaf(u, z.sn[i], y[i] * z.cs[i]);
      }
    }
  }
  if (!a.norm && !at.turns) return;          // as they are, a NaN's bits too
  w0 = pack(x, by);
  w1 = pack(y, by);
}

// kBits 0: q and k to bf16; 8 or 4: q to bf16, k and v into a cache of so many.
template <int kBits>
__global__ void __launch_bounds__(kWarps * 32) turn_kernel(const TurnArgs a, uint32_t items, int parts, int heads_per_part) {
  const uint32_t item = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= items) return;                 // warp-uniform
  const uint32_t group = item / static_cast<uint32_t>(parts);
  const int part = static_cast<int>(item - group * parts);
  const int lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(group) * kTokens + (lane >> 3);
  const bool live = t < static_cast<int64_t>(a.B) * a.S;
  const int b = live ? static_cast<int>(static_cast<uint32_t>(t) / static_cast<uint32_t>(a.S)) : 0;
  const int s = live ? static_cast<int>(t - static_cast<int64_t>(b) * a.S) : 0;
  const Lane at(lane, a.rope.rot);

  const int end = min((part + 1) * heads_per_part, a.Hq + a.Hk * (kBits == 0 ? 1 : 2));
  int64_t row0 = -1;                         // of head 0
  int64_t head_rows = 0;
  if constexpr (kBits != 0) {
    if (live && end > a.Hq) {
      const int slot = __ldg(a.slots + t), page = slot >> a.cache.page_shift;
      head_rows = 1ll << a.cache.page_shift;
      if (slot >= 0 && page < a.cache.num_pages)
        row0 = ((static_cast<int64_t>(page) * a.cache.H) << a.cache.page_shift) + (slot & ((1 << a.cache.page_shift) - 1));
      else if (slot >= 0 && at.l == 0)
        atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
    }
  }
  Turn z;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    z.cs[j] = 1.0f;
    z.sn[j] = 0.0f;
  }
  bool turned = false;

  // Heads [h0, h1) of one of q, k and v.
  auto run = [&](const uint16_t* src, int h0, int h1, const uint16_t* weight, auto which, auto&& put) {
    constexpr bool kTurn = decltype(which)::value;
    if (h0 >= h1) return;
    uint4 g0 = make_uint4(0u, 0u, 0u, 0u), g1 = g0;
    if (kTurn && weight != nullptr) {
      g0 = __ldg(reinterpret_cast<const uint4*>(weight) + at.c0);
      g1 = __ldg(reinterpret_cast<const uint4*>(weight) + at.c1);
    }
    for (int h = h0; h < h1; h += kAhead) {
      uint4 w[kAhead][2];
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
        if (live && h + i < h1) {
          const uint4* row = reinterpret_cast<const uint4*>(src + (h + i) * kHeadDim);
          w[i][0] = __ldcs(row + at.c0);
          w[i][1] = __ldcs(row + at.c1);
        }
      }
      if (kTurn && !turned && at.turns && live) turn_of(a.rope, a.positions + b * a.p_sb + s * a.p_ss, at, z);
      if (kTurn) turned = true;
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        if (h + i >= h1) break;
        if constexpr (kTurn) turn_row(w[i][0], w[i][1], a, weight != nullptr, g0, g1, at, z);
        put(h + i, w[i][0], w[i][1]);
      }
    }
  };
  auto to_bf16 = [&](uint16_t* out, int H) {
    return [=](int h, const uint4& w0, const uint4& w1) {
      if (!live) return;
      uint4* row = reinterpret_cast<uint4*>(out + (t * H + h) * kHeadDim);
      row[at.c0] = w0;
      row[at.c1] = w1;
    };
  };
  const int first = part * heads_per_part;
  if (first < a.Hq) run(a.q + b * a.q_sb + s * a.q_ss, first, min(end, a.Hq), a.q_weight, std::true_type(), to_bf16(a.q_out, a.Hq));
  const uint16_t* k = a.k + b * a.k_sb + s * a.k_ss;
  const int k0 = max(first - a.Hq, 0), k1 = min(end - a.Hq, a.Hk);
  if constexpr (kBits == 0) {
    run(k, k0, k1, a.k_weight, std::true_type(), to_bf16(a.k_out, a.Hk));
  } else {
    run(k, k0, k1, a.k_weight, std::true_type(), [&](int h, const uint4& w0, const uint4& w1) {
      put_row<kBits, false>(a.cache, w0, w1, row0 < 0 ? -1 : row0 + h * head_rows, at.l, at.c0, at.c1);
    });
    run(a.v + b * a.v_sb + s * a.v_ss, max(first - a.Hq - a.Hk, 0), min(end - a.Hq - a.Hk, a.Hk), nullptr, std::false_type(),
        [&](int h, const uint4& w0, const uint4& w1) {
          put_row<kBits, true>(a.cache, w0, w1, row0 < 0 ? -1 : row0 + h * head_rows, at.l, at.c0, at.c1);
        });
  }
}

}  // namespace

cudaError_t launch_turn(const TurnArgs& a, cudaStream_t stream) {
  const int bits = a.slots == nullptr ? 0 : a.cache.bits;
  const int heads = a.Hq + a.Hk * (bits == 0 ? 1 : 2);
  const int64_t groups = (static_cast<int64_t>(a.B) * a.S + kTokens - 1) / kTokens;
  // As few sines as the heads allow, but warps for every SM.
  int per = std::min(heads, kMaxHeads);
  while (per > 1 && groups * ((heads + per - 1) / per) < 152 * 16) per = (per + 1) / 2;
  const int parts = (heads + per - 1) / per;
  const uint32_t items = static_cast<uint32_t>(groups * parts);
  const unsigned ctas = (items + kWarps - 1) / kWarps;
  auto kernel = bits == 0 ? turn_kernel<0> : bits == 8 ? turn_kernel<8> : turn_kernel<4>;
  kernel<<<ctas, kWarps * 32, 0, stream>>>(a, items, parts, per);
  return cudaGetLastError();
}

}  // namespace sage
