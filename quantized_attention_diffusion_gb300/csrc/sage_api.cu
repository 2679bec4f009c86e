// sage_api.cu -- the extern "C" boundary: argument checks, workspace layout,
// stream-ordered scratch, launch sequences and error mapping.  Declarations
// and their contracts are in include/sage.h.
#include <algorithm>
#include <atomic>
#include <cinttypes>
#include <climits>
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <new>
#include <string>

#include "sage.h"
#include "sage_internal.cuh"

using namespace sage;

namespace {

thread_local std::string t_last_error;
thread_local cudaEvent_t t_attn_before = nullptr, t_attn_after = nullptr;
std::atomic<uint64_t> g_timeout_ns{2000000000ull};
constexpr uint64_t kDefaultTimeoutNs = 2000000000ull;

sage_status fail(sage_status s, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_last_error = buf;
  return s;
}

sage_status cuda_fail(cudaError_t e, const char* what) {
  return fail(SAGE_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

sage_status check_shape(int B, int S, int H, int D) {
  if (D != kHeadDim)
    return fail(SAGE_ERR_UNSUPPORTED, "head dimension %d is not supported: this kernel takes D = 128", D);
  if (B < 1 || S < 1 || H < 1) return fail(SAGE_ERR_INVALID_ARG, "B, S and H must be >= 1 (got %d, %d, %d)", B, S, H);
  if (static_cast<int64_t>(B) * H > INT_MAX) return fail(SAGE_ERR_INVALID_ARG, "B*H exceeds 2^31-1");
  if (S > (1 << 28)) return fail(SAGE_ERR_INVALID_ARG, "S = %d exceeds 2^28", S);
  return SAGE_OK;
}

sage_status check_scale(float softmax_scale) {
  if (!std::isfinite(softmax_scale) || !(softmax_scale > 0.0f))
    return fail(SAGE_ERR_INVALID_ARG, "softmax_scale must be finite and > 0 (got %g)", softmax_scale);
  return SAGE_OK;
}

sage_status check_ptrs(std::initializer_list<std::pair<const void*, const char*>> ptrs) {
  for (auto& pr : ptrs) {
    if (!pr.first) return fail(SAGE_ERR_INVALID_ARG, "%s is NULL", pr.second);
    if (!aligned(pr.first, 16)) return fail(SAGE_ERR_MISALIGNED, "%s is not 16-byte aligned", pr.second);
  }
  return SAGE_OK;
}

// The attention kernel writes each output row as 32-byte vectors.
sage_status check_out(const void* out) {
  if (!aligned(out, 32)) return fail(SAGE_ERR_MISALIGNED, "out is not 32-byte aligned");
  return SAGE_OK;
}

// Workspace layout (all offsets 256-byte aligned).
struct WsLayout {
  size_t q16, k16, vt, qs, ks, vs, vamax, ksum, kmean, total;
};

size_t align256(size_t x) { return (x + 255) & ~static_cast<size_t>(255); }

// Sq query rows, Sk key/value rows (equal for self-attention).
WsLayout ws_layout(int B, int Sq, int Sk, int H) {
  const size_t BH = static_cast<size_t>(B) * H;
  const size_t Sqp = padded_len(Sq), Skp = padded_len(Sk), nbq = num_blocks(Sq), nbk = num_blocks(Sk);
  WsLayout w;
  size_t off = 0;
  w.q16 = off; off += align256(BH * Sqp * kHeadDim * sizeof(__half));
  w.k16 = off; off += align256(BH * Skp * kHeadDim * sizeof(__half));
  w.vt = off; off += align256(BH * kHeadDim * Skp);
  w.qs = off; off += align256(BH * nbq * sizeof(float));
  w.ks = off; off += align256(BH * nbk * sizeof(float));
  w.vs = off; off += align256(BH * kHeadDim * sizeof(float));
  w.vamax = off; off += align256(BH * kHeadDim * sizeof(uint32_t));
  w.ksum = off; off += align256(BH * kHeadDim * sizeof(unsigned long long));
  w.kmean = off; off += align256(BH * kHeadDim * sizeof(float));
  w.total = off;
  return w;
}

template <typename T>
T* at(void* base, size_t off) {
  return reinterpret_cast<T*>(static_cast<uint8_t*>(base) + off);
}

// Host-only fault injection (a test hook, off by default): when armed for a
// site, the site's skip-th next event reports a failure without doing the
// work (no allocation, no launch), and the hook disarms.  Nothing faults on
// the device.
std::atomic<int> g_fault_site{0};
std::atomic<int> g_fault_skip{0};

bool fault_fires(int site) {
  if (g_fault_site.load(std::memory_order_relaxed) != site) return false;
  if (g_fault_skip.fetch_sub(1, std::memory_order_relaxed) > 0) return false;
  g_fault_site.store(0, std::memory_order_relaxed);
  return true;
}

// One private stream-ordered pool per device; memory is kept by the pool
// (release threshold = max) so steady-state calls do not go to the driver.
// A pool is published in g_pools only once its release threshold is set.
constexpr int kMaxDevices = 64;
std::mutex g_pool_mu;
cudaMemPool_t g_pools[kMaxDevices] = {};

sage_status current_device(int* dev) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (*dev < 0 || *dev >= kMaxDevices)
    return fail(SAGE_ERR_CUDA, "device index %d exceeds this library's %d-device table", *dev, kMaxDevices);
  return SAGE_OK;
}

// `bytes` of stream-ordered scratch for `what` on the current device.
sage_status pool_alloc(void** ptr, size_t bytes, cudaStream_t stream, const char* what) {
  if (fault_fires(SAGE_FAULT_POOL_ALLOC))
    return fail(SAGE_ERR_NO_MEMORY, "%s allocation of %zu bytes failed: injected fault", what, bytes);
  int dev = 0;
  sage_status s = current_device(&dev);
  if (s != SAGE_OK) return s;
  cudaMemPool_t pool;
  {
    std::lock_guard<std::mutex> lk(g_pool_mu);
    if (!g_pools[dev]) {
      cudaMemPoolProps props;
      std::memset(&props, 0, sizeof props);
      props.allocType = cudaMemAllocationTypePinned;
      props.location.type = cudaMemLocationTypeDevice;
      props.location.id = dev;
      cudaMemPool_t fresh = nullptr;
      // The first call may be one that is being captured: making a pool records
      // nothing, and is let through in the relaxed mode only.
      cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
      cudaError_t e = cudaThreadExchangeStreamCaptureMode(&mode);
      if (e != cudaSuccess) return cuda_fail(e, "stream capture mode");
      uint64_t thr = UINT64_MAX;
      const char* step = "memory pool creation";
      e = cudaMemPoolCreate(&fresh, &props);
      if (e == cudaSuccess) {
        step = "memory pool release threshold";
        e = cudaMemPoolSetAttribute(fresh, cudaMemPoolAttrReleaseThreshold, &thr);
        if (e != cudaSuccess) (void)cudaMemPoolDestroy(fresh);
      }
      (void)cudaThreadExchangeStreamCaptureMode(&mode);
      if (e != cudaSuccess) return cuda_fail(e, step);
      g_pools[dev] = fresh;
    }
    pool = g_pools[dev];
  }
  cudaError_t e = cudaMallocFromPoolAsync(ptr, bytes, pool, stream);
  if (e != cudaSuccess) {
    // An out-of-memory result is not sticky, but the runtime keeps it as the
    // thread's last error: clear it so that it is not reported by a later
    // call's launch check.
    (void)cudaGetLastError();
    return fail(SAGE_ERR_NO_MEMORY, "%s allocation of %zu bytes failed: %s", what, bytes, cudaGetErrorString(e));
  }
  return SAGE_OK;
}

// Allocate `bytes` of workspace from the pool, run `body(ws)`, release the
// workspace in stream order whatever body returned.
template <typename Body>
sage_status with_pool_workspace(size_t bytes, cudaStream_t st, Body body) {
  void* ws = nullptr;
  sage_status s = pool_alloc(&ws, bytes, st, "workspace");
  if (s != SAGE_OK) return s;
  s = body(ws);
  cudaError_t e = cudaFreeAsync(ws, st);
  if (s != SAGE_OK) return s;
  if (e != cudaSuccess) return cuda_fail(e, "workspace release");
  return SAGE_OK;
}

uint64_t timeout_ns() { return g_timeout_ns.load(std::memory_order_relaxed); }

// Arguments of the Q/K quantisation that feeds the attention kernel: integer
// codes stored as fp16 (the MMA operand type), [B, H, S_pad, 128].  With
// k_only, Q is left to the attention kernel; k_mean selects K smoothing.
QKQuantArgs<__half> staging_args(const void* q, const void* k, int B, int Sq, int Sk, int H, __half* q16,
                                 float* q_scale, __half* k16, float* k_scale, bool k_only, const float* k_mean) {
  QKQuantArgs<__half> qa;
  qa.q = static_cast<const uint16_t*>(q);
  qa.k = static_cast<const uint16_t*>(k);
  qa.q_codes = q16;
  qa.k_codes = k16;
  qa.q_scale = q_scale;
  qa.k_scale = k_scale;
  qa.BH = B * H;
  qa.H = H;
  qa.set_lengths(Sq, Sk);
  qa.first = k_only ? 1 : 0;
  qa.k_mean = k_mean;
  return qa;
}

// Arguments of the public INT8 quantisation (sage_quantize_qkv and its
// variants): codes [B, H, S_pad, 128].
QKQuantArgs<int8_t> public_args(const void* q, const void* k, int B, int S, int H, int8_t* q_i8, float* q_scale,
                                int8_t* k_i8, float* k_scale, const float* k_mean) {
  QKQuantArgs<int8_t> qa;
  qa.q = static_cast<const uint16_t*>(q);
  qa.k = static_cast<const uint16_t*>(k);
  qa.q_codes = q_i8;
  qa.k_codes = k_i8;
  qa.q_scale = q_scale;
  qa.k_scale = k_scale;
  qa.BH = B * H;
  qa.H = H;
  qa.set_lengths(S, S);
  qa.k_mean = k_mean;
  return qa;
}

// Quantise Q, K and V, then attend.  With fuse_q, only K and V are quantised
// here and the attention kernel quantises Q itself (q_dump / q_scale_dump
// then receive its codes and scales, if given).
sage_status run_fused(const void* q, const void* k, const void* v, void* out, int B, int Sq, int Sk,
                      int H, float softmax_scale, void* ws, cudaStream_t st, float* lse = nullptr,
                      bool fuse_q = false, int8_t* q_dump = nullptr, float* q_scale_dump = nullptr,
                      bool smooth_k = false) {
  const WsLayout w = ws_layout(B, Sq, Sk, H);
  if (smooth_k) {
    cudaError_t e0 = launch_k_channel_means(static_cast<const uint16_t*>(k), B, Sk, H, at<unsigned long long>(ws, w.ksum),
                                            at<float>(ws, w.kmean), st);
    if (e0 != cudaSuccess) return cuda_fail(e0, "K channel means launch");
  }
  const QKQuantArgs<__half> qa = staging_args(q, k, B, Sq, Sk, H, at<__half>(ws, w.q16), at<float>(ws, w.qs),
                                              at<__half>(ws, w.k16), at<float>(ws, w.ks), fuse_q,
                                              smooth_k ? at<float>(ws, w.kmean) : nullptr);
  if (fault_fires(SAGE_FAULT_QUANT_LAUNCH)) return fail(SAGE_ERR_CUDA, "quantisation launch: injected fault");
  cudaError_t e = launch_qkv_quantize<__half>(qa, static_cast<const uint16_t*>(v), at<uint32_t>(ws, w.vamax),
                                              at<uint8_t>(ws, w.vt), at<float>(ws, w.vs), st);
  if (e != cudaSuccess) return cuda_fail(e, "quantisation launch");
  AttnArgs aa;
  aa.q_bf16 = fuse_q ? static_cast<const uint16_t*>(q) : nullptr;
  aa.q_dump = q_dump;
  aa.q_scale_dump = q_scale_dump;
  aa.q_codes = fuse_q ? nullptr : qa.q_codes;
  aa.k_codes = qa.k_codes;
  aa.vt = at<uint8_t>(ws, w.vt);
  aa.q_scale = fuse_q ? nullptr : qa.q_scale;
  aa.k_scale = qa.k_scale;
  aa.v_scale = at<float>(ws, w.vs);
  aa.out = static_cast<uint16_t*>(out);
  aa.s_dump = nullptr;
  aa.lse = lse;
  aa.B = B;
  aa.Sq = Sq;
  aa.Skv = Sk;
  aa.H = H;
  aa.Sq_pad = padded_len(Sq);
  aa.Skv_pad = padded_len(Sk);
  aa.nbq = num_blocks(Sq);
  aa.nbk = num_blocks(Sk);
  aa.softmax_scale = softmax_scale;
  aa.timeout_ns = timeout_ns();
  if (t_attn_before && (e = cudaEventRecord(t_attn_before, st)) != cudaSuccess)
    return cuda_fail(e, "timing event record");
  if (fault_fires(SAGE_FAULT_ATTN_LAUNCH)) return fail(SAGE_ERR_CUDA, "attention launch: injected fault");
  e = launch_attention(aa, st);
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  if (t_attn_after && (e = cudaEventRecord(t_attn_after, st)) != cudaSuccess)
    return cuda_fail(e, "timing event record");
  return SAGE_OK;
}

sage_status run_quantized(const int8_t* q_i8, const float* q_scale, const int8_t* k_i8,
                          const float* k_scale, const uint8_t* vt, const float* v_scale, void* out,
                          int32_t* s_dump, int B, int S, int H, float softmax_scale, void* ws,
                          cudaStream_t st) {
  const WsLayout w = ws_layout(B, S, S, H);
  const int Sp = padded_len(S);
  const size_t n = static_cast<size_t>(B) * H * Sp * kHeadDim;
  cudaError_t e = launch_widen_codes(q_i8, at<__half>(ws, w.q16), n, st);
  if (e == cudaSuccess) e = launch_widen_codes(k_i8, at<__half>(ws, w.k16), n, st);
  if (e != cudaSuccess) return cuda_fail(e, "code widening launch");
  AttnArgs aa;
  aa.q_bf16 = nullptr;
  aa.q_dump = nullptr;
  aa.q_scale_dump = nullptr;
  aa.q_codes = at<__half>(ws, w.q16);
  aa.k_codes = at<__half>(ws, w.k16);
  aa.vt = vt;
  aa.q_scale = q_scale;
  aa.k_scale = k_scale;
  aa.v_scale = v_scale;
  aa.out = static_cast<uint16_t*>(out);
  aa.s_dump = s_dump;
  aa.lse = nullptr;
  aa.B = B;
  aa.Sq = S;
  aa.Skv = S;
  aa.H = H;
  aa.Sq_pad = Sp;
  aa.Skv_pad = Sp;
  aa.nbq = num_blocks(S);
  aa.nbk = num_blocks(S);
  aa.softmax_scale = softmax_scale;
  aa.timeout_ns = timeout_ns();
  e = launch_attention(aa, st);
  if (e != cudaSuccess) return cuda_fail(e, "attention launch");
  return SAGE_OK;
}

sage_status check_workspace(void* ws, size_t bytes, int B, int S, int H) {
  const size_t need = ws_layout(B, S, S, H).total;
  if (!ws) return fail(SAGE_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(ws, 256)) return fail(SAGE_ERR_MISALIGNED, "workspace is not 256-byte aligned");
  if (bytes < need)
    return fail(SAGE_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", bytes, need);
  return SAGE_OK;
}

// A cache of 8 or of 4 bits as the kernels take it, page_shift still to be found.
CacheView cache_view(const sage_kv_cache& c) {
  CacheView v = {};
  v.k_codes = reinterpret_cast<uint8_t*>(c.k_codes);
  v.k_scale = c.k_scale;
  v.v_codes = c.v_codes;
  v.v_scale = c.v_scale;
  v.num_pages = c.num_pages;
  v.H = c.H;
  v.bits = 8;
  return v;
}

CacheView cache_view(const sage_kv4_cache& c) {
  CacheView v = {};
  v.k_codes = c.k_codes;
  v.k_block = c.k_block;
  v.k_scale = c.k_scale;
  v.v_codes = c.v_codes;
  v.v_block = c.v_block;
  v.v_scale = c.v_scale;
  v.num_pages = c.num_pages;
  v.H = c.H;
  v.bits = 4;
  return v;
}

sage_status check_page_size(int page_size, int* shift) {
  if (page_size < 16 || page_size > 256 || (page_size & (page_size - 1)))
    return fail(SAGE_ERR_UNSUPPORTED, "page_size %d is not supported: 16, 32, 64, 128 or 256", page_size);
  *shift = 0;
  while ((1 << *shift) < page_size) ++*shift;
  return SAGE_OK;
}

sage_status check_table(const int32_t* table, int width, int64_t stride) {
  if (!table) return fail(SAGE_ERR_INVALID_ARG, "block_table is NULL");
  if (!aligned(table, 4)) return fail(SAGE_ERR_MISALIGNED, "block_table is not 4-byte aligned");
  if (width < 1 || stride < 0)
    return fail(SAGE_ERR_INVALID_ARG, "table_width must be >= 1 and table_stride >= 0 (got %d, %lld)", width,
                static_cast<long long>(stride));
  return SAGE_OK;
}

template <typename Cache>
sage_status check_cache(const Cache* c, int D, CacheView* view) {
  if (!c) return fail(SAGE_ERR_INVALID_ARG, "cache is NULL");
  if (D != kHeadDim)
    return fail(SAGE_ERR_UNSUPPORTED, "head dimension %d is not supported: this kernel takes D = 128", D);
  if (c->num_pages < 1 || c->H < 1)
    return fail(SAGE_ERR_INVALID_ARG, "a cache's num_pages and H must be >= 1 (got %d, %d)", c->num_pages, c->H);
  *view = cache_view(*c);
  sage_status s = check_page_size(c->page_size, &view->page_shift);
  if (s != SAGE_OK) return s;
  if (static_cast<int64_t>(c->num_pages) * c->H > INT_MAX / c->page_size)
    return fail(SAGE_ERR_INVALID_ARG, "num_pages * H * page_size exceeds 2^31-1");
  s = check_ptrs({{c->k_codes, "k_codes"}, {c->k_scale, "k_scale"}, {c->v_codes, "v_codes"}, {c->v_scale, "v_scale"}});
  if (s == SAGE_OK && view->bits == 4) s = check_ptrs({{view->k_block, "k_block"}, {view->v_block, "v_block"}});
  return s;
}

// A cache and its page table, as the cache entry points take them.
template <typename Cache>
sage_status check_cache(const Cache* c, int D, const int32_t* table, int width, int64_t stride, CacheView* view) {
  const sage_status s = check_cache(c, D, view);
  return s == SAGE_OK ? check_table(table, width, stride) : s;
}

// Device arrays of one int32 per sequence.
sage_status check_ints(const int32_t* p, const char* name) {
  if (!p) return fail(SAGE_ERR_INVALID_ARG, "%s is NULL", name);
  if (!aligned(p, 4)) return fail(SAGE_ERR_MISALIGNED, "%s is not 4-byte aligned", name);
  return SAGE_OK;
}

sage_status check_strides(int64_t sb, int64_t ss, const char* name) {
  if (sb < 0 || ss < 0) return fail(SAGE_ERR_INVALID_ARG, "%s has a negative stride", name);
  if ((sb | ss) % 8 != 0) return fail(SAGE_ERR_MISALIGNED, "%s's strides are not multiples of 8 elements", name);
  return SAGE_OK;
}

// sage_attn_fwd_cache and, with a prefix, sage_attn_fwd_cache_prefix, and their 4-bit forms.
template <typename Cache>
sage_status run_cache_attention(const void* q, int64_t q_sb, int64_t q_ss, const Cache* cache, const int32_t* prefix_table,
                                int prefix_len, const int32_t* table, int width, int64_t stride, const int32_t* lens, void* out, float* lse, int B, int Sq, int Hq,
                                int D, float softmax_scale, int causal, void* ws, size_t ws_bytes, void* stream) {
  CacheAttnArgs a;
  sage_status s = check_cache(cache, D, table, width, stride, &a.cache);
  if (s == SAGE_OK) s = check_shape(B, Sq, Hq, D);
  if (s == SAGE_OK && Hq % cache->H != 0)
    s = fail(SAGE_ERR_INVALID_ARG, "Hq = %d is not a multiple of the cache's H = %d", Hq, cache->H);
  if (s == SAGE_OK && static_cast<int64_t>(B) * Hq > INT_MAX / Sq)
    s = fail(SAGE_ERR_INVALID_ARG, "B*Sq*Hq exceeds 2^31-1");
  if (s == SAGE_OK && !cache_attn_fits(B, Sq, Hq, cache->H, cache->page_size, width, prefix_len))
    s = fail(SAGE_ERR_INVALID_ARG, "B = %d, Sq = %d, Hq = %d over tables of %d pages is too much for one call", B, Sq, Hq, width);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {out, "out"}});
  if (s == SAGE_OK) s = check_strides(q_sb, q_ss, "q");
  if (s == SAGE_OK) s = check_out(out);
  if (s == SAGE_OK && lse) s = check_ptrs({{lse, "lse"}});
  if (s == SAGE_OK) s = check_ints(lens, "lens");
  if (s != SAGE_OK) return s;
  const size_t need = cache_attn_workspace_bytes(B, Sq, Hq, cache->H, prefix_len);
  if (ws) {
    if (!aligned(ws, 256)) return fail(SAGE_ERR_MISALIGNED, "workspace is not 256-byte aligned");
    if (ws_bytes < need)
      return fail(SAGE_ERR_WORKSPACE, "workspace of %zu bytes is smaller than the %zu bytes needed", ws_bytes, need);
  }
  a.table = {table, width, stride};
  a.lens = lens;
  a.prefix_pages = prefix_table;
  a.prefix_len = prefix_len;
  a.q = static_cast<const uint16_t*>(q);
  a.q_sb = q_sb;
  a.q_ss = q_ss;
  a.out = static_cast<uint16_t*>(out);
  a.lse = lse;
  a.B = B;
  a.Sq = Sq;
  a.Hq = Hq;
  a.causal = causal != 0;
  a.softmax_scale = softmax_scale;
  a.timeout_ns = timeout_ns();
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "device error word");
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  auto launch = [&](void* w) {
    a.workspace = w;
    if (fault_fires(SAGE_FAULT_ATTN_LAUNCH)) return fail(SAGE_ERR_CUDA, "cache attention launch: injected fault");
    const cudaError_t err = launch_cache_attention(a, st);
    return err == cudaSuccess ? SAGE_OK : cuda_fail(err, "cache attention launch");
  };
  return ws || !cache_attn_needs_workspace(a) ? launch(ws) : with_pool_workspace(need, st, launch);
}

template <typename Cache>
sage_status run_prefix_attention(const void* q, int64_t q_sb, int64_t q_ss, const Cache* cache, const int32_t* prefix_table,
                                 int prefix_len, const int32_t* table, int width, int64_t stride, const int32_t* lens,
                                 void* out, float* lse, int B, int Sq, int Hq, int D, float softmax_scale, int causal,
                                 void* ws, size_t ws_bytes, void* stream) {
  const sage_status s = check_ints(prefix_table, "prefix_table");
  if (s != SAGE_OK) return s;
  if (prefix_len < 1 || prefix_len > kMaxCacheLen)
    return fail(SAGE_ERR_INVALID_ARG, "prefix_len must be in [1, 2^30] (got %d)", prefix_len);
  return run_cache_attention(q, q_sb, q_ss, cache, prefix_table, prefix_len, table, width, stride, lens, out, lse, B, Sq, Hq,
                             D, softmax_scale, causal, ws, ws_bytes, stream);
}

template <typename Cache>
sage_status run_cache_write(const Cache* cache, const void* k, const void* v, int64_t k_stride_b, int64_t k_stride_s,
                            int64_t v_stride_b, int64_t v_stride_s, int B, int S, int D,
                            const int32_t* block_table, int table_width, int64_t table_stride,
                            const int32_t* start, const int32_t* count, void* stream) {
  CacheWriteArgs a;
  sage_status s = check_cache(cache, D, block_table, table_width, table_stride, &a.cache);
  if (s == SAGE_OK) s = check_shape(B, S, cache->H, D);
  if (s == SAGE_OK && static_cast<int64_t>(B) * cache->H > INT_MAX / S)
    s = fail(SAGE_ERR_INVALID_ARG, "B*S*H exceeds 2^31-1");
  if (s == SAGE_OK) s = check_ptrs({{k, "k"}, {v, "v"}});
  if (s == SAGE_OK) s = check_strides(k_stride_b, k_stride_s, "k");
  if (s == SAGE_OK) s = check_strides(v_stride_b, v_stride_s, "v");
  if (s == SAGE_OK) s = check_ints(start, "start");
  if (s == SAGE_OK && count) s = check_ints(count, "count");
  if (s != SAGE_OK) return s;
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.k_sb = k_stride_b;
  a.k_ss = k_stride_s;
  a.v_sb = v_stride_b;
  a.v_ss = v_stride_s;
  a.B = B;
  a.S = S;
  a.table = {block_table, table_width, table_stride};
  a.start = start;
  a.count = count;
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "device error word");
  if (fault_fires(SAGE_FAULT_QUANT_LAUNCH)) return fail(SAGE_ERR_CUDA, "cache write launch: injected fault");
  e = launch_kv_cache_write(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache write launch");
  return SAGE_OK;
}

template <typename Cache>
sage_status run_cache_read(const Cache* cache, const int32_t* block_table, int table_width, int64_t table_stride,
                           const int32_t* lens, void* k, void* v, int B, int S, int D, void* stream) {
  CacheReadArgs a;
  sage_status s = check_cache(cache, D, block_table, table_width, table_stride, &a.cache);
  if (s == SAGE_OK) s = check_shape(B, S, cache->H, D);
  if (s == SAGE_OK && static_cast<int64_t>(B) * cache->H > INT_MAX / S)
    s = fail(SAGE_ERR_INVALID_ARG, "B*S*H exceeds 2^31-1");
  if (s == SAGE_OK) s = check_ptrs({{k, "k"}, {v, "v"}});
  if (s == SAGE_OK && !(aligned(k, 32) && aligned(v, 32)))
    s = fail(SAGE_ERR_MISALIGNED, "k or v is not 32-byte aligned");
  if (s == SAGE_OK) s = check_ints(lens, "lens");
  if (s != SAGE_OK) return s;
  a.table = {block_table, table_width, table_stride};
  a.lens = lens;
  a.k = static_cast<uint16_t*>(k);
  a.v = static_cast<uint16_t*>(v);
  a.B = B;
  a.S = S;
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "device error word");
  if (fault_fires(SAGE_FAULT_QUANT_LAUNCH)) return fail(SAGE_ERR_CUDA, "cache read launch: injected fault");
  e = launch_kv_cache_read(a, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cache read launch");
  return SAGE_OK;
}

// F = f / (2 pi) in 2^-64, to the nearest: 1 / (2 pi) in two doubles and the product's
// rounding error, for |f| <= 3.
uint64_t revolutions(double f) {
  constexpr double kHi = 0x1.45f306dc9c883p-3, kLo = -0x1.6b01ec5417056p-57;   // 1 / (2 pi)
  const double p = f * kHi, e = std::fma(f, kHi, -p) + f * kLo;
  const double whole = std::ldexp(p, 32), up = std::floor(whole);      // upper 32 bits
  const double rest = std::ldexp(whole - up, 32) + std::ldexp(e, 64);  // below 2^32 and a rounding
  return (static_cast<uint64_t>(static_cast<int64_t>(up)) << 32) + static_cast<uint64_t>(std::llrint(rest));
}

// The elements from the first to the last of a [B, S, H, 128] tensor of 16-bit values.
struct Extent {
  uintptr_t first, end;
  Extent(const void* p, int64_t sb, int64_t ss, int B, int S, int H)
      : first(reinterpret_cast<uintptr_t>(p)),
        end(p && H > 0 ? first + 2 * static_cast<uintptr_t>((B - 1) * sb + (S - 1) * ss + static_cast<int64_t>(H) * kHeadDim) : first) {}
  bool meets(const Extent& x) const { return first < x.end && x.first < end; }
};

// An output takes no input's place but, where that is dense, its own input's: other rows
// might be written before they are read.
sage_status check_place(const char* name, const Extent& out, const Extent& own, bool dense, std::initializer_list<Extent> others) {
  bool bad = out.meets(own) && !(dense && out.first == own.first);
  for (const Extent& x : others) bad = bad || out.meets(x);
  return bad ? fail(SAGE_ERR_INVALID_ARG, "%s overlaps an input or another output", name) : SAGE_OK;
}

bool is_dense(int64_t sb, int64_t ss, int B, int S, int H) {
  const int64_t row = static_cast<int64_t>(H) * kHeadDim;
  return (S == 1 || ss == row) && (B == 1 || sb == S * row);
}

// Norm and rotation as sage_qk_norm_rope and sage_kv_cache_append take them.
sage_status turn_args(TurnArgs* a, const sage_rope* rope, const int32_t* positions, int64_t p_sb, int64_t p_ss,
                      const void* q_weight, const void* k_weight, float eps) {
  if (!(eps >= 0.0f) || std::isinf(eps)) {
    if (eps != -1.0f) return fail(SAGE_ERR_INVALID_ARG, "eps must be finite and >= 0, or -1 for no norm (got %g)", eps);
    if (q_weight || k_weight) return fail(SAGE_ERR_INVALID_ARG, "weights without a norm");
  }
  if (q_weight && !aligned(q_weight, 16)) return fail(SAGE_ERR_MISALIGNED, "q_weight is not 16-byte aligned");
  if (k_weight && !aligned(k_weight, 16)) return fail(SAGE_ERR_MISALIGNED, "k_weight is not 16-byte aligned");
  a->norm = eps >= 0.0f;
  a->eps = eps;
  a->q_weight = static_cast<const uint16_t*>(q_weight);
  a->k_weight = static_cast<const uint16_t*>(k_weight);
  if (!rope) return SAGE_OK;
  if (rope->dim < 32 || rope->dim > kHeadDim || rope->dim % 32 != 0)
    return fail(SAGE_ERR_UNSUPPORTED, "%d rotated channels are not supported: 32, 64, 96 or 128", rope->dim);
  if (rope->axes < 1 || rope->axes > kMaxAxes)
    return fail(SAGE_ERR_UNSUPPORTED, "%d axes are not supported: 1 to %d", rope->axes, kMaxAxes);
  int pairs = 0;
  for (int i = 0; i < rope->axes; ++i) {
    if (rope->sections[i] < 0 || rope->sections[i] > kHeadDim)
      return fail(SAGE_ERR_INVALID_ARG, "section %d has %d pairs", i, rope->sections[i]);
    pairs += rope->sections[i];
    a->rope.ends[i] = pairs;
  }
  for (int i = rope->axes; i < kMaxAxes; ++i) a->rope.ends[i] = pairs;
  if (pairs != rope->dim / 2)
    return fail(SAGE_ERR_INVALID_ARG, "the sections have %d pairs, the rotated channels %d", pairs, rope->dim / 2);
  if (!std::isfinite(rope->factor)) return fail(SAGE_ERR_INVALID_ARG, "factor must be finite (got %g)", rope->factor);
  if (!rope->freq) return fail(SAGE_ERR_INVALID_ARG, "freq is NULL");
  if (!aligned(rope->freq, 8)) return fail(SAGE_ERR_MISALIGNED, "freq is not 8-byte aligned");
  sage_status s = check_ints(positions, "positions");
  if (s != SAGE_OK) return s;
  if (p_sb < 0 || p_ss < 0) return fail(SAGE_ERR_INVALID_ARG, "positions has a negative stride");
  a->rope.freq = rope->freq;
  a->rope.rot = rope->dim;
  a->rope.interleaved = rope->interleaved != 0;
  a->rope.axes = rope->axes;
  a->rope.factor = rope->factor;
  a->positions = positions;
  a->p_sb = p_sb;
  a->p_ss = p_ss;
  return SAGE_OK;
}

template <typename Cache>
sage_status run_cache_append(const Cache* cache, const void* q, const void* k, const void* v, int64_t q_sb, int64_t q_ss,
                             int64_t k_sb, int64_t k_ss, int64_t v_sb, int64_t v_ss, int B, int S, int Hq, int D,
                             const sage_rope* rope, const int32_t* positions, int64_t p_sb, int64_t p_ss,
                             const void* q_weight, const void* k_weight, float eps, const int32_t* slots, void* q_out,
                             void* stream) {
  TurnArgs a = {};
  sage_status s = check_cache(cache, D, &a.cache);
  if (s == SAGE_OK) s = check_shape(B, S, cache->H, D);
  if (s == SAGE_OK && Hq < 0) s = fail(SAGE_ERR_INVALID_ARG, "Hq must be >= 0 (got %d)", Hq);
  if (s == SAGE_OK && (static_cast<int64_t>(Hq) + 2ll * cache->H) * B > INT_MAX / S)
    s = fail(SAGE_ERR_INVALID_ARG, "B*S*(Hq+2H) exceeds 2^31-1");
  if (s == SAGE_OK) s = check_ptrs({{k, "k"}, {v, "v"}});
  if (s == SAGE_OK && Hq > 0) s = check_ptrs({{q, "q"}, {q_out, "q_out"}});
  if (s == SAGE_OK && Hq > 0) s = check_strides(q_sb, q_ss, "q");
  if (s == SAGE_OK) s = check_strides(k_sb, k_ss, "k");
  if (s == SAGE_OK) s = check_strides(v_sb, v_ss, "v");
  if (s == SAGE_OK) s = check_ints(slots, "slots");
  if (s == SAGE_OK) s = turn_args(&a, rope, positions, p_sb, p_ss, q_weight, k_weight, eps);
  if (s != SAGE_OK) return s;
  if (Hq > 0) {
    const int64_t q_row = static_cast<int64_t>(Hq) * kHeadDim;
    const Extent qo(q_out, S * q_row, q_row, B, S, Hq), qi(q, q_sb, q_ss, B, S, Hq);
    const Extent ki(k, k_sb, k_ss, B, S, cache->H), vi(v, v_sb, v_ss, B, S, cache->H);
    s = check_place("q_out", qo, qi, is_dense(q_sb, q_ss, B, S, Hq), {ki, vi});
    if (s != SAGE_OK) return s;
  }
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.v = static_cast<const uint16_t*>(v);
  a.q_sb = q_sb;
  a.q_ss = q_ss;
  a.k_sb = k_sb;
  a.k_ss = k_ss;
  a.v_sb = v_sb;
  a.v_ss = v_ss;
  a.B = B;
  a.S = S;
  a.Hq = Hq;
  a.Hk = cache->H;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.slots = slots;
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "device error word");
  if (fault_fires(SAGE_FAULT_QUANT_LAUNCH)) return fail(SAGE_ERR_CUDA, "cache append launch: injected fault");
  e = launch_turn(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SAGE_OK : cuda_fail(e, "cache append launch");
}

sage_status check_pages(int num_pages, int page_size, int B, const int32_t* table, int width, int64_t stride, int* shift,
                        int64_t* room) {
  sage_status s = check_page_size(page_size, shift);
  if (s == SAGE_OK && (num_pages < 1 || num_pages > INT_MAX / page_size))
    s = fail(SAGE_ERR_INVALID_ARG, "num_pages must be >= 1 and num_pages * page_size at most 2^31-1 (got %d)", num_pages);
  if (s == SAGE_OK && (B < 1 || B > (1 << 20))) s = fail(SAGE_ERR_INVALID_ARG, "B must be in [1, 2^20] (got %d)", B);
  if (s == SAGE_OK) s = check_table(table, width, stride);
  if (s == SAGE_OK && B > 1 && stride < width)
    s = fail(SAGE_ERR_INVALID_ARG, "rows of block_table that overlap (stride %lld, width %d)", static_cast<long long>(stride), width);
  *room = std::min<int64_t>(kMaxCacheLen, static_cast<int64_t>(width) << *shift);
  return s;
}

}  // namespace

// The host object behind sage_plan (opaque to callers).
struct sage_plan {
  int device;              // device the graph and workspace belong to
  void* ws;                // cudaMalloc'd workspace the recorded launches use
  cudaGraphExec_t exec;    // the recorded sage_attn_fwd_cross call
};

void sage::set_last_error(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  std::vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_last_error = buf;
}

extern "C" {

int64_t sage_padded_len(int S) { return S < 1 ? 0 : static_cast<int64_t>(padded_len(S)); }

int sage_attn_fwd_launches(int B, int Sq, int Skv, int H, int smooth_k) {
  if (B < 1 || Sq < 1 || Skv < 1 || H < 1) return -1;
  // Zeroing of the V maxima, Q/K quantisation with the V maxima, V encoding,
  // attention; K smoothing adds the channel sums and means.
  return 4 + (smooth_k ? 2 : 0);
}

size_t sage_workspace_bytes(int B, int S, int H, int D) {
  if (D != kHeadDim || B < 1 || S < 1 || H < 1 || static_cast<int64_t>(B) * H > INT_MAX || S > (1 << 28))
    return 0;
  return ws_layout(B, S, S, H).total;
}

sage_status sage_quantize_qkv(const void* q, const void* k, const void* v, int B, int S, int H, int D,
                              int8_t* q_i8, float* q_scale, int8_t* k_i8, float* k_scale,
                              uint8_t* vt_fp8, float* v_scale, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK)
    s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {q_i8, "q_i8"}, {q_scale, "q_scale"}, {k_i8, "k_i8"},
                    {k_scale, "k_scale"}, {vt_fp8, "vt_fp8"}, {v_scale, "v_scale"}});
  if (s != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  void* scratch = nullptr;
  s = pool_alloc(&scratch, static_cast<size_t>(B) * H * kHeadDim * sizeof(uint32_t), st, "V maxima scratch");
  if (s != SAGE_OK) return s;
  const QKQuantArgs<int8_t> qa = public_args(q, k, B, S, H, q_i8, q_scale, k_i8, k_scale, nullptr);
  cudaError_t e = launch_qkv_quantize<int8_t>(qa, static_cast<const uint16_t*>(v), static_cast<uint32_t*>(scratch),
                                              vt_fp8, v_scale, st);
  cudaError_t e2 = cudaFreeAsync(scratch, st);
  if (e != cudaSuccess) return cuda_fail(e, "quantisation launch");
  if (e2 != cudaSuccess) return cuda_fail(e2, "scratch release");
  return SAGE_OK;
}

sage_status sage_quantize_qkv_smooth_k(const void* q, const void* k, const void* v, int B, int S, int H, int D,
                                       int8_t* q_i8, float* q_scale, int8_t* k_i8, float* k_scale, uint8_t* vt_fp8,
                                       float* v_scale, float* k_mean, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK)
    s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {q_i8, "q_i8"}, {q_scale, "q_scale"}, {k_i8, "k_i8"},
                    {k_scale, "k_scale"}, {vt_fp8, "vt_fp8"}, {v_scale, "v_scale"}, {k_mean, "k_mean"}});
  if (s != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t BH = static_cast<size_t>(B) * H;
  const size_t sum_bytes = align256(BH * kHeadDim * sizeof(unsigned long long));
  void* scratch = nullptr;
  s = pool_alloc(&scratch, sum_bytes + BH * kHeadDim * sizeof(uint32_t), st, "K sums and V maxima scratch");
  if (s != SAGE_OK) return s;
  unsigned long long* sums = static_cast<unsigned long long*>(scratch);
  cudaError_t e = launch_k_channel_means(static_cast<const uint16_t*>(k), B, S, H, sums, k_mean, st);
  if (e == cudaSuccess) {
    const QKQuantArgs<int8_t> qa = public_args(q, k, B, S, H, q_i8, q_scale, k_i8, k_scale, k_mean);
    e = launch_qkv_quantize<int8_t>(qa, static_cast<const uint16_t*>(v), at<uint32_t>(scratch, sum_bytes), vt_fp8,
                                    v_scale, st);
  }
  cudaError_t e2 = cudaFreeAsync(scratch, st);
  if (e != cudaSuccess) return cuda_fail(e, "quantisation launch");
  if (e2 != cudaSuccess) return cuda_fail(e2, "scratch release");
  return SAGE_OK;
}

sage_status sage_attn_fwd_smooth_k(const void* q, const void* k, const void* v, void* out, int B, int S, int H,
                                   int D, float softmax_scale, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_pool_workspace(ws_layout(B, S, S, H).total, st, [&](void* ws) {
    return run_fused(q, k, v, out, B, S, S, H, softmax_scale, ws, st, nullptr, false, nullptr, nullptr, true);
  });
}

sage_status sage_attn_fwd_ws(const void* q, const void* k, const void* v, void* out, int B, int S,
                             int H, int D, float softmax_scale, void* workspace,
                             size_t workspace_bytes, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s == SAGE_OK) s = check_workspace(workspace, workspace_bytes, B, S, H);
  if (s != SAGE_OK) return s;
  return run_fused(q, k, v, out, B, S, S, H, softmax_scale, workspace, static_cast<cudaStream_t>(stream));
}

sage_status sage_attn_fwd(const void* q, const void* k, const void* v, void* out, int B, int S, int H,
                          int D, float softmax_scale, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_pool_workspace(ws_layout(B, S, S, H).total, st, [&](void* ws) {
    return run_fused(q, k, v, out, B, S, S, H, softmax_scale, ws, st);
  });
}

sage_status sage_attn_fwd_lse(const void* q, const void* k, const void* v, void* out, float* lse, int B,
                              int S, int H, int D, float softmax_scale, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}, {lse, "lse"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_pool_workspace(ws_layout(B, S, S, H).total, st, [&](void* ws) {
    return run_fused(q, k, v, out, B, S, S, H, softmax_scale, ws, st, lse);
  });
}

sage_status sage_attn_fwd_cross(const void* q, const void* k, const void* v, void* out, float* lse, int B,
                                int Sq, int Skv, int H, int D, float softmax_scale, void* stream) {
  sage_status s = check_shape(B, Sq, H, D);
  if (s == SAGE_OK) s = check_shape(B, Skv, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s == SAGE_OK && lse) s = check_ptrs({{lse, "lse"}});
  if (s != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_pool_workspace(ws_layout(B, Sq, Skv, H).total, st, [&](void* ws) {
    return run_fused(q, k, v, out, B, Sq, Skv, H, softmax_scale, ws, st, lse);
  });
}

sage_status sage_plan_create(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Sq,
                             int Skv, int H, int D, float softmax_scale, sage_plan** plan) {
  return sage_plan_create_ex(q, k, v, out, lse, B, Sq, Skv, H, D, softmax_scale, 0u, plan);
}

sage_status sage_plan_create_ex(const void* q, const void* k, const void* v, void* out, float* lse, int B, int Sq,
                                int Skv, int H, int D, float softmax_scale, unsigned flags, sage_plan** plan) {
  if (!plan) return fail(SAGE_ERR_INVALID_ARG, "plan is NULL");
  *plan = nullptr;
  if ((flags & ~(SAGE_PLAN_SMOOTH_K | SAGE_PLAN_FUSED_Q)) != 0u ||
      flags == (SAGE_PLAN_SMOOTH_K | SAGE_PLAN_FUSED_Q))
    return fail(SAGE_ERR_UNSUPPORTED, "plan flags 0x%x: no call offers that combination", flags);
  const bool smooth_k = (flags & SAGE_PLAN_SMOOTH_K) != 0u, fuse_q = (flags & SAGE_PLAN_FUSED_Q) != 0u;
  if (flags != 0u && (Sq != Skv || lse != nullptr))
    return fail(SAGE_ERR_INVALID_ARG, "plan flags 0x%x record a self-attention call without LSE (Sq %d, Skv %d%s)",
                flags, Sq, Skv, lse ? ", lse given" : "");
  sage_status s = check_shape(B, Sq, H, D);
  if (s == SAGE_OK) s = check_shape(B, Skv, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s == SAGE_OK && lse) s = check_ptrs({{lse, "lse"}});
  int dev = 0;
  if (s == SAGE_OK) s = current_device(&dev);
  if (s != SAGE_OK) return s;

  const size_t bytes = ws_layout(B, Sq, Skv, H).total;
  void* ws = nullptr;
  cudaError_t e = fault_fires(SAGE_FAULT_POOL_ALLOC) ? cudaErrorMemoryAllocation : cudaMalloc(&ws, bytes);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();
    return fail(SAGE_ERR_NO_MEMORY, "plan workspace allocation of %zu bytes failed: %s", bytes, cudaGetErrorString(e));
  }
  cudaStream_t cs = nullptr;
  cudaGraph_t graph = nullptr;
  cudaGraphExec_t exec = nullptr;
  e = load_quantize_kernels();                       // no module loading inside the capture
  if (e == cudaSuccess) e = load_attention_kernels();
  if (e != cudaSuccess) {
    cudaFree(ws);
    return cuda_fail(e, "plan kernel loading");
  }
  e = cudaStreamCreateWithFlags(&cs, cudaStreamNonBlocking);
  if (e != cudaSuccess) {
    cudaFree(ws);
    return cuda_fail(e, "plan capture stream");
  }
  // Record the launches of the call; the timing hook stays out of the graph.
  const cudaEvent_t before = t_attn_before, after = t_attn_after;
  t_attn_before = t_attn_after = nullptr;
  e = cudaStreamBeginCapture(cs, cudaStreamCaptureModeThreadLocal);
  if (e == cudaSuccess) {
    s = run_fused(q, k, v, out, B, Sq, Skv, H, softmax_scale, ws, cs, lse, fuse_q, nullptr, nullptr, smooth_k);
    const cudaError_t e_end = cudaStreamEndCapture(cs, &graph);   // ends the capture whatever happened
    if (s == SAGE_OK && e_end != cudaSuccess) s = cuda_fail(e_end, "plan capture");
  } else {
    s = cuda_fail(e, "plan capture start");
  }
  t_attn_before = before;
  t_attn_after = after;
  if (s == SAGE_OK) {
    e = cudaGraphInstantiate(&exec, graph, 0);
    if (e != cudaSuccess) s = cuda_fail(e, "plan graph instantiation");
  }
  if (graph) cudaGraphDestroy(graph);
  cudaStreamDestroy(cs);
  sage_plan* p = nullptr;
  if (s == SAGE_OK) {
    p = new (std::nothrow) sage_plan{dev, ws, exec};
    if (!p) s = fail(SAGE_ERR_NO_MEMORY, "plan object allocation failed");
  }
  if (s != SAGE_OK) {
    if (exec) cudaGraphExecDestroy(exec);
    cudaFree(ws);
    (void)cudaGetLastError();   // a failed capture leaves no error for the next call
    return s;
  }
  *plan = p;
  return SAGE_OK;
}

sage_status sage_plan_launch(sage_plan* plan, void* stream) {
  if (!plan) return fail(SAGE_ERR_INVALID_ARG, "plan is NULL");
  int dev = 0;
  sage_status s = current_device(&dev);
  if (s != SAGE_OK) return s;
  if (dev != plan->device)
    return fail(SAGE_ERR_INVALID_ARG, "plan was created on device %d, current device is %d", plan->device, dev);
  if (fault_fires(SAGE_FAULT_ATTN_LAUNCH)) return fail(SAGE_ERR_CUDA, "plan launch: injected fault");
  const cudaError_t e = cudaGraphLaunch(plan->exec, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "plan launch");
  return SAGE_OK;
}

sage_status sage_plan_destroy(sage_plan* plan) {
  if (!plan) return SAGE_OK;
  cudaError_t e = cudaGraphExecDestroy(plan->exec);
  const cudaError_t e2 = cudaFree(plan->ws);
  delete plan;
  if (e == cudaSuccess) e = e2;
  if (e != cudaSuccess) return cuda_fail(e, "plan release");
  return SAGE_OK;
}

sage_status sage_attn_fwd_quantized(const int8_t* q_i8, const float* q_scale, const int8_t* k_i8,
                                    const float* k_scale, const uint8_t* vt_fp8,
                                    const float* v_scale, void* out, int B, int S, int H, int D,
                                    float softmax_scale, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK)
    s = check_ptrs({{q_i8, "q_i8"}, {q_scale, "q_scale"}, {k_i8, "k_i8"}, {k_scale, "k_scale"},
                    {vt_fp8, "vt_fp8"}, {v_scale, "v_scale"}, {out, "out"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s == SAGE_OK) s = check_workspace(workspace, workspace_bytes, B, S, H);
  if (s != SAGE_OK) return s;
  return run_quantized(q_i8, q_scale, k_i8, k_scale, vt_fp8, v_scale, out, nullptr, B, S, H, softmax_scale,
                       workspace, static_cast<cudaStream_t>(stream));
}

sage_status sage_debug_qk_int32(const int8_t* q_i8, const float* q_scale, const int8_t* k_i8,
                                const float* k_scale, const uint8_t* vt_fp8, const float* v_scale,
                                void* out, int32_t* s_out, int B, int S, int H, int D,
                                float softmax_scale, void* workspace, size_t workspace_bytes,
                                void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK)
    s = check_ptrs({{q_i8, "q_i8"}, {q_scale, "q_scale"}, {k_i8, "k_i8"}, {k_scale, "k_scale"},
                    {vt_fp8, "vt_fp8"}, {v_scale, "v_scale"}, {out, "out"}, {s_out, "s_out"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s == SAGE_OK) s = check_workspace(workspace, workspace_bytes, B, S, H);
  if (s != SAGE_OK) return s;
  return run_quantized(q_i8, q_scale, k_i8, k_scale, vt_fp8, v_scale, out, s_out, B, S, H, softmax_scale,
                       workspace, static_cast<cudaStream_t>(stream));
}

sage_status sage_attn_fwd_fused_q(const void* q, const void* k, const void* v, void* out, int B, int S,
                                  int H, int D, float softmax_scale, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_pool_workspace(ws_layout(B, S, S, H).total, st, [&](void* ws) {
    return run_fused(q, k, v, out, B, S, S, H, softmax_scale, ws, st, nullptr, true);
  });
}

sage_status sage_kv_cache_write(const sage_kv_cache* cache, const void* k, const void* v, int64_t k_stride_b,
                                int64_t k_stride_s, int64_t v_stride_b, int64_t v_stride_s, int B, int S, int D,
                                const int32_t* block_table, int table_width, int64_t table_stride,
                                const int32_t* start, const int32_t* count, void* stream) {
  return run_cache_write(cache, k, v, k_stride_b, k_stride_s, v_stride_b, v_stride_s, B, S, D, block_table, table_width,
                         table_stride, start, count, stream);
}

sage_status sage_kv4_cache_write(const sage_kv4_cache* cache, const void* k, const void* v, int64_t k_stride_b,
                                 int64_t k_stride_s, int64_t v_stride_b, int64_t v_stride_s, int B, int S, int D,
                                 const int32_t* block_table, int table_width, int64_t table_stride,
                                 const int32_t* start, const int32_t* count, void* stream) {
  return run_cache_write(cache, k, v, k_stride_b, k_stride_s, v_stride_b, v_stride_s, B, S, D, block_table, table_width,
                         table_stride, start, count, stream);
}

sage_status sage_kv_cache_read(const sage_kv_cache* cache, const int32_t* block_table, int table_width,
                               int64_t table_stride, const int32_t* lens, void* k, void* v, int B, int S, int D,
                               void* stream) {
  return run_cache_read(cache, block_table, table_width, table_stride, lens, k, v, B, S, D, stream);
}

sage_status sage_kv4_cache_read(const sage_kv4_cache* cache, const int32_t* block_table, int table_width,
                                int64_t table_stride, const int32_t* lens, void* k, void* v, int B, int S, int D,
                                void* stream) {
  return run_cache_read(cache, block_table, table_width, table_stride, lens, k, v, B, S, D, stream);
}

sage_status sage_kv_cache_append(const sage_kv_cache* cache, const void* q, const void* k, const void* v, int64_t q_stride_b,
                                 int64_t q_stride_s, int64_t k_stride_b, int64_t k_stride_s, int64_t v_stride_b,
                                 int64_t v_stride_s, int B, int S, int Hq, int D, const sage_rope* rope,
                                 const int32_t* positions, int64_t pos_stride_b, int64_t pos_stride_s, const void* q_weight,
                                 const void* k_weight, float eps, const int32_t* slots, void* q_out, void* stream) {
  return run_cache_append(cache, q, k, v, q_stride_b, q_stride_s, k_stride_b, k_stride_s, v_stride_b, v_stride_s, B, S, Hq,
                          D, rope, positions, pos_stride_b, pos_stride_s, q_weight, k_weight, eps, slots, q_out, stream);
}

sage_status sage_kv4_cache_append(const sage_kv4_cache* cache, const void* q, const void* k, const void* v,
                                  int64_t q_stride_b, int64_t q_stride_s, int64_t k_stride_b, int64_t k_stride_s,
                                  int64_t v_stride_b, int64_t v_stride_s, int B, int S, int Hq, int D,
                                  const sage_rope* rope, const int32_t* positions, int64_t pos_stride_b,
                                  int64_t pos_stride_s, const void* q_weight, const void* k_weight, float eps,
                                  const int32_t* slots, void* q_out, void* stream) {
  return run_cache_append(cache, q, k, v, q_stride_b, q_stride_s, k_stride_b, k_stride_s, v_stride_b, v_stride_s, B, S, Hq,
                          D, rope, positions, pos_stride_b, pos_stride_s, q_weight, k_weight, eps, slots, q_out, stream);
}

sage_status sage_qk_norm_rope(const void* q, const void* k, int64_t q_stride_b, int64_t q_stride_s, int64_t k_stride_b,
                              int64_t k_stride_s, int B, int S, int Hq, int Hk, int D, const sage_rope* rope,
                              const int32_t* positions, int64_t pos_stride_b, int64_t pos_stride_s, const void* q_weight,
                              const void* k_weight, float eps, void* q_out, void* k_out, void* stream) {
  TurnArgs a = {};
  sage_status s = check_shape(B, S, Hq, D);
  if (s == SAGE_OK && Hk < 0) s = fail(SAGE_ERR_INVALID_ARG, "Hk must be >= 0 (got %d)", Hk);
  if (s == SAGE_OK && (static_cast<int64_t>(Hq) + Hk) * B > INT_MAX / S)
    s = fail(SAGE_ERR_INVALID_ARG, "B*S*(Hq+Hk) exceeds 2^31-1");
  if (s == SAGE_OK) s = check_ptrs({{q, "q"}, {q_out, "q_out"}});
  if (s == SAGE_OK) s = check_strides(q_stride_b, q_stride_s, "q");
  if (s == SAGE_OK && Hk > 0) s = check_ptrs({{k, "k"}, {k_out, "k_out"}});
  if (s == SAGE_OK && Hk > 0) s = check_strides(k_stride_b, k_stride_s, "k");
  if (s == SAGE_OK) s = turn_args(&a, rope, positions, pos_stride_b, pos_stride_s, q_weight, k_weight, eps);
  if (s != SAGE_OK) return s;
  const Extent qi(q, q_stride_b, q_stride_s, B, S, Hq), ki(k, k_stride_b, k_stride_s, B, S, Hk);
  const int64_t q_row = static_cast<int64_t>(Hq) * kHeadDim, k_row = static_cast<int64_t>(Hk) * kHeadDim;
  const Extent qo(q_out, S * q_row, q_row, B, S, Hq), ko(k_out, S * k_row, k_row, B, S, Hk);
  s = check_place("q_out", qo, qi, is_dense(q_stride_b, q_stride_s, B, S, Hq), {ki, ko});
  if (s == SAGE_OK && Hk > 0) s = check_place("k_out", ko, ki, is_dense(k_stride_b, k_stride_s, B, S, Hk), {qi});
  if (s != SAGE_OK) return s;
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k);
  a.q_sb = q_stride_b;
  a.q_ss = q_stride_s;
  a.k_sb = k_stride_b;
  a.k_ss = k_stride_s;
  a.B = B;
  a.S = S;
  a.Hq = Hq;
  a.Hk = Hk;
  a.q_out = static_cast<uint16_t*>(q_out);
  a.k_out = static_cast<uint16_t*>(k_out);
  if (fault_fires(SAGE_FAULT_QUANT_LAUNCH)) return fail(SAGE_ERR_CUDA, "norm and rotation launch: injected fault");
  const cudaError_t e = launch_turn(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SAGE_OK : cuda_fail(e, "norm and rotation launch");
}

sage_status sage_rope_frequencies(int dim, double base, int scaling, double factor, double original_len, double low,
                                  double high, uint64_t* freq, double* attention_factor) {
  if (!freq || !attention_factor) return fail(SAGE_ERR_INVALID_ARG, "freq and attention_factor must not be NULL");
  if (dim < 2 || dim > kHeadDim || dim % 2 != 0)
    return fail(SAGE_ERR_INVALID_ARG, "dim must be even and in [2, 128] (got %d)", dim);
  if (!std::isfinite(base) || base <= 1.0) return fail(SAGE_ERR_INVALID_ARG, "base must be finite and > 1 (got %g)", base);
  if (scaling < SAGE_ROPE_PLAIN || scaling > SAGE_ROPE_BANDS)
    return fail(SAGE_ERR_UNSUPPORTED, "scaling %d is not one of SAGE_ROPE_*", scaling);
  if (scaling != SAGE_ROPE_PLAIN && (!std::isfinite(factor) || factor < 1.0))
    return fail(SAGE_ERR_INVALID_ARG, "factor must be finite and >= 1 (got %g)", factor);
  const bool by_len = scaling == SAGE_ROPE_YARN || scaling == SAGE_ROPE_BANDS;
  if (by_len && (!std::isfinite(original_len) || original_len < 1.0 || !std::isfinite(low) || !std::isfinite(high) || low <= 0.0 || high <= low))
    return fail(SAGE_ERR_INVALID_ARG, "original_len must be >= 1 and 0 < low < high (got %g, %g, %g)", original_len, low, high);
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  if (scaling == SAGE_ROPE_NTK && dim > 2) base *= std::pow(factor, dim / (dim - 2.0));
  double lo = 0.0, hi = 0.0;                 // of the ramp over the pairs
  if (scaling == SAGE_ROPE_YARN) {
    lo = std::max(0.0, std::floor(dim * std::log(original_len / (high * kTwoPi)) / (2.0 * std::log(base))));
    hi = std::min(dim - 1.0, std::ceil(dim * std::log(original_len / (low * kTwoPi)) / (2.0 * std::log(base))));
  }
  for (int i = 0; i < dim / 2; ++i) {
    double f = std::pow(base, -2.0 * i / dim);
    if (scaling == SAGE_ROPE_LINEAR) f /= factor;
    if (scaling == SAGE_ROPE_YARN) {
      // hi <= 0: pair 0, which turns most, turns `low` times or less.
      const double ramp = hi <= 0.0 ? 1.0 : std::min(1.0, std::max(0.0, (i - lo) / std::max(1e-3, hi - lo)));
      f = f / factor * ramp + f * (1.0 - ramp);
    }
    if (scaling == SAGE_ROPE_BANDS) {
      const double keep = std::min(1.0, std::max(0.0, (original_len * f / kTwoPi - low) / (high - low)));
      f = f / factor * (1.0 - keep) + f * keep;
    }
    freq[i] = revolutions(f);
  }
  *attention_factor = scaling == SAGE_ROPE_YARN ? 0.1 * std::log(factor) + 1.0 : 1.0;
  return SAGE_OK;
}

uint64_t sage_rope_frequency(double radians) { return std::isfinite(radians) && std::fabs(radians) <= 3.0 ? revolutions(radians) : 0; }

sage_status sage_kv_pages_reserve(const int32_t* free_pages, const int32_t* free_count, int num_pages, int page_size,
                                  const int32_t* lens, const int32_t* counts, int B, int32_t* block_table, int table_width,
                                  int64_t table_stride, int layout, int tokens, int32_t* start, int32_t* taken,
                                  int32_t* new_lens, int32_t* first, int32_t* free_left, int32_t* slots,
                                  int32_t* positions, void* stream) {
  PagesArgs a = {};
  sage_status s = check_pages(num_pages, page_size, B, block_table, table_width, table_stride, &a.page_shift, &a.room);
  if (s == SAGE_OK && (layout < SAGE_TOKENS_PACKED || layout > SAGE_TOKENS_END))
    s = fail(SAGE_ERR_UNSUPPORTED, "layout %d is not one of SAGE_TOKENS_*", layout);
  if (s == SAGE_OK && (tokens < 1 || (layout != SAGE_TOKENS_PACKED && tokens > INT_MAX / B)))
    s = fail(SAGE_ERR_INVALID_ARG, "tokens must be >= 1, B * tokens at most 2^31-1 (got %d)", tokens);
  const std::pair<const int32_t*, const char*> arrays[] = {
      {free_pages, "free_pages"}, {free_count, "free_count"}, {lens, "lens"}, {counts, "counts"}, {start, "start"}, {taken, "taken"},
      {new_lens, "new_lens"}, {first, "first"}, {free_left, "free_left"}, {slots, "slots"}, {positions, "positions"}};
  for (auto& x : arrays)
    if (s == SAGE_OK) s = check_ints(x.first, x.second);
  if (s != SAGE_OK) return s;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.lens = lens;
  a.counts = counts;
  a.table = block_table;
  a.table_stride = table_stride;
  a.num_pages = num_pages;
  a.B = B;
  a.layout = layout;
  a.tokens = tokens;
  a.start = start;
  a.taken = taken;
  a.new_lens = new_lens;
  a.first = first;
  a.free_left = free_left;
  a.slots = slots;
  a.positions = positions;
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "device error word");
  if (fault_fires(SAGE_FAULT_QUANT_LAUNCH)) return fail(SAGE_ERR_CUDA, "page reservation launch: injected fault");
  e = launch_pages_reserve(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SAGE_OK : cuda_fail(e, "page reservation launch");
}

sage_status sage_kv_pages_release(int32_t* free_pages, int32_t* free_count, int num_pages, int page_size, int32_t* lens,
                                  const int32_t* keep, int B, int32_t* block_table, int table_width, int64_t table_stride,
                                  void* stream) {
  ReleaseArgs a = {};
  sage_status s = check_pages(num_pages, page_size, B, block_table, table_width, table_stride, &a.page_shift, &a.room);
  if (s == SAGE_OK) s = check_ints(free_pages, "free_pages");
  if (s == SAGE_OK) s = check_ints(free_count, "free_count");
  if (s == SAGE_OK) s = check_ints(lens, "lens");
  if (s == SAGE_OK) s = check_ints(keep, "keep");
  if (s != SAGE_OK) return s;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.lens = lens;
  a.keep = keep;
  a.table = block_table;
  a.table_stride = table_stride;
  a.num_pages = num_pages;
  a.B = B;
  cudaError_t e = device_error_word(&a.err);
  if (e != cudaSuccess) return cuda_fail(e, "device error word");
  if (fault_fires(SAGE_FAULT_QUANT_LAUNCH)) return fail(SAGE_ERR_CUDA, "page release launch: injected fault");
  e = launch_pages_release(a, static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SAGE_OK : cuda_fail(e, "page release launch");
}

sage_status sage_attn_fwd_cache(const void* q, int64_t q_stride_b, int64_t q_stride_s, const sage_kv_cache* cache,
                                const int32_t* block_table, int table_width, int64_t table_stride,
                                const int32_t* lens, void* out, float* lse, int B, int Sq, int Hq, int D,
                                float softmax_scale, int causal, void* workspace, size_t workspace_bytes,
                                void* stream) {
  return run_cache_attention(q, q_stride_b, q_stride_s, cache, nullptr, 0, block_table, table_width, table_stride,
                             lens, out, lse, B, Sq, Hq, D, softmax_scale, causal, workspace, workspace_bytes, stream);
}

sage_status sage_attn_fwd_cache_prefix(const void* q, int64_t q_stride_b, int64_t q_stride_s,
                                       const sage_kv_cache* cache, const int32_t* prefix_table, int prefix_len,
                                       const int32_t* block_table, int table_width, int64_t table_stride,
                                       const int32_t* lens, void* out, float* lse, int B, int Sq, int Hq, int D,
                                       float softmax_scale, int causal, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  return run_prefix_attention(q, q_stride_b, q_stride_s, cache, prefix_table, prefix_len, block_table, table_width,
                              table_stride, lens, out, lse, B, Sq, Hq, D, softmax_scale, causal, workspace,
                              workspace_bytes, stream);
}

sage_status sage_attn_fwd_kv4_cache(const void* q, int64_t q_stride_b, int64_t q_stride_s, const sage_kv4_cache* cache,
                                    const int32_t* block_table, int table_width, int64_t table_stride,
                                    const int32_t* lens, void* out, float* lse, int B, int Sq, int Hq, int D,
                                    float softmax_scale, int causal, void* workspace, size_t workspace_bytes,
                                    void* stream) {
  return run_cache_attention(q, q_stride_b, q_stride_s, cache, nullptr, 0, block_table, table_width, table_stride,
                             lens, out, lse, B, Sq, Hq, D, softmax_scale, causal, workspace, workspace_bytes, stream);
}

sage_status sage_attn_fwd_kv4_cache_prefix(const void* q, int64_t q_stride_b, int64_t q_stride_s,
                                           const sage_kv4_cache* cache, const int32_t* prefix_table, int prefix_len,
                                           const int32_t* block_table, int table_width, int64_t table_stride,
                                           const int32_t* lens, void* out, float* lse, int B, int Sq, int Hq, int D,
                                           float softmax_scale, int causal, void* workspace, size_t workspace_bytes,
                                           void* stream) {
  return run_prefix_attention(q, q_stride_b, q_stride_s, cache, prefix_table, prefix_len, block_table, table_width,
                              table_stride, lens, out, lse, B, Sq, Hq, D, softmax_scale, causal, workspace,
                              workspace_bytes, stream);
}

size_t sage_attn_fwd_cache_workspace_bytes(int B, int Sq, int Hq, int H, int prefix_len) {
  if (B < 1 || Sq < 1 || Hq < 1 || H < 1 || Hq % H != 0 || prefix_len < 0 || prefix_len > kMaxCacheLen ||
      static_cast<int64_t>(B) * Hq > INT_MAX || static_cast<int64_t>(B) * Hq > INT_MAX / Sq)
    return 0;
  return cache_attn_workspace_bytes(B, Sq, Hq, H, prefix_len);
}

sage_status sage_debug_fused_q(const void* q, const void* k, const void* v, void* out, int B, int S, int H,
                               int D, float softmax_scale, int8_t* q_i8, float* q_scale, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK) s = check_scale(softmax_scale);
  if (s == SAGE_OK)
    s = check_ptrs({{q, "q"}, {k, "k"}, {v, "v"}, {out, "out"}, {q_i8, "q_i8"}, {q_scale, "q_scale"}});
  if (s == SAGE_OK) s = check_out(out);
  if (s != SAGE_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return with_pool_workspace(ws_layout(B, S, S, H).total, st, [&](void* ws) {
    return run_fused(q, k, v, out, B, S, S, H, softmax_scale, ws, st, nullptr, true, q_i8, q_scale);
  });
}

sage_status sage_debug_staging_codes(const void* q, const void* k, int B, int S, int H, int D, void* q16,
                                     float* q_scale, void* k16, float* k_scale, void* stream) {
  sage_status s = check_shape(B, S, H, D);
  if (s == SAGE_OK)
    s = check_ptrs({{q, "q"}, {k, "k"}, {q16, "q16"}, {q_scale, "q_scale"}, {k16, "k16"}, {k_scale, "k_scale"}});
  if (s != SAGE_OK) return s;
  const QKQuantArgs<__half> qa = staging_args(q, k, B, S, S, H, static_cast<__half*>(q16), q_scale,
                                              static_cast<__half*>(k16), k_scale, false, nullptr);
  cudaError_t e = launch_qkv_quantize<__half>(qa, nullptr, nullptr, nullptr, nullptr, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "Q/K quantisation launch");
  return SAGE_OK;
}

sage_status sage_debug_inject_fault(int site, int skip) {
  if (site < SAGE_FAULT_NONE || site > SAGE_FAULT_ATTN_LAUNCH || skip < 0)
    return fail(SAGE_ERR_INVALID_ARG, "fault site %d / skip %d out of range", site, skip);
  g_fault_site.store(SAGE_FAULT_NONE, std::memory_order_relaxed);
  g_fault_skip.store(skip, std::memory_order_relaxed);
  g_fault_site.store(site, std::memory_order_relaxed);
  return SAGE_OK;
}

sage_status sage_debug_pool_state(int* created, uint64_t* used_bytes) {
  if (!created || !used_bytes) return fail(SAGE_ERR_INVALID_ARG, "created and used_bytes must not be NULL");
  int dev = 0;
  sage_status s = current_device(&dev);
  if (s != SAGE_OK) return s;
  cudaMemPool_t pool;
  {
    std::lock_guard<std::mutex> lk(g_pool_mu);
    pool = g_pools[dev];
  }
  *created = pool != nullptr;
  *used_bytes = 0;
  if (pool) {
    cuuint64_t used = 0;
    cudaError_t e = cudaMemPoolGetAttribute(pool, cudaMemPoolAttrUsedMemCurrent, &used);
    if (e != cudaSuccess) return cuda_fail(e, "memory pool query");
    *used_bytes = static_cast<uint64_t>(used);
  }
  return SAGE_OK;
}

sage_status sage_debug_wait_timeout(uint64_t ns, void* stream) {
  if (ns < 1 || ns > 10000000000ull) return fail(SAGE_ERR_INVALID_ARG, "timeout_ns must be in [1, 1e10]");
  cudaError_t e = launch_wait_timeout_probe(ns, static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "wait probe launch");
  return SAGE_OK;
}

sage_status sage_sync_status(void* stream) {
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaStreamSynchronize(st);
  if (e != cudaSuccess) return cuda_fail(e, "stream synchronise");
  int code = 0;
  e = read_and_clear_device_error(&code, st);
  if (e != cudaSuccess) return cuda_fail(e, "device error word read");
  if (code == SAGE_DEVERR_TIMEOUT)
    return fail(SAGE_ERR_TIMEOUT, "a device-side wait gave up after its time limit");
  if (code == SAGE_DEVERR_BAD_PAGE)
    return fail(SAGE_ERR_BAD_PAGE, "a page table led out of the cache, or a position out of its table");
  if (code == SAGE_DEVERR_NO_PAGES)
    return fail(SAGE_ERR_NO_PAGES, "the free list had too few pages for all sequences");
  return SAGE_OK;
}

void sage_set_attention_events(void* before, void* after) {
  t_attn_before = static_cast<cudaEvent_t>(before);
  t_attn_after = static_cast<cudaEvent_t>(after);
}

void sage_set_wait_timeout_ns(uint64_t ns) { g_timeout_ns.store(ns ? ns : kDefaultTimeoutNs); }

const char* sage_last_error(void) { return t_last_error.c_str(); }

const char* sage_status_string(sage_status s) {
  switch (s) {
    case SAGE_OK: return "SAGE_OK";
    case SAGE_ERR_INVALID_ARG: return "SAGE_ERR_INVALID_ARG";
    case SAGE_ERR_UNSUPPORTED: return "SAGE_ERR_UNSUPPORTED";
    case SAGE_ERR_MISALIGNED: return "SAGE_ERR_MISALIGNED";
    case SAGE_ERR_CUDA: return "SAGE_ERR_CUDA";
    case SAGE_ERR_NO_MEMORY: return "SAGE_ERR_NO_MEMORY";
    case SAGE_ERR_TIMEOUT: return "SAGE_ERR_TIMEOUT";
    case SAGE_ERR_WORKSPACE: return "SAGE_ERR_WORKSPACE";
    case SAGE_ERR_BAD_PAGE: return "SAGE_ERR_BAD_PAGE";
    case SAGE_ERR_NO_PAGES: return "SAGE_ERR_NO_PAGES";
  }
  return "SAGE_ERR_UNKNOWN";
}

}  // extern "C"
