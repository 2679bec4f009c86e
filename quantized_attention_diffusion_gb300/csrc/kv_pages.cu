// kv_pages.cu -- pages of the KV cache given to new tokens and taken back, on the
// GPU: block tables, slots and positions from lengths and counts (sm_103a).
//
// Sequence b holds len tokens in held = ceil(len / page) pages and asks for need =
// ceil((len + count) / page) - held more.  With upto_b the sum of need over sequences
// 0 .. b, the sequences with need = 0 or upto_b <= free are served: page j of b is
// entry free - 1 - (upto_b - need_b) - j of the free list, a stack.  Taking back puts
// pages where this found them, in the same order.  Of packed tokens a sequence's have to
// have rows as well; behind one that has too few none is served that has tokens.
//
// A few hundred bytes for a generation step: what it costs is the launch and a chain
// of loads, sums over the warps and barriers.  One CTA does the sums, 1024 sequences at a
// time; where tokens are few it does them and the pages too, a search for each (48
// sequences, one token each: 3.2 us), and otherwise a second kernel does, a CTA or some
// for a sequence.  Up to 1024 sequences its CTAs find their pages by a sum of their own
// over what the first has written (256 sequences, 200000 tokens in 12000 new pages:
// 8.6 us for both; with all pages in the first kernel 16.6).
#include <algorithm>
#include <climits>
#include <cuda_runtime.h>

#include "sage_internal.cuh"

namespace sage {

namespace {

constexpr int kThreads = 1024;
constexpr int kFewTokens = 8192;       // of a call that needs no second kernel
constexpr int kFillThreads = 256;

// Inclusive sums of a and b over the block; `part` has 2 x 32 values.  All threads.
__device__ __forceinline__ void block_sums(long long& a, long long& b, long long (*part)[32]) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long x = __shfl_up_sync(0xFFFFFFFFu, a, d), y = __shfl_up_sync(0xFFFFFFFFu, b, d);
    if (lane >= d) {
      a += x;
      b += y;
    }
  }
  if (lane == 31) {
    part[0][warp] = a;
    part[1][warp] = b;
  }
  __syncthreads();
  if (warp < 2) {
    long long x = part[warp][lane];
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long y = __shfl_up_sync(0xFFFFFFFFu, x, d);
      if (lane >= d) x += y;
    }
    part[warp][lane] = x;
  }
  __syncthreads();
  if (warp > 0) {
    a += part[0][warp - 1];
    b += part[1][warp - 1];
  }
}

// The first of n ascending values that is above x (n if none is).
__device__ __forceinline__ int above(const long long* v, int n, long long x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// The rows that a sequence's tokens take, served or not: none of a count that is not one.
__device__ __forceinline__ int rows_of(const PagesArgs& a, int count) { return count >= 0 && count <= a.tokens ? count : 0; }

// -1 where the table or the free list named a page that there is not.
__device__ __forceinline__ int slot_in(const PagesArgs& a, int page, int pos) {
  if (page < 0 || page >= a.num_pages) {
    atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
    return -1;
  }
  return (page << a.page_shift) + (pos & ((1 << a.page_shift) - 1));
}

__device__ __forceinline__ int slot_of(const PagesArgs& a, int b, int pos) {
  return slot_in(a, a.table[b * a.table_stride + (pos >> a.page_shift)], pos);
}

__global__ void __launch_bounds__(kThreads) reserve_kernel(const PagesArgs a, int do_tokens, int do_pages) {
  __shared__ long long s_upto[kThreads], s_rows[kThreads], part[2][32];
  __shared__ int s_start[kThreads], s_count[kThreads], s_served[kThreads];
  __shared__ long long s_gone;
  const int tid = threadIdx.x;
  const int page = 1 << a.page_shift;
  // The tokens of a padded call need nothing from the sums but who is served.
  const int raw = __ldg(a.free_count);
  const int free = max(0, min(raw, a.num_pages));
  bool bad = raw != free;
  if (tid == 0) s_gone = 0;
  long long pages_before = 0, rows_before = 0;
  for (int b0 = 0; b0 < a.B; b0 += kThreads) {
    const int b = b0 + tid, n = min(kThreads, a.B - b0);
    int len = 0, count = 0;
    bool fits = true;
    if (b < a.B) {
      len = a.lens[b];
      count = __ldg(a.counts + b);
      fits = len >= 0 && count >= 0 && static_cast<long long>(len) + count <= a.room && count <= a.tokens;
      if (!fits) bad = true;
    }
    const int held = fits ? (len + page - 1) >> a.page_shift : 0;
    const int need = fits ? ((len + count + page - 1) >> a.page_shift) - held : 0;
    long long upto = need, rows = rows_of(a, count);
    __syncthreads();                         // the arrays of the sequences before have been read
    block_sums(upto, rows, part);
    const bool has_rows = a.layout != kPagesPacked || count == 0 || rows_before + rows <= a.tokens;
    const bool served = fits && has_rows && (need == 0 || pages_before + upto <= free);
    // Ordinary, and told by `taken`: in the place of no error that is pending.
    if (b < a.B && fits && has_rows && !served) atomicCAS(a.err, SAGE_DEVERR_NONE, SAGE_DEVERR_NO_PAGES);
    s_upto[tid] = upto;
    s_rows[tid] = rows;
    s_start[tid] = len;
    s_count[tid] = count;
    s_served[tid] = served ? 1 : 0;
    if (b < a.B) {
      const int taken = served ? count : 0;
      a.start[b] = len;
      a.taken[b] = taken;
      a.new_lens[b] = len + taken;
      const long long at = a.layout == kPagesPacked ? rows_before + rows - rows_of(a, count)
                                                    : static_cast<long long>(b) * a.tokens + (a.layout == kPagesEnd ? a.tokens - rows_of(a, count) : 0);
      a.first[b] = static_cast<int>(min(at, static_cast<long long>(INT_MAX)));
      if (served && need > 0) atomicMax(&s_gone, pages_before + upto);
    }
    __syncthreads();
    // The pages of these sequences, those of the served.
    const long long total = s_upto[n - 1];
    for (long long j = tid; do_pages && j < total && pages_before + j < free; j += kThreads) {
      const int i = above(s_upto, n, j);
      if (s_served[i] == 0) break;           // nor is any behind it
      const long long in = j - (i > 0 ? s_upto[i - 1] : 0);
      const int at = ((s_start[i] + page - 1) >> a.page_shift) + static_cast<int>(in);
      a.table[(b0 + i) * a.table_stride + at] = __ldg(a.free_pages + (free - 1 - (pages_before + j)));
    }
    pages_before += total;
    rows_before += s_rows[n - 1];
  }
  __syncthreads();
  if (a.layout == kPagesPacked && rows_before > a.tokens) bad = true;   // tokens without a slot
  if (bad) atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
  if (tid == 0) *a.free_left = free - static_cast<int>(s_gone);
  if (do_tokens) {                           // B <= kThreads: all sequences are in the arrays
    const int rows = a.layout == kPagesPacked ? a.tokens : a.tokens * a.B;
    for (int r = tid; r < rows; r += kThreads) {
      int b, i;
      if (a.layout == kPagesPacked) {
        b = above(s_rows, a.B, r);
        i = b < a.B ? r - static_cast<int>(b > 0 ? s_rows[b - 1] : 0) : 0;
      } else {
        b = r / a.tokens;
        i = r - b * a.tokens - (a.layout == kPagesEnd ? a.tokens - rows_of(a, s_count[b]) : 0);
      }
      const bool live = b < a.B && s_served[b] != 0 && i >= 0 && i < s_count[b];
      const int pos = live ? s_start[b] + i : 0;
      a.slots[r] = live ? slot_of(a, b, pos) : -1;
      a.positions[r] = pos;
    }
  }
}

// Slots and positions of sequence blockIdx.x's tokens; for packed tokens block B has
// the rows behind the last.  do_pages: and its new pages, which the first kernel has left:
// a sequence that was served, and it alone, has taken tokens that need some.
__global__ void __launch_bounds__(kFillThreads) fill_kernel(const PagesArgs a, int do_pages) {
  __shared__ int s_before, s_all;            // pages of the sequences before this one, of all
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int b = blockIdx.x, tid = threadIdx.x;
  const bool packed = a.layout == kPagesPacked;
  const int step = gridDim.y * kFillThreads, i0 = blockIdx.y * kFillThreads + tid;
  if (b == a.B) {
    const long long end = static_cast<long long>(a.first[a.B - 1]) + rows_of(a, __ldg(a.counts + a.B - 1));
    for (long long r = end + i0; r < a.tokens; r += step) {
      a.slots[r] = -1;
      a.positions[r] = 0;
    }
    return;
  }
  const int count = rows_of(a, __ldg(a.counts + b)), taken = a.taken[b], start = a.start[b];
  const int page = 1 << a.page_shift;
  int held = INT_MAX, top = 0;               // the page of index j >= held is free_pages[top - (j - held)]
  if (do_pages) {                            // the sums are of pages that there are: below 2^31
    if (tid == 0) s_before = s_all = 0;
    __syncthreads();
    int before = 0, all = 0;
    for (int i = tid; i < a.B; i += kFillThreads) {
      const int t = a.taken[i], n = a.start[i];
      const int need = t > 0 ? ((n + t + page - 1) >> a.page_shift) - ((n + page - 1) >> a.page_shift) : 0;
      all += need;
      before += i < b ? need : 0;
    }
    all = __reduce_add_sync(0xFFFFFFFFu, all);
    before = __reduce_add_sync(0xFFFFFFFFu, before);
    if ((tid & 31) == 0) {
      atomicAdd(&s_all, all);
      atomicAdd(&s_before, before);
    }
    __syncthreads();
    if (taken > 0) {
      held = (start + page - 1) >> a.page_shift;
      top = *a.free_left + s_all - 1 - s_before;
      const int end = (start + taken + page - 1) >> a.page_shift;
      for (int j = held + i0; j < end; j += step) a.table[b * a.table_stride + j] = __ldg(a.free_pages + (top - (j - held)));
    }
  }
  const long long base = packed ? a.first[b] : static_cast<long long>(b) * a.tokens;
  const int skip = a.layout == kPagesEnd ? a.tokens - count : 0;
  const long long rows = packed ? min(static_cast<long long>(count), a.tokens - base) : a.tokens;
  for (long long r = i0; r < rows; r += step) {
    const long long i = r - skip;
    const bool live = i >= 0 && i < taken;
    const int pos = live ? start + static_cast<int>(i) : 0;
    int slot = -1;
    if (live) {
      const int j = pos >> a.page_shift;
      slot = slot_in(a, j >= held ? __ldg(a.free_pages + (top - (j - held))) : a.table[b * a.table_stride + j], pos);
    }
    a.slots[base + r] = slot;
    a.positions[base + r] = pos;
  }
}

// An entry that is no page stays off the list.  Usually there is none, and the place of a
// page is known from the lengths: one that turns up is taken out again at the end (to look
// at all entries first took 27 us for 12000 pages where this takes 19).  Where the list
// has no room for all entries the pages are counted first.
__global__ void __launch_bounds__(kThreads) release_kernel(const ReleaseArgs a) {
  __shared__ long long s_upto[kThreads], part[2][32];
  __shared__ int s_kept[kThreads];
  const int tid = threadIdx.x;
  const int page = 1 << a.page_shift;
  const int raw = *a.free_count;
  const int free = max(0, min(raw, a.num_pages));
  bool bad = raw != free, odd = false;       // odd: an entry that is no page has been put on the list
  // The sum of all, for the order of the stack: page j of what is given back, counted
  // over the sequences, goes to entry free + pages - 1 - j.
  long long total = 0, pages = 0, none = 0;
  bool room = true;                          // the list's, for all entries
  auto is_page = [&](int p) { return p >= 0 && p < a.num_pages; };
  // The sum of n up to this thread; in part[0][31] that of all.
  auto sum = [&](long long n) {
    __syncthreads();                         // the sums before have been read
    block_sums(n, none, part);
    return n;
  };
  enum { kSum, kCount, kMove };
  for (int pass = kSum; pass <= kMove; ++pass) {
    if (pass == kCount && room) continue;
    long long before = 0, met = 0;
    for (int b0 = 0; b0 < a.B; b0 += kThreads) {
      const int b = b0 + tid, n = min(kThreads, a.B - b0);
      int len = 0, keep = 0;
      bool fits = false;
      if (b < a.B) {
        len = a.lens[b];
        keep = max(0, __ldg(a.keep + b));
        fits = len >= 0 && len <= a.room;
        if (!fits) bad = true;
      }
      const bool less = fits && keep < len;
      const int kept = less ? (keep + page - 1) >> a.page_shift : 0;
      const int give = less ? ((len + page - 1) >> a.page_shift) - kept : 0;
      const long long upto = sum(give);
      s_upto[tid] = upto;
      s_kept[tid] = kept;
      __syncthreads();
      const long long here = s_upto[n - 1];
      auto entry_of = [&](long long j) {
        const int i = above(s_upto, n, j);
        return a.table + (b0 + i) * a.table_stride + s_kept[i] + static_cast<int>(j - (i > 0 ? s_upto[i - 1] : 0));
      };
      if (pass == kMove && room) {
        for (long long j = tid; j < here; j += kThreads) {
          int32_t* entry = entry_of(j);
          const int p = *entry;
          odd |= !is_page(p);
          a.free_pages[free + total - 1 - (before + j)] = p;
          *entry = -1;
        }
      } else if (pass != kSum) {
        for (long long j0 = 0; j0 < here; j0 += kThreads) {      // all threads together
          int32_t* entry = j0 + tid < here ? entry_of(j0 + tid) : nullptr;
          const int p = entry != nullptr ? *entry : -1;
          const long long to = free + pages - met - sum(is_page(p) ? 1 : 0);
          met += part[0][31];
          if (pass == kMove) {
            if (is_page(p) && to < a.num_pages) a.free_pages[to] = p;
            if (entry != nullptr) *entry = -1;
          }
        }
      }
      if (pass == kMove && less) a.lens[b] = keep;
      before += here;
    }
    if (pass == kSum) {
      total = pages = before;
      room = free + total <= a.num_pages;
      bad |= !room;
    }
    if (pass == kCount) pages = met;
  }
  if (__syncthreads_or(odd)) {
    bad = true;
    pages = 0;
    for (long long i0 = 0; i0 < total; i0 += kThreads) {
      const int p = i0 + tid < total ? a.free_pages[free + i0 + tid] : -1;
      const long long to = free + pages + sum(is_page(p) ? 1 : 0) - 1;   // not above any that is still to be read
      if (is_page(p)) a.free_pages[to] = p;
      pages += part[0][31];
    }
  }
  if (bad) atomicExch(a.err, SAGE_DEVERR_BAD_PAGE);
  __syncthreads();                           // free_count has been read by all
  if (tid == 0) *a.free_count = static_cast<int>(min(static_cast<long long>(a.num_pages), free + pages));
}

}  // namespace

cudaError_t launch_pages_reserve(const PagesArgs& a, cudaStream_t stream) {
  const bool packed = a.layout == kPagesPacked;
  const int64_t rows = packed ? a.tokens : static_cast<int64_t>(a.tokens) * a.B;
  const bool one = a.B <= kThreads && rows <= kFewTokens;
  const int fill_pages = !one && a.B <= kThreads ? 1 : 0;
  reserve_kernel<<<1, kThreads, 0, stream>>>(a, one ? 1 : 0, fill_pages ? 0 : 1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || one) return e;
  const int64_t each = packed ? a.tokens / a.B + 1 : a.tokens;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) + (packed ? 1u : 0u),
                     static_cast<unsigned>(std::min<int64_t>(64, (each + 1023) / 1024)));
  cfg.blockDim = dim3(kFillThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, fill_kernel, a, fill_pages);
}

cudaError_t launch_pages_release(const ReleaseArgs& a, cudaStream_t stream) {
  release_kernel<<<1, kThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace sage
