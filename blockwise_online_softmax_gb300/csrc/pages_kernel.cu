// Page bookkeeping on the GPU: block tables, slots and positions of a step,
// and the pages of finished requests back on the free list.
//
// Both are a prefix sum over the requests and then one independent piece of
// work per token or page.  A few microseconds of latency are all there is to
// win, so a small step is one CTA that does everything.  A large one is that
// CTA with the sums alone (kept in scratch) and a second launch over the
// whole GPU that finds each token's or page's request by search.
//
// Every index into the table, the stack or an output is derived from clamped
// lengths and sums, so values that make no sense give outputs that make no
// sense, or a status, but no access outside the arrays.
#include <cstdint>

#include "launch.cuh"
#include "serve_internal.h"

namespace ra {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kBook = 1024;  // threads of the bookkeeping CTA, requests per chunk
constexpr int kSpread = 256; // threads of the second launch's CTAs

// Exclusive prefix sum of one value per thread of the CTA; *total gets the
// sum.  Every thread calls it; it synchronizes before it returns.
template <typename V>
__device__ __forceinline__ V block_scan(V v, V* total) {
  __shared__ V s_warp[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // s_warp of an earlier call has been read
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  // Each warp scans the 32 warp sums for itself.
  V w = s_warp[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(kAll, w, o);
    if (lane >= o) w += y;
  }
  *total = __shfl_sync(kAll, w, 31);
  const V before = __shfl_sync(kAll, w, warp ? warp - 1 : 0);
  return x - v + (warp ? before : 0);
}

// The last i in [0, n) with first[i] <= x (first nondecreasing, first[0] <= x).
__device__ __forceinline__ int find_last(const int* first, int n, int x) {
  int a = 0, b = n;
  while (b - a > 1) {
    const int mid = (a + b) >> 1;
    if (first[mid] <= x) a = mid; else b = mid;
  }
  return a;
}

__device__ __forceinline__ int at_least_0(int x) { return x < 0 ? 0 : x; }

__device__ __forceinline__ int stack_count(const int* count, int capacity) {
  const int c = *count;
  return c < 0 ? 0 : (c > capacity ? capacity : c);
}

// ------------------------------------------------------------------ extend
// The sums and the status; with ALL also the pages and tokens.  Pass 1 adds
// up what the step needs; with any of it missing the step changes nothing.
// Pass 2 takes the requests in chunks of one per thread: prefix sums of the
// new pages and tokens and, with ALL, the chunk's pages, then its tokens,
// dealt to the threads by search in those sums.
template <bool ALL>
__global__ void __launch_bounds__(kBook) paged_extend_kernel(const ExtendArgs a) {
  __shared__ int s_page[kBook], s_cu[kBook], s_len[kBook];
  __shared__ long long s_need, s_toks;
  __shared__ int s_bad;
  const int tid = threadIdx.x, sh = a.page_shift;
  const long long ps1 = (1LL << sh) - 1;
  let_next_start();
  wait_for_previous();
  const int count = stack_count(a.free_count, a.free_capacity);
  if (tid == 0) {
    s_need = s_toks = 0;
    s_bad = 0;
  }
  // One request per thread stays in registers for pass 2 (the first chunk).
  const int len0 = tid < a.n_req ? at_least_0(a.lengths[tid]) : 0;
  const int new0 = tid < a.n_req ? at_least_0(a.new_tokens[tid]) : 0;
  long long need = 0, toks = 0;
  int bad = 0;
  for (int i = tid; i < a.n_req; i += kBook) {
    const long long len = i == tid ? len0 : at_least_0(a.lengths[i]);
    const long long nw = i == tid ? new0 : at_least_0(a.new_tokens[i]);
    const long long pages = (len + nw + ps1) >> sh;
    need += pages - ((len + ps1) >> sh);
    toks += nw;
    bad += pages > a.max_pages;
  }
  __syncthreads();
  if (tid < ((a.n_req + 31) & ~31)) {  // whole warps that hold a request
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      need += __shfl_xor_sync(kAll, need, o);
      toks += __shfl_xor_sync(kAll, toks, o);
    }
    bad = __reduce_add_sync(kAll, bad);
    if ((tid & 31) == 0) {  // integer sums: their order does not matter
      atomicAdd(reinterpret_cast<unsigned long long*>(&s_need), static_cast<unsigned long long>(need));
      atomicAdd(reinterpret_cast<unsigned long long*>(&s_toks), static_cast<unsigned long long>(toks));
      if (bad) atomicAdd(&s_bad, bad);
    }
  }
  __syncthreads();
  need = s_need;
  toks = s_toks;
  bad = s_bad;
  const bool ok = need <= count && bad == 0 && toks <= a.tokens;
  if (tid == 0) {
    const long long lack = need - count, over = toks - a.tokens;
    a.status[0] = lack > 0 ? static_cast<int>(lack > 0x7fffffff ? 0x7fffffff : lack) : 0;
    a.status[1] = bad;
    a.status[2] = over > 0 ? static_cast<int>(over > 0x7fffffff ? 0x7fffffff : over) : 0;
    *a.free_count_out = ok ? count - static_cast<int>(need) : count;
    a.cu_tokens[0] = 0;
    if (!ALL) a.first_page[a.n_req] = count;
  }
  int page0 = 0, tok0 = 0;  // pages and tokens of the chunks before
  for (int i0 = 0; i0 < a.n_req; i0 += kBook) {
    const int i = i0 + tid;
    const bool in = i < a.n_req;
    const int len = i0 == 0 ? len0 : (in ? at_least_0(a.lengths[i]) : 0);
    const int nw = !ok ? 0 : (i0 == 0 ? new0 : (in ? at_least_0(a.new_tokens[i]) : 0));
    const int old = static_cast<int>((len + ps1) >> sh);
    const int fresh = ok ? static_cast<int>((static_cast<long long>(len) + nw + ps1) >> sh) - old : 0;
    // Both sums fit 31 bits once the step is known to fit.
    unsigned long long both;
    const unsigned long long at = block_scan<unsigned long long>(
        (static_cast<unsigned long long>(fresh) << 32) | static_cast<unsigned>(nw), &both);
    const int p = static_cast<int>(at >> 32), t = static_cast<int>(at & 0xffffffffu);
    const int pages = static_cast<int>(both >> 32), tokens = static_cast<int>(both & 0xffffffffu);
    if (in) {
      a.lengths_out[i] = len + nw;
      a.cu_tokens[i + 1] = tok0 + t + nw;
      if (!ALL) a.first_page[i] = page0 + p;
    }
    if (ALL) {
      s_page[tid] = p;
      s_cu[tid] = t;
      s_len[tid] = len;
      __syncthreads();
      for (int x = tid; x < pages; x += kBook) {
        const int r = find_last(s_page, kBook, x);
        const int c = static_cast<int>((s_len[r] + ps1) >> sh) + (x - s_page[r]);
        a.block_table[static_cast<long long>(i0 + r) * a.max_pages + c] =
            a.free_pages[count - 1 - (page0 + x)];
      }
      for (int x = tid; x < tokens; x += kBook) {
        const int r = find_last(s_cu, kBook, x);
        const int pos = s_len[r] + (x - s_cu[r]);
        // A page that is new comes off the stack here too, without waiting
        // for the table.
        const int c = pos >> sh, fresh_at = c - static_cast<int>((s_len[r] + ps1) >> sh);
        const long long page = fresh_at >= 0
            ? a.free_pages[count - 1 - (page0 + s_page[r] + fresh_at)]
            : a.block_table[static_cast<long long>(i0 + r) * a.max_pages + c];
        a.slots[tok0 + x] = page < 0 ? -1 : (page << sh) + (pos & ps1);
        a.positions[tok0 + x] = pos;
      }
      __syncthreads();
    }
    page0 += pages;
    tok0 += tokens;
  }
  if (!ALL) return;
  for (long long x = tok0 + tid; x < a.tokens; x += kBook) {
    a.slots[x] = -1;
    a.positions[x] = 0;
  }
}

// One token row per thread.  A new page starts with a new token, whose thread
// writes the table entry.
__global__ void __launch_bounds__(kSpread) paged_extend_tokens_kernel(const ExtendArgs a) {
  const long long x = static_cast<long long>(blockIdx.x) * kSpread + threadIdx.x;
  const int sh = a.page_shift;
  const long long ps1 = (1LL << sh) - 1;
  let_next_start();
  wait_for_previous();
  if (x >= a.tokens) return;
  const int t = static_cast<int>(x);
  if (a.n_req == 0 || t >= a.cu_tokens[a.n_req]) {
    a.slots[t] = -1;
    a.positions[t] = 0;
    return;
  }
  const int r = find_last(a.cu_tokens, a.n_req, t);
  const int c0 = a.cu_tokens[r], len = a.lengths_out[r] - (a.cu_tokens[r + 1] - c0);
  const int pos = len + (t - c0);
  const int c = pos >> sh, fresh_at = c - static_cast<int>((len + ps1) >> sh);
  int* entry = a.block_table + static_cast<long long>(r) * a.max_pages + c;
  long long page;
  if (fresh_at >= 0) {
    page = a.free_pages[a.first_page[a.n_req] - 1 - (a.first_page[r] + fresh_at)];
    if ((pos & ps1) == 0) *entry = static_cast<int>(page);
  } else {
    page = *entry;
  }
  a.slots[t] = page < 0 ? -1 : (page << sh) + (pos & ps1);
  a.positions[t] = pos;
}

// ------------------------------------------------------------------ release
// The sums; with ALL also the pages.  Every access to the stack is checked
// against its capacity, every table read against the row.
template <bool ALL>
__global__ void __launch_bounds__(kBook) paged_release_kernel(const ReleaseArgs a) {
  __shared__ int s_page[kBook];
  const int tid = threadIdx.x, sh = a.page_shift;
  const long long ps1 = (1LL << sh) - 1;
  let_next_start();
  wait_for_previous();
  const long long count = stack_count(a.free_count, a.free_capacity);
  int top = 0;  // pages of the chunks before (at most the table's entries)
  for (int i0 = 0; i0 < a.n_req; i0 += kBook) {
    const int i = i0 + tid;
    const bool in = i < a.n_req;
    const int len = in ? at_least_0(a.lengths[i]) : 0;
    const bool fin = in && a.finished[i] != 0;
    const long long have = fin ? (len + ps1) >> sh : 0;
    int pages;
    const int p = block_scan<int>(static_cast<int>(have < a.max_pages ? have : a.max_pages), &pages);
    if (in) {
      a.lengths_out[i] = fin ? 0 : len;
      if (!ALL) a.first_page[i] = top + p;
    }
    if (ALL) {
      s_page[tid] = p;
      __syncthreads();
      for (int x = tid; x < pages; x += kBook) {
        const int r = find_last(s_page, kBook, x);
        if (count + top + x < a.free_capacity)
          a.free_pages[count + top + x] =
              a.block_table[static_cast<long long>(i0 + r) * a.max_pages + (x - s_page[r])];
      }
      __syncthreads();
    }
    top += pages;
  }
  if (tid) return;
  const long long end = count + top;
  *a.free_count_out = static_cast<int>(end < a.free_capacity ? end : a.free_capacity);
  if (!ALL) {
    a.first_page[a.n_req] = top;
    a.first_page[a.n_req + 1] = static_cast<int>(count);
  }
}

__global__ void __launch_bounds__(kSpread) paged_release_pages_kernel(const ReleaseArgs a) {
  let_next_start();
  wait_for_previous();
  const int total = a.first_page[a.n_req];
  const long long count = a.first_page[a.n_req + 1];
  for (long long x = static_cast<long long>(blockIdx.x) * kSpread + threadIdx.x; x < total;
       x += static_cast<long long>(gridDim.x) * kSpread) {
    if (count + x >= a.free_capacity) return;
    const int r = find_last(a.first_page, a.n_req, static_cast<int>(x));
    a.free_pages[count + x] =
        a.block_table[static_cast<long long>(r) * a.max_pages + (x - a.first_page[r])];
  }
}

}  // namespace

// One CTA passes about 1 token or page per nanosecond; a second launch and its
// scratch cost some 4 us.
bool paged_extend_needs_scratch(const ExtendArgs& a) { return a.tokens > 4096; }
bool paged_release_needs_scratch(const ReleaseArgs& a) {
  return static_cast<long long>(a.n_req) * a.max_pages > 16384;
}

cudaError_t launch_paged_extend(const ExtendArgs& a, cudaStream_t st) {
  return launch_early(a.first_page ? paged_extend_kernel<false> : paged_extend_kernel<true>, dim3(1), kBook, 0, st, a);
}

cudaError_t launch_paged_extend_tokens(const ExtendArgs& a, cudaStream_t st) {
  return launch_early(paged_extend_tokens_kernel,
                      dim3(static_cast<unsigned>((a.tokens + kSpread - 1) / kSpread)), kSpread, 0, st, a);
}

cudaError_t launch_paged_release(const ReleaseArgs& a, cudaStream_t st) {
  return launch_early(a.first_page ? paged_release_kernel<false> : paged_release_kernel<true>, dim3(1), kBook, 0, st, a);
}

cudaError_t launch_paged_release_pages(const ReleaseArgs& a, cudaStream_t st) {
  const long long most = (static_cast<long long>(a.n_req) * a.max_pages + kSpread - 1) / kSpread;
  return launch_early(paged_release_pages_kernel, dim3(static_cast<unsigned>(most < 608 ? most : 608)), kSpread, 0,
                      st, a);
}

}  // namespace ra
