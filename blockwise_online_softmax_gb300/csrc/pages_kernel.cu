// Page bookkeeping on the GPU: block tables, slots and positions of a step,
// and the pages of finished requests back on the free list.
#include <cstdint>

#include "serve_internal.h"

namespace ra {

namespace {

constexpr unsigned kAll = 0xffffffffu;

// ------------------------------------------------------------------ bookkeeping
constexpr int kBook = 1024;  // threads of the bookkeeping CTA, requests per chunk

// Exclusive prefix sum of one value per thread of the CTA; *total gets the
// sum.  Every thread calls it; it synchronizes before it returns.
__device__ __forceinline__ int block_scan(int v, int* total) {
  __shared__ int s_warp[33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();  // s_warp of an earlier call has been read
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    int w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(kAll, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[31];
  return x - v + (warp ? s_warp[warp - 1] : 0);
}

__device__ __forceinline__ long long block_sum(long long v) {
  __shared__ long long s_sum[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  __syncthreads();
  if (lane == 0) s_sum[warp] = v;
  __syncthreads();
  long long s = s_sum[lane];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(kAll, s, o);
  return s;
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

// One CTA.  Pass 1 sums what the step needs and sets the status; with any
// of it missing the step changes nothing.  Pass 2 takes the requests in
// chunks of one per thread: prefix sums of the new pages and tokens, then
// the chunk's pages, and after them its tokens, are dealt to the threads by
// search in those sums.
__global__ void __launch_bounds__(kBook) paged_extend_kernel(const ExtendArgs a) {
  __shared__ int s_page[kBook + 1], s_cu[kBook + 1], s_len[kBook], s_old[kBook];
  const int tid = threadIdx.x, sh = a.page_shift;
  const long long ps1 = (1LL << sh) - 1;
  int count = *a.free_count;
  count = count < 0 ? 0 : (count > a.free_capacity ? a.free_capacity : count);
  long long need = 0, toks = 0, bad = 0;
  for (int i = tid; i < a.n_req; i += kBook) {
    const long long len = at_least_0(a.lengths[i]), nw = at_least_0(a.new_tokens[i]);
    const long long pages = (len + nw + ps1) >> sh;
    need += pages - ((len + ps1) >> sh);
    toks += nw;
    bad += pages > a.max_pages;
  }
  need = block_sum(need);
  toks = block_sum(toks);
  bad = block_sum(bad);
  const bool ok = need <= count && bad == 0 && toks <= a.tokens;
  if (tid == 0) {
    const long long lack = need - count, over = toks - a.tokens;
    a.status[0] = lack > 0 ? static_cast<int>(lack > 0x7fffffff ? 0x7fffffff : lack) : 0;
    a.status[1] = static_cast<int>(bad);
    a.status[2] = over > 0 ? static_cast<int>(over > 0x7fffffff ? 0x7fffffff : over) : 0;
    *a.free_count_out = ok ? count - static_cast<int>(need) : count;
    a.cu_tokens[0] = 0;
  }
  int page0 = 0, tok0 = 0;  // pages and tokens of the chunks before
  for (int i0 = 0; i0 < a.n_req; i0 += kBook) {
    const int i = i0 + tid;
    const bool in = i < a.n_req;
    const int len = in ? at_least_0(a.lengths[i]) : 0;
    const int nw = in && ok ? at_least_0(a.new_tokens[i]) : 0;
    const int old = static_cast<int>((len + ps1) >> sh);
    const int fresh = ok ? static_cast<int>((static_cast<long long>(len) + nw + ps1) >> sh) - old : 0;
    int pages, tokens;
    const int p = block_scan(fresh, &pages), t = block_scan(nw, &tokens);
    s_page[tid] = p;
    s_cu[tid] = t;
    s_len[tid] = len;
    s_old[tid] = old;
    if (tid == 0) {
      s_page[kBook] = pages;
      s_cu[kBook] = tokens;
    }
    if (in) {
      a.lengths_out[i] = len + nw;
      a.cu_tokens[i + 1] = tok0 + t + nw;
    }
    __syncthreads();
    for (int x = tid; x < pages; x += kBook) {
      const int r = find_last(s_page, kBook, x);
      a.block_table[static_cast<long long>(i0 + r) * a.max_pages + s_old[r] + (x - s_page[r])] =
          a.free_pages[count - 1 - (page0 + x)];
    }
    __syncthreads();
    for (int x = tid; x < tokens; x += kBook) {
      const int r = find_last(s_cu, kBook, x);
      const int pos = s_len[r] + (x - s_cu[r]);
      const long long page = a.block_table[static_cast<long long>(i0 + r) * a.max_pages + (pos >> sh)];
      a.slots[tok0 + x] = page < 0 ? -1 : (page << sh) + (pos & ps1);
      a.positions[tok0 + x] = pos;
    }
    page0 += pages;
    tok0 += tokens;
    __syncthreads();
  }
  for (long long x = tok0 + tid; x < a.tokens; x += kBook) {
    a.slots[x] = -1;
    a.positions[x] = 0;
  }
}

// One CTA; chunks as above.  Every access to the free list is checked
// against its capacity, every table read against the row.
__global__ void __launch_bounds__(kBook) paged_release_kernel(const ReleaseArgs a) {
  __shared__ int s_page[kBook + 1];
  const int tid = threadIdx.x, sh = a.page_shift;
  const long long ps1 = (1LL << sh) - 1;
  int count = *a.free_count;
  count = count < 0 ? 0 : (count > a.free_capacity ? a.free_capacity : count);
  long long top = count;
  for (int i0 = 0; i0 < a.n_req; i0 += kBook) {
    const int i = i0 + tid;
    const bool in = i < a.n_req;
    const int len = in ? at_least_0(a.lengths[i]) : 0;
    const bool fin = in && a.finished[i] != 0;
    const long long have = fin ? (len + ps1) >> sh : 0;
    int pages;
    s_page[tid] = block_scan(static_cast<int>(have < a.max_pages ? have : a.max_pages), &pages);
    if (in) a.lengths_out[i] = fin ? 0 : len;
    __syncthreads();
    for (int x = tid; x < pages; x += kBook) {
      const int r = find_last(s_page, kBook, x);
      if (top + x < a.free_capacity)
        a.free_pages[top + x] =
            a.block_table[static_cast<long long>(i0 + r) * a.max_pages + (x - s_page[r])];
    }
    top += pages;
    __syncthreads();
  }
  if (tid == 0) *a.free_count_out = static_cast<int>(top < a.free_capacity ? top : a.free_capacity);
}

}  // namespace

cudaError_t launch_paged_extend(const ExtendArgs& a, cudaStream_t st) {
  paged_extend_kernel<<<1, kBook, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_paged_release(const ReleaseArgs& a, cudaStream_t st) {
  paged_release_kernel<<<1, kBook, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace ra
