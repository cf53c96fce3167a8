// Page bookkeeping on the GPU, and decode attention over paged keys and
// values.
#include <cmath>
#include <cstdint>

#include <cuda_bf16.h>

#include "ptx.cuh"
#include "serve_internal.h"

namespace ra {

__device__ int g_paged_status = 0;

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

// ------------------------------------------------------------------ paged decode
// One CTA per (query row, head): warp w takes keys w, w + 8, ... with the
// lanes over the columns and its own running (m, l, O~); the warps' states
// meet in shared memory.
template <int D>
__global__ void __launch_bounds__(256) paged_decode_kernel(const PagedArgs a) {
  constexpr int CPL = D / 32, W = 8;
  __shared__ float s_m[W], s_l[W], s_o[W][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long t = blockIdx.x;
  const int h = blockIdx.y, kh = h / (a.heads / a.kv_heads);
  long long r = t / a.n_q, first = r * a.n_q, last = first + a.n_q;
  if (a.cu_q) {
    r = find_last(a.cu_q, a.n_req, static_cast<int>(t));
    first = a.cu_q[r];
    last = a.cu_q[r + 1];
    if (t < first || t >= last) return;  // a row behind the last request: left as it was
  }
  const int sh = a.page_shift;
  long long len = a.lengths[r];
  const long long most = static_cast<long long>(a.max_pages) << sh;
  len = len < 0 ? 0 : (len > most ? most : len);
  long long hi = len - (last - t) + 1;
  if (hi < 0) hi = 0;
  const long long lo = a.window > 0 && hi - a.window > 0 ? hi - a.window : 0;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) + (t * a.heads + h) * D + CPL * lane;
  float qv[CPL], o[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    qv[c] = __bfloat162float(q[c]);
    o[c] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (long long key = lo + warp; key < hi; key += W) {
    const int page = a.block_table[r * a.max_pages + (key >> sh)];
    if (page < 0 || page >= a.n_pages) continue;
    const long long in = ((key & ((1LL << sh) - 1)) * a.kv_heads + kh) * D + CPL * lane;
    const __nv_bfloat16* k = static_cast<const __nv_bfloat16*>(a.kc) + page * a.kc_page + in;
    const __nv_bfloat16* v = static_cast<const __nv_bfloat16*>(a.vc) + page * a.vc_page + in;
    float s = 0.f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) s = fmaf(qv[c], __bfloat162float(k[c]), s);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) s += __shfl_xor_sync(kAll, s, x);
    s *= a.scale_log2;
    if (s == -INFINITY) continue;
    const float mn = fmaxf(m, s), al = exp2f(m - mn), p = exp2f(s - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int c = 0; c < CPL; ++c) o[c] = fmaf(p, __bfloat162float(v[c]), o[c] * al);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int c = 0; c < CPL; ++c) s_o[warp][CPL * lane + c] = o[c];
  __syncthreads();
  float mx = -INFINITY, lt = 0.f;
  for (int w = 0; w < W; ++w) mx = fmaxf(mx, s_m[w]);
  const float ref = mx == -INFINITY ? 0.f : mx;
  for (int w = 0; w < W; ++w) lt += s_l[w] * exp2f(s_m[w] - ref);
  const float inv = lt > 0.f ? 1.f / lt : 0.f;
  for (int x = threadIdx.x; x < D; x += 256) {
    float y = 0.f;
    for (int w = 0; w < W; ++w) y = fmaf(s_o[w][x], exp2f(s_m[w] - ref), y);
    const long long at = (t * a.heads + h) * D + x;
    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y * inv);
    else static_cast<float*>(a.out)[at] = y * inv;
  }
  if (threadIdx.x == 0) a.lse[t * a.heads + h] = lt > 0.f ? mx * kLn2 + logf(lt) : -INFINITY;
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

cudaError_t launch_paged_decode(const PagedArgs& a, int d, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.T), static_cast<unsigned>(a.heads));
  if (d == 128) paged_decode_kernel<128><<<grid, 256, 0, st>>>(a);
  else paged_decode_kernel<64><<<grid, 256, 0, st>>>(a);
  return cudaGetLastError();
}

cudaError_t take_paged_status(int* code) {
  int zero = 0;
  cudaError_t e = cudaMemcpyFromSymbol(code, g_paged_status, sizeof(int));
  if (e != cudaSuccess) return e;
  return cudaMemcpyToSymbol(g_paged_status, &zero, sizeof(int));
}

}  // namespace ra
