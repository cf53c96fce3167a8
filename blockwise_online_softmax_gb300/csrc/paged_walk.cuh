// What the paged decode kernels share: the work list over requests, row tiles,
// KV heads and key tiles, and the page loads.  Device code only.
#pragma once
#include <atomic>
#include <cstdint>

#include "launch.cuh"
#include "ptx.cuh"
#include "serve_internal.h"

namespace ra {
namespace paged {

constexpr unsigned kAll = 0xffffffffu;

// What a CTA that starts a cut item leaves for the joining launch.
struct Cut {
  int last;   // last CTA of the item; -1: none
  int row0;   // first row of the q tensor of the request
  int rr0;    // first row of the tile (row rr: token rr / g, head kh * g + rr % g)
  int rows;
  int kh;
};

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const void* tmap, uint32_t bar, int c0,
                                            int c1, int c2, int c3) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3)
      : "memory");
}
// 16 bytes to shared memory, zeros when `bytes` is 0; the arrival on `bar`
// follows when the calling thread's copies have landed.
__device__ __forceinline__ void copy16(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void copies_arrive(uint32_t bar) {
  asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
// ------------------------------------------------------------------ the work list
struct Request {
  int row0;  // first row of q
  int n;     // new tokens
  int len;   // keys, the new tokens' included
  bool group;  // kBoth: a group of requests
};

// What the rows of a kernel are: the new tokens of requests, which see the keys up
// to themselves (kPlain: finished here; kOwn: partial states of them, for a
// launch that joins them with others), or all the tokens of a group of requests,
// which see every key of the group's prefix (kShared: partial states), or the one
// after the other in one launch (kBoth: the groups are its requests n_own and on).
constexpr int kPlain = kPagedPlain, kOwn = kPagedOwn, kShared = kPagedShared, kBoth = kPagedBoth;

// With kBoth two launches follow one another, else three: kOwn, kShared, the join.  The
// first two do not need each other, so kOwn lets the next start only once what was
// before it is done, and kShared does not wait before its work but after it: its
// CTAs take the SMs as kOwn's leave them, and its end means the end of both.
template <int MODE>
__device__ __forceinline__ void start_early() {
  if (MODE != kOwn) let_next_start();
}
template <int MODE>
__device__ __forceinline__ void start_wait() {
  if (MODE != kShared) wait_for_previous();
  if (MODE == kOwn) let_next_start();
}
template <int MODE>
__device__ __forceinline__ void end_wait() {
  if (MODE == kShared) wait_for_previous();
}

// Where the partial states of a row are: `first` and the count, -1 where the item
// is whole; + kWithPrefix in the own rows of requests that have a prefix.
constexpr int kWithPrefix = 1 << 20;  // (more than CTAs)
__device__ __forceinline__ int2 part_record(int first, int parts) { return make_int2(first, parts); }
// The requests that are one of a group: groups follow one another.
struct Joined {
  int first = 0, end = 0;
  __device__ __forceinline__ Joined(const PagedArgs& a) {
    if (a.n_groups > 0) {
      first = a.cu_req[0];
      end = a.cu_req[a.n_groups];
    }
  }
  __device__ __forceinline__ int mark(int r) const { return first <= r && r < end ? kWithPrefix : 0; }
};

template <int MODE>
__device__ __forceinline__ Request load_request(const PagedArgs& a, int r) {
  Request q;
  q.group = MODE == kShared || (MODE == kBoth && r >= a.n_own);
  const int* lengths = a.lengths;
  int pages = a.max_pages;
  if (q.group) {
    if (MODE == kBoth) {
      r -= a.n_own;
      lengths = a.prefix_lengths;
      pages = a.prefix_pages;
    }
    // The rows of requests [b, e), whatever the arrays say inside q and out.
    const int T = static_cast<int>(a.T), x = a.cu_req[r], y = a.cu_req[r + 1];
    const int b = x < 0 ? 0 : (x > a.n_own ? a.n_own : x), e = y < b ? b : (y > a.n_own ? a.n_own : y);
    const int v = a.cu_q ? a.cu_q[b] : b * static_cast<int>(a.n_q), w = a.cu_q ? a.cu_q[e] : e * static_cast<int>(a.n_q);
    q.row0 = v < 0 ? 0 : (v > T ? T : v);
    q.n = (w < q.row0 ? q.row0 : (w > T ? T : w)) - q.row0;
  } else if (a.cu_q) {
    // A malformed cu_q must not reach outside q and out.
    const int T = static_cast<int>(a.T), x = a.cu_q[r], y = a.cu_q[r + 1];
    q.row0 = x < 0 ? 0 : (x > T ? T : x);
    q.n = (y < q.row0 ? q.row0 : (y > T ? T : y)) - q.row0;
  } else {
    q.row0 = r * static_cast<int>(a.n_q);
    q.n = static_cast<int>(a.n_q);
  }
  const int most = pages << a.page_shift, len = lengths[r];
  q.len = len < 0 ? 0 : (len > most ? most : len);
  return q;
}

// Row rr of a request belongs to token rr / g (mostly the first one).
__device__ __forceinline__ int token_of(int rr, int g) { return rr < g ? 0 : rr / g; }

// a / b for b > 0, in 32 bits where that is enough.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((static_cast<unsigned long long>(a) | static_cast<unsigned long long>(b)) >> 32) == 0)
    return static_cast<unsigned>(a) / static_cast<unsigned>(b);
  return a / b;
}

// Token j of the request sees keys [begin, end).
template <int MODE>
__device__ __forceinline__ int key_end(const Request& q, int j, bool clamp = true) {
  if (MODE == kShared || (MODE == kBoth && q.group)) return q.len;
  const int e = q.len - q.n + j + 1;
  return clamp && e < 0 ? 0 : e;
}
__device__ __forceinline__ int key_begin(const PagedArgs& a, int end) {
  return a.window > 0 && end > a.window ? end - static_cast<int>(a.window) : 0;
}

// Row tile rt of a request: rows [rr0, rr1), keys [lo, hi) over all of them,
// key tiles [t0, t0 + nt) (one, with no key, when there is none).
struct RowTile {
  int rr0, rr1;
  int lo, hi;
  int t0, nt;
};

template <int BT, int MODE>
__device__ __forceinline__ RowTile row_tile(const PagedArgs& a, const Request& q, int g, int RT,
                                            int rt) {
  RowTile t;
  t.rr0 = rt * RT;
  const int all = q.n * g;
  t.rr1 = t.rr0 + RT < all ? t.rr0 + RT : all;
  t.hi = key_end<MODE>(q, token_of(t.rr1 - 1, g));
  t.lo = key_begin(a, key_end<MODE>(q, token_of(t.rr0, g)));
  t.t0 = t.lo / BT;
  t.nt = t.hi > t.lo ? (t.hi - 1) / BT + 1 - t.t0 : 1;
  return t;
}

__device__ __forceinline__ int row_tiles(const Request& q, int g, int RT) {
  return (q.n * g + RT - 1) / RT;
}

// The units of a request: its key tiles, and EXTRA for every item, what an
// item's beginning and end cost in tiles.
template <int BT, int EXTRA, int MODE>
__device__ __forceinline__ long long request_units(const PagedArgs& a, int r, int g, int RT) {
  const Request q = load_request<MODE>(a, r);
  const int n = row_tiles(q, g, RT);
  long long u = 0;
  if (q.group) u = n ? static_cast<long long>(n) * (row_tile<BT, MODE>(a, q, g, RT, 0).nt + EXTRA) : 0;
  else
    for (int rt = 0; rt < n; ++rt) u += row_tile<BT, MODE>(a, q, g, RT, rt).nt + EXTRA;
  return u * a.kv_heads;
}

// A walk over a CTA's run of units, item by item.  An item's units are its key
// tiles and, after them, its EXTRA.
template <int BT, int EXTRA, int MODE>
struct Walk {
  int r, rt, kh, nrt;
  Request q;
  RowTile t;
  int k;  // key tile inside the item

  __device__ __forceinline__ void enter(const PagedArgs& a, int g, int RT) {
    q = load_request<MODE>(a, r);
    nrt = row_tiles(q, g, RT);
  }
  // Start at unit x of request r; k may be past the last tile (in the EXTRA).
  __device__ __forceinline__ void start(const PagedArgs& a, int g, int RT, int r_, long long x) {
    r = r_;
    enter(a, g, RT);
    for (rt = 0;; ++rt) {
      t = row_tile<BT, MODE>(a, q, g, RT, rt);
      const long long w = static_cast<long long>(t.nt + EXTRA) * a.kv_heads;
      if (x < w || rt + 1 >= nrt) break;
      x -= w;
    }
    const long long h = divide(x, t.nt + EXTRA);
    kh = static_cast<int>(h);
    k = static_cast<int>(x - h * (t.nt + EXTRA));
  }
  // To the next item; the caller knows that there is one (the bound on r only
  // keeps arrays that change under the kernel from leading it outside).
  __device__ __forceinline__ void next(const PagedArgs& a, int g, int RT) {
    k = 0;
    if (++kh < a.kv_heads) return;
    kh = 0;
    if (++rt >= nrt) {
      rt = 0;
      do {
        if (r + 1 < a.n_req) ++r;
        enter(a, g, RT);
      } while (nrt == 0 && r + 1 < a.n_req);
    }
    t = row_tile<BT, MODE>(a, q, g, RT, rt);
  }
};

// Prefix sum over the requests: every thread of the CTA learns how the total is
// cut into runs of `size` or, the first `longer` of them, size + 1 units, and the
// first unit of the CTA's own as (request, offset).  With fewer units than CTAs
// only `ctas` of them work, so the CTAs of a cut item all hold a part of it.
// `stop`: the abort flag as the CTA's thread 0 set it.  It is read between the
// two barriers here: a wait may raise it as soon as a warp is past the second,
// and warps that read it later could part ways, some leaving while the others
// meet them at a barrier.
struct Run {
  long long first, last;
  long long size;
  int longer, ctas;
  int r;
  long long x;
  bool stop;
};

template <int BT, int EXTRA, int MODE, int kThreads>
__device__ __forceinline__ Run find_run(const PagedArgs& a, int g, int RT, void* scratch,
                                        const volatile int* abort_flag) {
  long long* s_sum = static_cast<long long*>(scratch);  // [kThreads / 32], then the location
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (a.n_req + kThreads - 1) / kThreads;
  const int i0 = tid * per, i1 = i0 + per < a.n_req ? i0 + per : a.n_req;
  long long mine = 0;
  for (int i = i0; i < i1; ++i) mine += request_units<BT, EXTRA, MODE>(a, i, g, RT);
  long long x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(kAll, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  long long before = x - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) before += s_sum[w];
    total += s_sum[w];
  }
  Run run;
  run.stop = *abort_flag != 0;
  run.ctas = total < gridDim.x ? static_cast<int>(total) : static_cast<int>(gridDim.x);
  run.first = run.last = total;
  const int me = static_cast<int>(blockIdx.x);
  if (run.ctas > 0) {
    run.size = divide(total, run.ctas);
    run.longer = static_cast<int>(total - run.size * run.ctas);
    if (me < run.ctas) {
      run.first = run.size * me + (me < run.longer ? me : run.longer);
      run.last = run.first + run.size + (me < run.longer ? 1 : 0);
    }
  }
  if (run.first < run.last && before <= run.first && run.first < before + mine) {
    long long at = run.first - before;
    int i = i0;
    for (; i + 1 < i1; ++i) {
      const long long u = request_units<BT, EXTRA, MODE>(a, i, g, RT);
      if (at < u) break;
      at -= u;
    }
    s_sum[kThreads / 32] = at;
    s_sum[kThreads / 32 + 1] = i;
  }
  __syncthreads();
  run.x = s_sum[kThreads / 32];
  run.r = static_cast<int>(s_sum[kThreads / 32 + 1]);
  return run;
}

// CTA whose run holds unit u.
__device__ __forceinline__ int cta_of(long long u, const Run& run) {
  const long long big = run.longer * (run.size + 1);
  return static_cast<int>(u < big ? divide(u, run.size + 1) : run.longer + divide(u - big, run.size));
}

// The page ids of an item's key tiles, as a producer warp needs them: 32 table
// entries at a time, and the next 32 before they are needed (a lookup per tile
// would put its latency, some 700 cycles, between the requests).  Box p of a
// tile is `rows` keys of one page; lane p gets its page, or -1.
struct PageIds {
  const int* table;
  int begin, end;  // entries that hold the item's pages
  int first;       // entry of lane 0
  int ids, more;

  __device__ __forceinline__ int at(int p) const { return p >= begin && p < end ? table[p] : -1; }
  template <int MODE>
  __device__ __forceinline__ void start(const PagedArgs& a, int r, int lo, int hi, int key0, int lane) {
    table = MODE == kBoth && r >= a.n_own ? a.prefix_table + static_cast<long long>(r - a.n_own) * a.prefix_pages
                                          : a.block_table + static_cast<long long>(r) * a.max_pages;
    end = hi > lo ? ((hi - 1) >> a.page_shift) + 1 : 0;
    begin = lo >> a.page_shift;
    first = key0 >> a.page_shift;
    ids = at(first + lane);
    more = at(first + 32 + lane);
  }
  __device__ __forceinline__ int get(const PagedArgs& a, int key0, int rows, int boxes, int lane) {
    if ((key0 >> a.page_shift) >= first + 32) {
      first += 32;
      ids = more;
      more = at(first + 32 + lane);
    }
    const int p = (key0 + (lane < boxes ? lane : 0) * rows) >> a.page_shift;
    const int page = __shfl_sync(kAll, ids, (p - first) & 31);
    return lane < boxes && page >= 0 && page < a.n_pages ? page : -1;
  }
};

// Opts a kernel into its dynamic shared memory, once per device.
template <typename K>
cudaError_t allow_smem(K* kernel, uint32_t bytes, std::atomic<unsigned long long>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const unsigned long long bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace paged
}  // namespace ra
