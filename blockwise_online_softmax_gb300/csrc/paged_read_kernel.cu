// 8-bit pages read back as dense bf16 rows (include/ra.h, ra_paged_read_fp8):
//   out[row][h][c] = code 2^e, exact in bf16 (fp8.cuh).
//
// Bound by HBM: a byte in and two out per entry.  A warp takes a few rows that
// follow one another.  Lane j finds where row j lies (its request by a search
// in which every step narrows 32-fold, its page from the table); then the lanes
// take eight columns each of the rows' k and v, in order, so that loads and stores
// are whole lines, with kBatch loads of a lane in flight.
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "fp8.cuh"
#include "launch.cuh"
#include "ptx.cuh"
#include "serve_internal.h"

namespace ra {
namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr int kWarps = 8;
constexpr int kBatch = 4;

// The request that row t belongs to: the last i with cu[i] <= t, for a
// nondecreasing cu (for any other some i in range).
__device__ __forceinline__ int request_of(const int* cu, int n_req, long long t, int lane) {
  int lo = 0, n = n_req;
  while (n > 1) {
    const int step = (n + 31) / 32;
    const int at = (lane + 1) * step;
    const int below = __popc(__ballot_sync(kAll, at < n && cu[lo + (at < n ? at : 0)] <= t));
    lo += below * step;
    n = n - below * step < step ? n - below * step : step;
  }
  return lo;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32) paged_read_kernel(const ReadArgs a) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const unsigned row_chunks = static_cast<unsigned>(a.kv_heads) * (D / 8);  // of k, as many of v
  const long long warps = static_cast<long long>(gridDim.x) * kWarps;
  long long first = a.cu[0], end = a.cu[a.n_req];
  if (first < 0) first = 0;
  if (end > a.tokens) end = a.tokens;
  for (long long t0 = first + (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * a.per_warp; t0 < end;
       t0 += warps * a.per_warp) {
    const int rows = static_cast<int>(end - t0 < a.per_warp ? end - t0 : a.per_warp);
    int req = request_of(a.cu, a.n_req, t0, lane);
    // Row t0 + lane: its page (-1: none, zeros) and its row there.
    int page = -1, in = 0;
    if (lane < rows) {
      const long long t = t0 + lane;
      while (req + 1 < a.n_req && a.cu[req + 1] <= t) ++req;
      const long long most = static_cast<long long>(a.max_pages) << a.page_shift;
      long long len = a.lengths[req];
      if (len > most) len = most;
      const long long pos = len - (a.cu[req + 1] - t);
      if (pos >= 0 && pos < len) {
        page = a.block_table[static_cast<long long>(req) * a.max_pages + (pos >> a.page_shift)];
        if (page < 0 || page >= a.n_pages) page = -1;
        in = static_cast<int>(pos & ((1LL << a.page_shift) - 1));
      }
    }
    const unsigned all = static_cast<unsigned>(rows) * 2u * row_chunks;
    for (unsigned x0 = 0; x0 < all; x0 += 32 * kBatch) {
      uint2 raw[kBatch];
      unsigned scale[kBatch];
      uint4* dst[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const unsigned x = x0 + 32 * j + lane;
        const unsigned half = x / row_chunks, c = x - half * row_chunks;  // k of row 0, v of row 0, k of row 1, ...
        const int r = static_cast<int>(half >> 1);
        const int pg = __shfl_sync(kAll, page, r & 31), row = __shfl_sync(kAll, in, r & 31);
        const bool is_v = half & 1;
        raw[j] = make_uint2(0u, 0u);
        scale[j] = 127u;
        dst[j] = nullptr;
        if (x < all) {
          dst[j] = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(is_v ? a.vo : a.ko)) + (t0 + r) * row_chunks + c;
          if (pg >= 0) {
            const uint8_t* codes = (is_v ? a.vc + pg * a.vc_page : a.kc + pg * a.kc_page) +
                                   static_cast<long long>(row) * row_chunks * 8 + c * 8;
            const uint8_t* s = (is_v ? a.vs + pg * a.vs_page : a.ks + pg * a.ks_page) +
                               (static_cast<long long>(c / (D / 8)) << a.page_shift) + row;
            raw[j] = __ldg(reinterpret_cast<const uint2*>(codes));
            scale[j] = __ldg(s);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        if (!dst[j]) continue;
        const float f = scale_of(scale[j]);
        uint32_t w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const uint32_t src = e < 2 ? raw[j].x : raw[j].y;
          const uint32_t h = halves2(static_cast<uint16_t>(src >> 16 * (e & 1)));
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
          w[e] = bf16x2_rn(v.x * f, v.y * f);
        }
        *dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_read(const ReadArgs& args, int d, cudaStream_t st) {
  ReadArgs a = args;
  const long long most = 8LL * sm_count() * kWarps;  // resident warps
  const long long per = (a.tokens + most - 1) / most;
  a.per_warp = static_cast<int>(per < 1 ? 1 : (per > 8 ? 8 : per));
  const long long need = (a.tokens + static_cast<long long>(a.per_warp) * kWarps - 1) / (a.per_warp * kWarps);
  const unsigned grid = static_cast<unsigned>(need < most / kWarps ? need : most / kWarps);
  return launch_early(d == 128 ? paged_read_kernel<128> : paged_read_kernel<64>, dim3(grid), kWarps * 32, 0, st, a);
}

}  // namespace ra
