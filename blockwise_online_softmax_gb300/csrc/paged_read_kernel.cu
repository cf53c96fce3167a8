// 8-bit pages read back as dense bf16 rows (include/ra.h, ra_paged_read_fp8):
//   out[row][h][c] = code 2^e, exact in bf16 (fp8.cuh).
//
// Bound by HBM: a byte in and two out per entry.  A warp takes a few rows that
// follow one another.  Lane j finds where row j lies (its request by a search
// in which every step narrows 32-fold, its page from the table); then the lanes
// take sixteen columns each of the rows' k, then of their v, in order, with
// kBatch loads of a lane in flight, and store 32 bytes at once where the output is
// aligned to them.  348K tokens of 8 heads, d = 128: 358 us, 6.2 TB/s (0.91 of the
// copy rate); as two 16-byte stores 382, eight columns a lane 368; 6000 tokens 7.1,
// 10.2 and 7.5 us (floor 5.4), and 8.0 where other work comes between the calls.
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
constexpr int CH = 16;  // codes of a lane

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

// The same for one lane, from a request lo with cu[lo] <= t on: mostly lo itself, else
// by steps that double and then halve.  (Where few of many requests have rows, one by
// one were as many loads in turn as there are idle requests: two of 5000, 30K tokens
// each, 365 us against 58.)
__device__ __forceinline__ int request_from(const int* cu, int n_req, int lo, long long t) {
  auto below = [&](unsigned step) { return step < static_cast<unsigned>(n_req - lo) && cu[lo + step] <= t; };
  unsigned step = 1;
  for (; below(step); step *= 2) lo += static_cast<int>(step);
  for (step /= 2; step > 0; step /= 2)
    if (below(step)) lo += static_cast<int>(step);
  return lo;
}

template <int D>
__global__ void __launch_bounds__(kWarps * 32, 4) paged_read_kernel(const ReadArgs a) {
  let_next_start();
  wait_for_previous();
  const int lane = threadIdx.x & 31;
  const unsigned row_chunks = static_cast<unsigned>(a.kv_heads) * (D / CH);  // of a row of k, or of v
  const unsigned step_rows = 32 / row_chunks, step_chunks = 32 - step_rows * row_chunks;
  const long long warps = static_cast<long long>(gridDim.x) * kWarps;
  long long first = a.cu[0], end = a.cu[a.n_req];
  if (first < 0) first = 0;
  if (end > a.tokens) end = a.tokens;
  for (long long t0 = first + (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * a.per_warp; t0 < end;
       t0 += warps * a.per_warp) {
    const int rows = static_cast<int>(end - t0 < a.per_warp ? end - t0 : a.per_warp);
    const int req0 = request_of(a.cu, a.n_req, t0, lane);
    // Row t0 + lane: its page (-1: none, zeros) and its row there.
    int page = -1, in = 0;
    if (lane < rows) {
      const long long t = t0 + lane;
      const int req = request_from(a.cu, a.n_req, req0, t);
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
    // Where that row is in the four tensors.
    const long long k_at = page * a.kc_page + static_cast<long long>(in) * row_chunks * CH;
    const long long v_at = page * a.vc_page + static_cast<long long>(in) * row_chunks * CH;
    const long long ks_at = page * a.ks_page + in, vs_at = page * a.vs_page + in;
    const unsigned all = static_cast<unsigned>(rows) * row_chunks;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint8_t* const codes = side ? a.vc : a.kc;
      const uint8_t* const scales = side ? a.vs : a.ks;
      __nv_bfloat16* const out = static_cast<__nv_bfloat16*>(side ? a.vo : a.ko) + t0 * row_chunks * CH;
      unsigned r = lane / row_chunks, c = lane - r * row_chunks;
      for (unsigned x0 = lane; x0 < all + lane; x0 += 32 * kBatch) {
        uint4 raw[kBatch];
        unsigned scale[kBatch];
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const long long at = __shfl_sync(kAll, side ? v_at : k_at, r & 31);
          const long long s_at = __shfl_sync(kAll, side ? vs_at : ks_at, r & 31);
          raw[j] = make_uint4(0u, 0u, 0u, 0u);
          scale[j] = 127u;
          if (x0 + 32 * j < all && at >= 0) {
            raw[j] = __ldg(reinterpret_cast<const uint4*>(codes + at + c * CH));
            scale[j] = __ldg(scales + s_at + (static_cast<long long>(c / (D / CH)) << a.page_shift));
          }
          r += step_rows;
          c += step_chunks;
          if (c >= row_chunks) {
            c -= row_chunks;
            ++r;
          }
        }
#pragma unroll
        for (int j = 0; j < kBatch; ++j) {
          const unsigned x = x0 + 32 * j;
          if (x >= all) break;
          const float f = scale_of(scale[j]);
          const uint64_t f2 = f2pack(f, f);
          uint32_t w[CH / 2];
#pragma unroll
          for (int e = 0; e < CH / 2; ++e) {
            const uint32_t h = halves2(static_cast<uint16_t>((e < 2 ? raw[j].x : e < 4 ? raw[j].y : e < 6 ? raw[j].z : raw[j].w) >> 16 * (e & 1)));
            const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
            float lo, hi;
            f2unpack(fmul2(f2pack(v.x, v.y), f2), lo, hi);
            w[e] = bf16x2_rn(lo, hi);
          }
          __nv_bfloat16* const dst = out + static_cast<long long>(x) * CH;
          if (a.wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]),
                         "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                         : "memory");
          } else {
            reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
            reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
          }
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_paged_read(const ReadArgs& args, int d, cudaStream_t st) {
  ReadArgs a = args;
  a.wide = ((reinterpret_cast<uintptr_t>(a.ko) | reinterpret_cast<uintptr_t>(a.vo)) & 31) == 0;
  const long long most = 8LL * sm_count() * kWarps;  // two turns of what is resident: 7.1 us against 7.7 for 6000 rows
  const long long per = (a.tokens + most - 1) / most;
  // At most 512 chunks of each side, or a row for each lane: with 8 rows of one head, d =
  // 64, a lane had one load a side (970K tokens 67 -> 46 us; four heads 334 -> 327).
  const int chunks = a.kv_heads * (d / CH), cap = chunks >= 64 ? 8 : (chunks > 16 ? 512 / chunks : 32);
  a.per_warp = static_cast<int>(per < 1 ? 1 : (per > cap ? cap : per));
  const long long need = (a.tokens + static_cast<long long>(a.per_warp) * kWarps - 1) / (a.per_warp * kWarps);
  const unsigned grid = static_cast<unsigned>(need < most / kWarps ? need : most / kWarps);
  return launch_early(d == 128 ? paged_read_kernel<128> : paged_read_kernel<64>, dim3(grid), kWarps * 32, 0, st, a);
}

}  // namespace ra
