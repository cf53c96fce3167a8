// Host side of the serving and training calls around the attention kernels
// (declared in include/ra.h): argument checks, scratch and launches.  Host
// code only.
#include <atomic>
#include <cmath>
#include <cstdint>

#include <cuda.h>
#include <cuda_runtime.h>

#include "api_util.h"
#include "ra.h"
#include "serve_internal.h"

using namespace ra::api;

namespace ra {

int sm_count() {
  constexpr int kMax = 64;
  static std::atomic<int> known[kMax];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return 152;
  int n = dev < kMax ? known[dev].load(std::memory_order_relaxed) : 0;
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
  if (dev < kMax) known[dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace ra

namespace {

constexpr long long kMaxInt = 0x7fffffffLL;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int check_words(std::initializer_list<const void*> ps, int bytes) {
  int i = 0;
  for (const void* p : ps) {
    if (!p) return fail(RA_ERR_INVALID, "array argument %d is NULL", i);
    if (!aligned(p, bytes)) return fail(RA_ERR_INVALID, "array argument %d is not %d-byte aligned", i, bytes);
    ++i;
  }
  return RA_OK;
}

int page_shift(int page_size, int* shift) {
  for (int s = 3; s <= 8; ++s)
    if (page_size == 1 << s) {
      *shift = s;
      return RA_OK;
    }
  return fail(RA_ERR_UNSUPPORTED, "page_size=%d (supported: 8, 16, 32, 64, 128, 256)", page_size);
}

// prefix: the table is of prefixes, [n_groups, prefix_max_pages].
int check_table(int n, int pages, int page_size, int* shift, bool prefix = false) {
  const char* n_name = prefix ? "n_groups" : "n_req";
  const char* pages_name = prefix ? "prefix_max_pages" : "max_pages";
  int rc;
  if ((rc = page_shift(page_size, shift)) != RA_OK) return rc;
  if (n < 0) return fail(RA_ERR_INVALID, "%s=%d is negative", n_name, n);
  if (pages < 1) return fail(RA_ERR_INVALID, "%s=%d must be >= 1", pages_name, pages);
  if (static_cast<long long>(n) * pages > kMaxInt)
    return fail(RA_ERR_UNSUPPORTED, "%s * %s = %lld exceeds 2^31 - 1%s", n_name, pages_name,
                static_cast<long long>(n) * pages, prefix ? ", as n_req * max_pages may not" : "");
  if (static_cast<long long>(pages) * page_size > kMaxInt - 255)  // a tile of headroom for the kernels' 32-bit positions
    return fail(RA_ERR_UNSUPPORTED, "%s * page_size = %lld exceeds 2^31 - 256", pages_name,
                static_cast<long long>(pages) * page_size);
  return RA_OK;
}

// The pages of one cache tensor: dense inside a page, 16-byte aligned from
// page to page.
int check_cache(const char* name, long long stride, long long page_elems) {
  if (stride < page_elems)
    return fail(RA_ERR_INVALID, "%s=%lld is less than a page's %lld elements", name, stride, page_elems);
  if (stride % 8 != 0) return fail(RA_ERR_INVALID, "%s=%lld is not a multiple of 8 elements", name, stride);
  return RA_OK;
}

// The same of pages in 8 bits and of their scales: strides in bytes.
int check_cache_fp8(const char* name, long long stride, long long page_bytes) {
  if (stride < page_bytes)
    return fail(RA_ERR_INVALID, "%s=%lld is less than a page's %lld bytes", name, stride, page_bytes);
  if (stride % 16 != 0) return fail(RA_ERR_INVALID, "%s=%lld is not a multiple of 16 bytes", name, stride);
  return RA_OK;
}
int check_pages_fp8(int page_size, int kv_heads, int d, long long k_page, long long v_page, long long k_scale,
                    long long v_scale) {
  if (page_size < 16) return fail(RA_ERR_UNSUPPORTED, "page_size=%d (pages in 8 bits: 16, 32, 64, 128, 256)", page_size);
  const long long rows = static_cast<long long>(page_size) * kv_heads;
  int rc;
  if ((rc = check_cache_fp8("k_page_stride", k_page, rows * d)) != RA_OK) return rc;
  if ((rc = check_cache_fp8("v_page_stride", v_page, rows * d)) != RA_OK) return rc;
  if ((rc = check_cache_fp8("k_scale_stride", k_scale, rows)) != RA_OK) return rc;
  return check_cache_fp8("v_scale_stride", v_scale, rows);
}

int check_stride(const char* name, long long stride, long long row, int dtype) {
  const int unit = dtype == RA_BF16 ? 8 : 4;  // 16 bytes
  if (stride < row) return fail(RA_ERR_INVALID, "%s=%lld is less than a token's %lld elements", name, stride, row);
  if (stride % unit != 0) return fail(RA_ERR_INVALID, "%s=%lld is not a multiple of 16 bytes", name, stride);
  return RA_OK;
}

// 4-D map over the pages of one cache tensor; a box is one KV head's rows of
// a page (64 of a larger one), 64 columns wide, 128-byte swizzle.
int page_map(CUtensorMap* map, const void* base, int n_pages, int page_size, long long page_stride,
             int kv_heads, int d) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(kv_heads),
                              static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(n_pages)};
  const cuuint64_t row = static_cast<cuuint64_t>(kv_heads) * d * 2;
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d) * 2, row, static_cast<cuuint64_t>(page_stride) * 2};
  const cuuint32_t box[4] = {64, 1, static_cast<cuuint32_t>(page_size < 64 ? page_size : 64), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  // L2 fetches of one head's row: 256 bytes at d = 128, 128 at d = 64, where
  // 256 would also fetch the next head's row, which another CTA reads much
  // later (152 requests of 1K keys, d = 64: 421 instead of 321 MB, 77 against
  // 56 us).
  const CUtensorMapL2promotion promote = d == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_256B : CU_TENSOR_MAP_L2_PROMOTION_L2_128B;
  CUresult r = encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides,
                        box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        promote, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled (pages) failed (CUresult %d)", (int)r);
  return RA_OK;
}

// The same of pages in 8 bits: a box is the whole rows of a head, or of two with
// twice the d.  A row is 128 bytes, or 64, and as much is fetched to L2 (see above).
int page_map_fp8(CUtensorMap* map, const void* base, int n_pages, int page_size, long long page_stride,
                 int kv_heads, int d) {
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(kv_heads),
                              static_cast<cuuint64_t>(page_size), static_cast<cuuint64_t>(n_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(kv_heads) * d,
                                 static_cast<cuuint64_t>(page_stride)};
  const int most = ra::paged_fp8_box_rows();
  const cuuint32_t box[4] = {static_cast<cuuint32_t>(d), 1, static_cast<cuuint32_t>(page_size < most ? page_size : most), 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = encode_tiled(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(base), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        d == 128 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_64B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(RA_ERR_CUDA, "cuTensorMapEncodeTiled (8-bit pages) failed (CUresult %d)", (int)r);
  return RA_OK;
}

// What the decode calls share: the checks of everything but the pages, which
// fill a.
int decode_args(ra::PagedArgs& a, const void* q, void* out, float* lse, long long T, int n_req, int n_q, const int* cu_q,
                const int* block_table, int max_pages, const int* lengths, int n_pages, int page_size, long long window,
                int d, int heads, int kv_heads, int dtype, int out_dtype) {
  int rc;
  if ((rc = check_common(d, heads, dtype)) != RA_OK) return rc;
  if ((rc = check_heads(heads, kv_heads)) != RA_OK) return rc;
  if (dtype != RA_BF16) return fail(RA_ERR_UNSUPPORTED, "the paged decode takes bf16 q and pages");
  if (out_dtype != RA_F32 && out_dtype != RA_BF16) return fail(RA_ERR_INVALID, "out_dtype %d is not RA_F32 or RA_BF16", out_dtype);
  if (heads / kv_heads > 128)
    return fail(RA_ERR_UNSUPPORTED, "heads / kv_heads = %d query heads per KV head exceeds 128", heads / kv_heads);
  if ((rc = check_table(n_req, max_pages, page_size, &a.page_shift)) != RA_OK) return rc;
  if (n_pages < 0) return fail(RA_ERR_INVALID, "n_pages=%d is negative", n_pages);
  if (T < 0 || T > kMaxInt) return fail(RA_ERR_INVALID, "T=%lld out of range [0, 2^31 - 1]", T);
  if (n_q < 0) return fail(RA_ERR_INVALID, "n_q=%d is negative", n_q);
  if (!cu_q && static_cast<long long>(n_req) * n_q != T)
    return fail(RA_ERR_INVALID, "T=%lld is not n_req * n_q = %d * %d (and cu_q is NULL)", T, n_req, n_q);
  if (T * heads > kMaxInt - 255) return fail(RA_ERR_UNSUPPORTED, "T * heads = %lld rows exceeds 2^31 - 256", T * heads);
  if (window < 0) return fail(RA_ERR_INVALID, "window=%lld is negative", window);
  a.q = q;
  a.block_table = block_table;
  a.lengths = lengths;
  a.cu_q = cu_q;
  a.out = out;
  a.lse = lse;
  a.T = T;
  a.n_q = !cu_q || n_q > 0 || n_req == 0 ? n_q : (T + n_req - 1) / n_req;
  a.window = window > kMaxInt ? 0 : window;  // wider than any sequence
  a.out_bf16 = out_dtype == RA_BF16;
  a.n_req = n_req;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.item_heads = 1;
  a.scale_log2 = static_cast<float>(1.4426950408889634 / std::sqrt(static_cast<double>(d)));
  a.wait_limit = kWaitLimit;
  return RA_OK;
}

int decode_pointers(const ra::PagedArgs& a, std::initializer_list<const void*> pages) {
  int rc;
  if ((rc = check_ptrs({a.q, a.out, a.lse})) != RA_OK) return rc;
  if (a.n_pages > 0 && (rc = check_ptrs(pages)) != RA_OK) return rc;
  if ((rc = check_words({a.block_table, a.lengths}, 4)) != RA_OK) return rc;
  if (a.cu_q && !aligned(a.cu_q, 4)) return fail(RA_ERR_INVALID, "cu_q is not 4-byte aligned");
  return RA_OK;
}

// Scratch, the decode over the pages and the launch that joins its cut items.
int decode_launch(ra::PagedArgs& a, int d, int rt, const CUtensorMap& tk, const CUtensorMap& tv, bool fp8, void* stream) {
  const int ctas = (rt == 128 ? 1 : 2) * ra::sm_count();
  const size_t rows = static_cast<size_t>(2) * ctas * rt * a.item_heads;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  float* part = nullptr;
  cudaError_t e = scratch_alloc(reinterpret_cast<void**>(&part), rows * (d + 2) * sizeof(float) + ra::paged_cut_bytes(ctas), st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(RA_ERR_ALLOC, "pool allocation of the partial states failed: %s", cudaGetErrorString(e));
  }
  a.po = part;
  a.pm = part + rows * d;
  a.pl = a.pm + rows;
  a.cuts = a.pl + rows;
  {
    TraceScope ts(fp8 ? RA_KERNEL_PAGED_DECODE_FP8 : RA_KERNEL_PAGED_DECODE, st);
    e = fp8 ? ra::launch_paged_fp8(a, d, ctas, rt, tk, tv, st) : ra::launch_paged_decode(a, ra::kPagedPlain, d, ctas, rt, tk, tv, st);
    ts.done(e == cudaSuccess);
  }
  if (e == cudaSuccess) {
    TraceScope ts(RA_KERNEL_PAGED_COMBINE, st);
    e = ra::launch_paged_combine(a, d, ctas, rt, st);
    ts.done(e == cudaSuccess);
  }
  const cudaError_t ef = cudaFreeAsync(part, st);
  if (e != cudaSuccess) return cuda_fail(e, "paged-decode launch");
  return ef == cudaSuccess ? RA_OK : cuda_fail(ef, "cudaFreeAsync");
}

// A prefix call's own rows and, right behind them, its groups' rows.  The second
// launch starts before the first has ended and reads without a wait of its own what
// was there before both: the first lets it start only after waiting for that
// (start_wait in paged_walk.cuh).  So the two are made here and nowhere else.
cudaError_t launch_apart(const ra::PagedArgs& own, int own_tile, int own_ctas, const ra::PagedArgs& shared, int shared_tile,
                         int shared_ctas, int d, const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st) {
  cudaError_t e;
  {
    TraceScope ts(RA_KERNEL_PAGED_DECODE, st);
    e = ra::launch_paged_decode(own, ra::kPagedOwn, d, own_ctas, own_tile, tk, tv, st);
    ts.done(e == cudaSuccess);
  }
  if (e != cudaSuccess || shared.n_groups == 0) return e;
  TraceScope ts(RA_KERNEL_PAGED_PREFIX, st);
  e = ra::launch_paged_decode(shared, ra::kPagedShared, d, shared_ctas, shared_tile, tk, tv, st);
  ts.done(e == cudaSuccess);
  return e;
}

// What the three rope calls share.
int rope_common(ra::RopeArgs& a, long long T, int d, int heads, int kv_heads, int dtype, int rot,
                int interleaved, const void* phases, const void* qw, const void* kw, int w_dtype,
                float eps, float mscale) {
  int rc;
  if ((rc = check_common(d, heads, dtype)) != RA_OK) return rc;
  if ((rc = check_heads(heads, kv_heads)) != RA_OK) return rc;
  if (T < 0 || T > kMaxInt) return fail(RA_ERR_INVALID, "T=%lld out of range [0, 2^31 - 1]", T);
  if (rot < 0 || rot > d || rot % 16 != 0)
    return fail(RA_ERR_UNSUPPORTED, "rot_dim=%d (supported: multiples of 16 up to d=%d)", rot, d);
  if (interleaved != 0 && interleaved != 1) return fail(RA_ERR_INVALID, "interleaved=%d is not 0 or 1", interleaved);
  if (rot > 0 && (rc = check_words({phases}, 8)) != RA_OK) return rc;
  if (w_dtype != RA_F32 && w_dtype != RA_BF16) return fail(RA_ERR_INVALID, "w_dtype %d is not RA_F32 or RA_BF16", w_dtype);
  if ((qw && !aligned16(qw)) || (kw && !aligned16(kw))) return fail(RA_ERR_INVALID, "a norm weight is not 16-byte aligned");
  if (!(eps >= 0.f)) return fail(RA_ERR_INVALID, "eps=%g is not >= 0", eps);
  if (!std::isfinite(mscale)) return fail(RA_ERR_INVALID, "mscale=%g is not finite", mscale);
  a.T = T;
  a.heads = heads;
  a.kv_heads = kv_heads;
  a.rot = rot;
  a.interleaved = interleaved;
  a.phases = static_cast<const unsigned long long*>(phases);
  a.qw = qw;
  a.kw = kw;
  a.w_bf16 = w_dtype == RA_BF16;
  a.eps = eps;
  a.mscale = mscale;
  return RA_OK;
}

int rope_layout(ra::RopeArgs& a, const int* positions, int layout, int P) {
  if (layout != RA_LAYOUT_CONTIGUOUS && layout != RA_LAYOUT_ZIGZAG && layout != RA_LAYOUT_STRIPED)
    return fail(RA_ERR_INVALID, "layout=%d is not a ra_layout value", layout);
  if (P < 1 || P > 65535) return fail(RA_ERR_INVALID, "P=%d out of range [1, 65535]", P);
  if (a.T % P != 0) return fail(RA_ERR_INVALID, "T=%lld is not a multiple of P=%d", a.T, P);
  if (layout == RA_LAYOUT_ZIGZAG && (a.T / P) % 2 != 0)
    return fail(RA_ERR_INVALID, "zigzag layout: the block length T/P=%lld is odd", a.T / P);
  if (positions && !aligned(positions, 4)) return fail(RA_ERR_INVALID, "positions is not 4-byte aligned");
  a.positions = positions;
  a.layout = layout;
  a.P = P;
  a.c = a.T / P;
  return RA_OK;
}

// ra_paged_append and its form in 8 bits: what they share.  The strides of the
// pages have been checked.
int append_common(ra::RopeArgs& a, bool fp8, const void* q, const void* k, const void* v, void* q_out, void* k_cache,
                  void* v_cache, long long T, int d, int heads, int kv_heads, long long q_stride, long long k_stride,
                  long long v_stride, int n_pages, int page_size, long long k_page_stride, long long v_page_stride,
                  const long long* slots, const int* positions, void* stream) {
  int rc;
  const long long krow = static_cast<long long>(kv_heads) * d;
  if ((rc = check_stride("q_stride", q_stride, static_cast<long long>(heads) * d, RA_BF16)) != RA_OK) return rc;
  if ((rc = check_stride("k_stride", k_stride, krow, RA_BF16)) != RA_OK) return rc;
  if ((rc = check_stride("v_stride", v_stride, krow, RA_BF16)) != RA_OK) return rc;
  if (T == 0) return RA_OK;
  if ((rc = check_ptrs({q, k, v, q_out})) != RA_OK) return rc;
  if (n_pages > 0 && (rc = check_ptrs({k_cache, v_cache})) != RA_OK) return rc;
  if (n_pages > 0 && fp8 && (rc = check_ptrs({a.ks, a.vs})) != RA_OK) return rc;
  if ((rc = check_words({slots}, 8)) != RA_OK) return rc;
  if ((rc = check_words({positions}, 4)) != RA_OK) return rc;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_str = q_stride;
  a.k_str = k_stride;
  a.v_str = v_stride;
  a.qo = q_out;
  a.qo_str = static_cast<long long>(heads) * d;
  a.kc = k_cache;
  a.vc = v_cache;
  a.kc_page = k_page_stride;
  a.vc_page = v_page_stride;
  a.n_slots = static_cast<long long>(n_pages) * page_size;
  a.slots = slots;
  a.positions = positions;
  a.layout = RA_LAYOUT_CONTIGUOUS;
  a.P = 1;
  a.c = T;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope ts(fp8 ? RA_KERNEL_PAGED_APPEND_FP8 : RA_KERNEL_PAGED_APPEND, st);
  cudaError_t e = ra::launch_rope_append(a, d, fp8, st);
  ts.done(e == cudaSuccess);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "paged-append launch");
}

}  // namespace

extern "C" {

int ra_paged_extend(const int* lengths, const int* new_tokens, int n_req, int* block_table,
                    int max_pages, const int* free_pages, int free_capacity,
                    const int* free_count, int page_size, long long tokens, int* lengths_out,
                    int* free_count_out, long long* slots, int* positions, int* cu_tokens,
                    int* status, void* stream) {
  ra::ExtendArgs a{};
  int rc = check_table(n_req, max_pages, page_size, &a.page_shift);
  if (rc != RA_OK) return rc;
  if (free_capacity < 0) return fail(RA_ERR_INVALID, "free_capacity=%d is negative", free_capacity);
  if (tokens < 0 || tokens > kMaxInt) return fail(RA_ERR_INVALID, "tokens=%lld out of range [0, 2^31 - 1]", tokens);
  if ((rc = check_words({free_count, free_count_out, cu_tokens, status}, 4)) != RA_OK) return rc;
  if (n_req > 0 && (rc = check_words({lengths, new_tokens, block_table, lengths_out}, 4)) != RA_OK) return rc;
  if (free_capacity > 0 && (rc = check_words({free_pages}, 4)) != RA_OK) return rc;
  if (tokens > 0) {
    if ((rc = check_words({slots}, 8)) != RA_OK) return rc;
    if ((rc = check_words({positions}, 4)) != RA_OK) return rc;
  }
  a.lengths = lengths;
  a.new_tokens = new_tokens;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.lengths_out = lengths_out;
  a.free_count_out = free_count_out;
  a.slots = slots;
  a.positions = positions;
  a.cu_tokens = cu_tokens;
  a.status = status;
  a.tokens = tokens;
  a.n_req = n_req;
  a.max_pages = max_pages;
  a.free_capacity = free_capacity;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (ra::paged_extend_needs_scratch(a)) {
    e = scratch_alloc(reinterpret_cast<void**>(&a.first_page), (static_cast<size_t>(n_req) + 2) * sizeof(int), st);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(RA_ERR_ALLOC, "pool allocation of the page sums failed: %s", cudaGetErrorString(e));
    }
  }
  {
    TraceScope ts(RA_KERNEL_PAGED_EXTEND, st);
    e = ra::launch_paged_extend(a, st);
    ts.done(e == cudaSuccess);
  }
  if (a.first_page && e == cudaSuccess) {
    TraceScope ts(RA_KERNEL_PAGED_EXTEND, st);
    e = ra::launch_paged_extend_tokens(a, st);
    ts.done(e == cudaSuccess);
  }
  const cudaError_t ef = a.first_page ? cudaFreeAsync(a.first_page, st) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "paged-extend launch");
  return ef == cudaSuccess ? RA_OK : cuda_fail(ef, "cudaFreeAsync");
}

int ra_paged_release(const int* lengths, const int* finished, int n_req, const int* block_table,
                     int max_pages, int* free_pages, int free_capacity, const int* free_count,
                     int page_size, int* lengths_out, int* free_count_out, void* stream) {
  ra::ReleaseArgs a{};
  int rc = check_table(n_req, max_pages, page_size, &a.page_shift);
  if (rc != RA_OK) return rc;
  if (free_capacity < 0) return fail(RA_ERR_INVALID, "free_capacity=%d is negative", free_capacity);
  if ((rc = check_words({free_count, free_count_out}, 4)) != RA_OK) return rc;
  if (n_req > 0 && (rc = check_words({lengths, finished, block_table, lengths_out}, 4)) != RA_OK) return rc;
  if (free_capacity > 0 && (rc = check_words({free_pages}, 4)) != RA_OK) return rc;
  a.lengths = lengths;
  a.finished = finished;
  a.block_table = block_table;
  a.free_pages = free_pages;
  a.free_count = free_count;
  a.lengths_out = lengths_out;
  a.free_count_out = free_count_out;
  a.n_req = n_req;
  a.max_pages = max_pages;
  a.free_capacity = free_capacity;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (ra::paged_release_needs_scratch(a)) {
    e = scratch_alloc(reinterpret_cast<void**>(&a.first_page), (static_cast<size_t>(n_req) + 2) * sizeof(int), st);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(RA_ERR_ALLOC, "pool allocation of the page sums failed: %s", cudaGetErrorString(e));
    }
  }
  {
    TraceScope ts(RA_KERNEL_PAGED_RELEASE, st);
    e = ra::launch_paged_release(a, st);
    ts.done(e == cudaSuccess);
  }
  if (a.first_page && e == cudaSuccess) {
    TraceScope ts(RA_KERNEL_PAGED_RELEASE, st);
    e = ra::launch_paged_release_pages(a, st);
    ts.done(e == cudaSuccess);
  }
  const cudaError_t ef = a.first_page ? cudaFreeAsync(a.first_page, st) : cudaSuccess;
  if (e != cudaSuccess) return cuda_fail(e, "paged-release launch");
  return ef == cudaSuccess ? RA_OK : cuda_fail(ef, "cudaFreeAsync");
}

int ra_qk_norm_rope(const void* q, const void* k, void* q_out, void* k_out, long long T, int d,
                    int heads, int kv_heads, long long q_stride, long long k_stride,
                    const int* positions, int layout, int P, int rot_dim, int interleaved,
                    const void* phases, float mscale, const void* q_weight, const void* k_weight,
                    int w_dtype, float eps, int dtype, void* stream) {
  ra::RopeArgs a{};
  int rc = rope_common(a, T, d, heads, kv_heads, dtype, rot_dim, interleaved, phases, q_weight,
                       k_weight, w_dtype, eps, mscale);
  if (rc != RA_OK) return rc;
  if ((rc = rope_layout(a, positions, layout, P)) != RA_OK) return rc;
  if ((rc = check_stride("q_stride", q_stride, static_cast<long long>(heads) * d, dtype)) != RA_OK) return rc;
  if ((rc = check_stride("k_stride", k_stride, static_cast<long long>(kv_heads) * d, dtype)) != RA_OK) return rc;
  if (T == 0) return RA_OK;
  if ((rc = check_ptrs({q, k, q_out, k_out})) != RA_OK) return rc;
  a.q = q;
  a.k = k;
  a.q_str = q_stride;
  a.k_str = k_stride;
  a.qo = q_out;
  a.ko = k_out;
  a.qo_str = static_cast<long long>(heads) * d;
  a.ko_str = static_cast<long long>(kv_heads) * d;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope ts(RA_KERNEL_QK_NORM_ROPE, st);
  cudaError_t e = ra::launch_rope_forward(a, d, dtype == RA_BF16, st);
  ts.done(e == cudaSuccess);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "qk-norm-rope launch");
}

int ra_qk_norm_rope_backward(const void* q, const void* k, const float* dq_out,
                             const float* dk_out, void* dq, void* dk, float* dq_weight,
                             float* dk_weight, long long T, int d, int heads, int kv_heads,
                             long long q_stride, long long k_stride, long long dq_stride,
                             long long dk_stride, const int* positions, int layout, int P,
                             int rot_dim, int interleaved, const void* phases, float mscale,
                             const void* q_weight, const void* k_weight, int w_dtype, float eps,
                             int dtype, void* stream) {
  ra::RopeArgs a{};
  int rc = rope_common(a, T, d, heads, kv_heads, dtype, rot_dim, interleaved, phases, q_weight,
                       k_weight, w_dtype, eps, mscale);
  if (rc != RA_OK) return rc;
  if ((rc = rope_layout(a, positions, layout, P)) != RA_OK) return rc;
  const long long qrow = static_cast<long long>(heads) * d, krow = static_cast<long long>(kv_heads) * d;
  if ((rc = check_stride("q_stride", q_stride, qrow, dtype)) != RA_OK) return rc;
  if ((rc = check_stride("k_stride", k_stride, krow, dtype)) != RA_OK) return rc;
  if ((rc = check_stride("dq_stride", dq_stride, qrow, dtype)) != RA_OK) return rc;
  if ((rc = check_stride("dk_stride", dk_stride, krow, dtype)) != RA_OK) return rc;
  if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr))
    return fail(RA_ERR_INVALID, "a norm weight and its gradient are given together or not at all");
  if ((dq_weight && !aligned16(dq_weight)) || (dk_weight && !aligned16(dk_weight)))
    return fail(RA_ERR_INVALID, "a weight gradient is not 16-byte aligned");
  if (T > 0 && (rc = check_ptrs({q, k, dq_out, dk_out, dq, dk})) != RA_OK) return rc;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (T == 0) {  // no row: the weight gradients are zero
    if (dq_weight && (e = cudaMemsetAsync(dq_weight, 0, d * sizeof(float), st)) != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    if (dk_weight && (e = cudaMemsetAsync(dk_weight, 0, d * sizeof(float), st)) != cudaSuccess) return cuda_fail(e, "cudaMemsetAsync");
    return RA_OK;
  }
  a.q = q;
  a.k = k;
  a.q_str = q_stride;
  a.k_str = k_stride;
  a.qo = dq;
  a.ko = dk;
  a.qo_str = dq_stride;
  a.ko_str = dk_stride;
  a.dqo = dq_out;
  a.dko = dk_out;
  a.dqw = dq_weight;
  a.dkw = dk_weight;
  const int ctas = ra::rope_grad_ctas(a, d);
  if (dq_weight || dk_weight) {
    e = scratch_alloc(reinterpret_cast<void**>(&a.dw), static_cast<size_t>(ctas) * 2 * d * sizeof(float2), st);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return fail(RA_ERR_ALLOC, "pool allocation of the partial weight gradients failed: %s", cudaGetErrorString(e));
    }
  }
  {
    TraceScope ts(RA_KERNEL_QK_NORM_ROPE_BWD, st);
    e = ra::launch_rope_backward(a, ctas, d, dtype == RA_BF16, st);
    ts.done(e == cudaSuccess);
  }
  if (a.dw) {
    if (e == cudaSuccess) {
      TraceScope ts(RA_KERNEL_QK_NORM_WEIGHT_GRAD, st);
      e = ra::launch_rope_weight_grad(a, ctas, d, st);
      ts.done(e == cudaSuccess);
    }
    const cudaError_t ef = cudaFreeAsync(a.dw, st);
    if (e == cudaSuccess && ef != cudaSuccess) return cuda_fail(ef, "cudaFreeAsync");
  }
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "qk-norm-rope backward launch");
}

int ra_paged_append(const void* q, const void* k, const void* v, void* q_out, void* k_cache,
                    void* v_cache, long long T, int d, int heads, int kv_heads,
                    long long q_stride, long long k_stride, long long v_stride, int n_pages,
                    int page_size, long long k_page_stride, long long v_page_stride,
                    const long long* slots, const int* positions, int rot_dim, int interleaved,
                    const void* phases, float mscale, const void* q_weight, const void* k_weight,
                    int w_dtype, float eps, int dtype, void* stream) {
  ra::RopeArgs a{};
  int rc = rope_common(a, T, d, heads, kv_heads, dtype, rot_dim, interleaved, phases, q_weight,
                       k_weight, w_dtype, eps, mscale);
  if (rc != RA_OK) return rc;
  if (dtype != RA_BF16) return fail(RA_ERR_UNSUPPORTED, "the paged cache takes bf16 q, k, v");
  if ((rc = page_shift(page_size, &a.page_shift)) != RA_OK) return rc;
  if (n_pages < 0) return fail(RA_ERR_INVALID, "n_pages=%d is negative", n_pages);
  const long long page_elems = static_cast<long long>(kv_heads) * d * page_size;
  if ((rc = check_cache("k_page_stride", k_page_stride, page_elems)) != RA_OK) return rc;
  if ((rc = check_cache("v_page_stride", v_page_stride, page_elems)) != RA_OK) return rc;
  return append_common(a, false, q, k, v, q_out, k_cache, v_cache, T, d, heads, kv_heads, q_stride, k_stride, v_stride,
                       n_pages, page_size, k_page_stride, v_page_stride, slots, positions, stream);
}

int ra_paged_append_fp8(const void* q, const void* k, const void* v, void* q_out, void* k_cache,
                        void* v_cache, void* k_scale, void* v_scale, long long T, int d, int heads,
                        int kv_heads, long long q_stride, long long k_stride, long long v_stride,
                        int n_pages, int page_size, long long k_page_stride,
                        long long v_page_stride, long long k_scale_stride,
                        long long v_scale_stride, const long long* slots, const int* positions,
                        int rot_dim, int interleaved, const void* phases, float mscale,
                        const void* q_weight, const void* k_weight, int w_dtype, float eps,
                        int dtype, void* stream) {
  ra::RopeArgs a{};
  int rc = rope_common(a, T, d, heads, kv_heads, dtype, rot_dim, interleaved, phases, q_weight,
                       k_weight, w_dtype, eps, mscale);
  if (rc != RA_OK) return rc;
  if (dtype != RA_BF16) return fail(RA_ERR_UNSUPPORTED, "the paged cache takes bf16 q, k, v");
  if ((rc = page_shift(page_size, &a.page_shift)) != RA_OK) return rc;
  if (n_pages < 0) return fail(RA_ERR_INVALID, "n_pages=%d is negative", n_pages);
  if ((rc = check_pages_fp8(page_size, kv_heads, d, k_page_stride, v_page_stride, k_scale_stride, v_scale_stride)) != RA_OK) return rc;
  a.ks = k_scale;
  a.vs = v_scale;
  a.ks_page = k_scale_stride;
  a.vs_page = v_scale_stride;
  return append_common(a, true, q, k, v, q_out, k_cache, v_cache, T, d, heads, kv_heads, q_stride, k_stride, v_stride,
                       n_pages, page_size, k_page_stride, v_page_stride, slots, positions, stream);
}

int ra_paged_read_fp8(const void* k_cache, const void* v_cache, const void* k_scale,
                      const void* v_scale, void* k_out, void* v_out, long long tokens, int n_req,
                      const int* cu_k, const int* block_table, int max_pages, const int* lengths,
                      int n_pages, int page_size, long long k_page_stride, long long v_page_stride,
                      long long k_scale_stride, long long v_scale_stride, int d, int kv_heads,
                      void* stream) {
  ra::ReadArgs a{};
  int rc;
  if ((rc = check_common(d, kv_heads, RA_BF16)) != RA_OK) return rc;
  if ((rc = check_table(n_req, max_pages, page_size, &a.page_shift)) != RA_OK) return rc;
  if (n_pages < 0) return fail(RA_ERR_INVALID, "n_pages=%d is negative", n_pages);
  if (tokens < 0 || tokens > kMaxInt) return fail(RA_ERR_INVALID, "tokens=%lld out of range [0, 2^31 - 1]", tokens);
  if ((rc = check_pages_fp8(page_size, kv_heads, d, k_page_stride, v_page_stride, k_scale_stride, v_scale_stride)) != RA_OK) return rc;
  if (tokens == 0 || n_req == 0) return RA_OK;
  if ((rc = check_ptrs({k_out, v_out})) != RA_OK) return rc;
  if (n_pages > 0 && (rc = check_ptrs({k_cache, v_cache, k_scale, v_scale})) != RA_OK) return rc;
  if ((rc = check_words({cu_k, block_table, lengths}, 4)) != RA_OK) return rc;
  a.kc = static_cast<const uint8_t*>(k_cache);
  a.vc = static_cast<const uint8_t*>(v_cache);
  a.ks = static_cast<const uint8_t*>(k_scale);
  a.vs = static_cast<const uint8_t*>(v_scale);
  a.kc_page = k_page_stride;
  a.vc_page = v_page_stride;
  a.ks_page = k_scale_stride;
  a.vs_page = v_scale_stride;
  a.ko = k_out;
  a.vo = v_out;
  a.block_table = block_table;
  a.lengths = lengths;
  a.cu = cu_k;
  a.tokens = tokens;
  a.n_req = n_req;
  a.max_pages = max_pages;
  a.n_pages = n_pages;
  a.kv_heads = kv_heads;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  TraceScope ts(RA_KERNEL_PAGED_READ_FP8, st);
  cudaError_t e = ra::launch_paged_read(a, d, st);
  ts.done(e == cudaSuccess);
  return e == cudaSuccess ? RA_OK : cuda_fail(e, "paged-read launch");
}

int ra_paged_decode(const void* q, const void* k_cache, const void* v_cache, void* out, float* lse,
                    long long T, int n_req, int n_q, const int* cu_q, const int* block_table,
                    int max_pages, const int* lengths, int n_pages, int page_size,
                    long long k_page_stride, long long v_page_stride, long long window, int d,
                    int heads, int kv_heads, int dtype, int out_dtype, void* stream) {
  ra::PagedArgs a{};
  int rc = decode_args(a, q, out, lse, T, n_req, n_q, cu_q, block_table, max_pages, lengths, n_pages, page_size, window,
                       d, heads, kv_heads, dtype, out_dtype);
  if (rc != RA_OK) return rc;
  const long long page_elems = static_cast<long long>(page_size) * kv_heads * d;
  if ((rc = check_cache("k_page_stride", k_page_stride, page_elems)) != RA_OK) return rc;
  if ((rc = check_cache("v_page_stride", v_page_stride, page_elems)) != RA_OK) return rc;
  if (T == 0 || n_req == 0) return RA_OK;
  if ((rc = decode_pointers(a, {k_cache, v_cache})) != RA_OK) return rc;
  if ((rc = get_encoder()) != RA_OK) return rc;
  CUtensorMap tk, tv;
  // Without pages no load is ever issued; the maps still need an address.
  if ((rc = page_map(&tk, n_pages ? k_cache : q, n_pages ? n_pages : 1, page_size, k_page_stride, kv_heads, d)) != RA_OK) return rc;
  if ((rc = page_map(&tv, n_pages ? v_cache : q, n_pages ? n_pages : 1, page_size, v_page_stride, kv_heads, d)) != RA_OK) return rc;
  return decode_launch(a, d, ra::paged_row_tile(a, d), tk, tv, false, stream);
}

int ra_paged_decode_prefix(const void* q, const void* k_cache, const void* v_cache, void* out,
                           float* lse, long long T, int n_groups, const int* cu_req,
                           const int* prefix_table, int prefix_max_pages,
                           const int* prefix_lengths, int n_req, int n_q, const int* cu_q,
                           const int* block_table, int max_pages, const int* lengths, int n_pages,
                           int page_size, long long k_page_stride, long long v_page_stride, int d,
                           int heads, int kv_heads, int dtype, int out_dtype, void* stream) {
  ra::PagedArgs own{};
  int rc = decode_args(own, q, out, lse, T, n_req, n_q, cu_q, block_table, max_pages, lengths, n_pages, page_size, 0,
                       d, heads, kv_heads, dtype, out_dtype);
  if (rc != RA_OK) return rc;
  int shift = 0;
  if ((rc = check_table(n_groups, prefix_max_pages, page_size, &shift, true)) != RA_OK) return rc;
  const long long page_elems = static_cast<long long>(page_size) * kv_heads * d;
  if ((rc = check_cache("k_page_stride", k_page_stride, page_elems)) != RA_OK) return rc;
  if ((rc = check_cache("v_page_stride", v_page_stride, page_elems)) != RA_OK) return rc;
  if (T == 0 || n_req == 0) return RA_OK;
  if ((rc = decode_pointers(own, {k_cache, v_cache})) != RA_OK) return rc;
  if (n_groups > 0 && (rc = check_words({cu_req, prefix_table, prefix_lengths}, 4)) != RA_OK) return rc;
  if ((rc = get_encoder()) != RA_OK) return rc;
  CUtensorMap tk, tv;
  if ((rc = page_map(&tk, n_pages ? k_cache : q, n_pages ? n_pages : 1, page_size, k_page_stride, kv_heads, d)) != RA_OK) return rc;
  if ((rc = page_map(&tv, n_pages ? v_cache : q, n_pages ? n_pages : 1, page_size, v_page_stride, kv_heads, d)) != RA_OK) return rc;
  own.cu_req = cu_req;
  own.n_groups = n_groups;
  const long long rows = T * heads;
  ra::PagedArgs group = own;  // as if a group were a request
  const long long expected = own.n_q * n_req < T ? own.n_q * n_req : T;  // rows; without a word of the caller's T
  group.n_q = n_groups ? (expected + n_groups - 1) / n_groups : 1;
  group.n_req = n_groups;
  group.max_pages = prefix_max_pages;
  const int own_tile = ra::paged_row_tile(own, d), group_tile = ra::paged_row_tile(group, d);
  const bool both = own_tile <= 16 && ra::paged_prefix_both(group) && 2 * rows <= kMaxInt &&
                    static_cast<long long>(n_req) + n_groups <= kMaxInt;
  // Launches: one of both, or the own and then the shared one, whose requests are
  // the groups.
  ra::PagedArgs shared = own;
  int shared_tile = 128;
  if (both) {
    own.n_req = n_req + n_groups;
    own.n_own = n_req;
    own.prefix_table = prefix_table;
    own.prefix_lengths = prefix_lengths;
    own.prefix_pages = prefix_max_pages;
    shared_tile = own_tile > group_tile ? own_tile : (group_tile < 16 ? group_tile : 16);
  } else {
    shared.n_own = n_req;
    shared.n_req = n_groups;
    shared.block_table = prefix_table;
    shared.max_pages = prefix_max_pages;
    shared.lengths = prefix_lengths;
  }
  const int tile = both ? shared_tile : own_tile;
  // Scratch of a launch: the states of its cut items and of all rows (of both, own
  // ones first), and as many records.
  auto ctas_of = [](int t) { return (t == 128 ? 1 : 2) * ra::sm_count(); };
  auto size_of = [&](ra::PagedArgs& a, int t, long long n) {
    a.whole = 2LL * ctas_of(t) * t;
    const size_t bytes = static_cast<size_t>(a.whole + n) * (d + 2) * sizeof(float) + n * sizeof(int2);
    return (bytes + 255) / 256 * 256;
  };
  const long long own_rows = both ? 2 * rows : rows;
  const size_t own_bytes = size_of(own, tile, own_rows), shared_bytes = both ? 0 : size_of(shared, shared_tile, rows);
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  char* scratch = nullptr;
  cudaError_t e = scratch_alloc(reinterpret_cast<void**>(&scratch), own_bytes + shared_bytes, st);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return fail(RA_ERR_ALLOC, "pool allocation of the partial states failed: %s", cudaGetErrorString(e));
  }
  auto place = [&](ra::PagedArgs& a, char* at, long long n) {
    a.po = reinterpret_cast<float*>(at);
    a.pm = a.po + (a.whole + n) * d;
    a.pl = a.pm + (a.whole + n);
    a.parts = reinterpret_cast<int2*>(a.pl + (a.whole + n));
  };
  place(own, scratch, own_rows);
  if (both) {
    shared = own;
    shared.whole += rows;
    shared.parts += rows;
  } else {
    place(shared, scratch + own_bytes, rows);
  }
  if (both) {
    TraceScope ts(RA_KERNEL_PAGED_PREFIX, st);
    e = ra::launch_paged_decode(own, ra::kPagedBoth, d, ctas_of(tile), tile, tk, tv, st);
    ts.done(e == cudaSuccess);
  } else {
    e = launch_apart(own, tile, ctas_of(tile), shared, shared_tile, ctas_of(shared_tile), d, tk, tv, st);
  }
  if (e == cudaSuccess) {
    own.n_req = n_req;
    TraceScope ts(RA_KERNEL_PAGED_COMBINE, st);
    e = ra::launch_paged_join(own, shared, d, tile, shared_tile, st);
    ts.done(e == cudaSuccess);
  }
  const cudaError_t ef = cudaFreeAsync(scratch, st);
  if (e != cudaSuccess) return cuda_fail(e, "paged-prefix launch");
  return ef == cudaSuccess ? RA_OK : cuda_fail(ef, "cudaFreeAsync");
}

int ra_paged_decode_fp8(const void* q, const void* k_cache, const void* v_cache, const void* k_scale,
                        const void* v_scale, void* out, float* lse, long long T, int n_req, int n_q,
                        const int* cu_q, const int* block_table, int max_pages, const int* lengths,
                        int n_pages, int page_size, long long k_page_stride,
                        long long v_page_stride, long long k_scale_stride,
                        long long v_scale_stride, long long window, int d, int heads, int kv_heads,
                        int dtype, int out_dtype, void* stream) {
  ra::PagedArgs a{};
  int rc = decode_args(a, q, out, lse, T, n_req, n_q, cu_q, block_table, max_pages, lengths, n_pages, page_size, window,
                       d, heads, kv_heads, dtype, out_dtype);
  if (rc != RA_OK) return rc;
  if ((rc = check_pages_fp8(page_size, kv_heads, d, k_page_stride, v_page_stride, k_scale_stride, v_scale_stride)) != RA_OK) return rc;
  if (T == 0 || n_req == 0) return RA_OK;
  if ((rc = decode_pointers(a, {k_cache, v_cache, k_scale, v_scale})) != RA_OK) return rc;
  a.ks = static_cast<const uint8_t*>(k_scale);
  a.vs = static_cast<const uint8_t*>(v_scale);
  a.ks_page = k_scale_stride;
  a.vs_page = v_scale_stride;
  if ((rc = get_encoder()) != RA_OK) return rc;
  CUtensorMap tk, tv;
  const int row_tile = ra::paged_fp8_row_tile(a);
  a.item_heads = ra::paged_fp8_item_heads(a, d, row_tile);
  a.kv_heads = kv_heads / a.item_heads;
  if ((rc = page_map_fp8(&tk, n_pages ? k_cache : q, n_pages ? n_pages : 1, page_size, k_page_stride, a.kv_heads, d * a.item_heads)) != RA_OK) return rc;
  if ((rc = page_map_fp8(&tv, n_pages ? v_cache : q, n_pages ? n_pages : 1, page_size, v_page_stride, a.kv_heads, d * a.item_heads)) != RA_OK) return rc;
  return decode_launch(a, d, row_tile, tk, tv, true, stream);
}

}  // extern "C"
