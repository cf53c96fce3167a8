// Internal interface of the serving and training operators around the
// attention kernels (page bookkeeping, q/k norm with rotary positions,
// paged decode) between serve_api.cu and the kernel units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ra_internal.h"

namespace ra {

// SMs of the current device (looked up once per device).
int sm_count();

// ------------------------------------------------------------------ pages
struct ExtendArgs {
  const int* lengths;     // [n_req] tokens cached before
  const int* new_tokens;  // [n_req]
  int* block_table;       // [n_req, max_pages]
  const int* free_pages;  // [free_capacity], a stack: entries [0, *free_count)
  const int* free_count;
  int* lengths_out;
  int* free_count_out;
  long long* slots;       // [tokens]
  int* positions;         // [tokens]
  int* cu_tokens;         // [n_req + 1]
  int* status;            // [3]
  long long tokens;
  int n_req;
  int max_pages;
  int free_capacity;
  int page_shift;         // log2 of the page size
  // Scratch of a large step, else null: per request the new pages of the
  // requests before it, then the stack's count before the step.
  int* first_page;        // [n_req + 1]
};
bool paged_extend_needs_scratch(const ExtendArgs& a);
cudaError_t launch_paged_extend(const ExtendArgs& a, cudaStream_t st);
// The second launch of a large step (with scratch).
cudaError_t launch_paged_extend_tokens(const ExtendArgs& a, cudaStream_t st);

struct ReleaseArgs {
  const int* lengths;
  const int* finished;
  const int* block_table;
  int* free_pages;
  const int* free_count;
  int* lengths_out;
  int* free_count_out;
  int n_req;
  int max_pages;
  int free_capacity;
  int page_shift;
  int* first_page;  // [n_req + 2], or null: as above, the total, the count before
};
bool paged_release_needs_scratch(const ReleaseArgs& a);
cudaError_t launch_paged_release(const ReleaseArgs& a, cudaStream_t st);
cudaError_t launch_paged_release_pages(const ReleaseArgs& a, cudaStream_t st);

// ------------------------------------------------------------------ q/k norm and rotary positions
struct RopeArgs {
  const void* q;  // [T, heads, d], tokens q_str elements apart
  const void* k;  // [T, kv_heads, d]
  const void* v;  // append: [T, kv_heads, d]
  long long q_str, k_str, v_str;
  void* qo;       // forward: rotated q; backward: dq
  void* ko;       // forward: rotated k; backward: dk
  long long qo_str, ko_str;
  const float* dqo;  // backward: gradients of the outputs, dense fp32
  const float* dko;
  void* kc;          // append: pages [n_pages, page_size, kv_heads, d] bf16
  void* vc;
  long long kc_page, vc_page;  // elements from page to page
  void* ks;          // append in 8 bits: scales [n_pages, kv_heads, page_size], e8m0
  void* vs;
  long long ks_page, vs_page;
  long long n_slots;           // n_pages * page_size
  int page_shift;
  const long long* slots;
  const int* positions;  // null: by layout
  int layout;
  int P;
  long long c;           // T / P
  long long T;
  int heads;
  int kv_heads;
  int rot;               // rotated columns (a multiple of 16, 0: none)
  int interleaved;
  const unsigned long long* phases;  // [rot / 2] turns per position, units of 2^-64
  const void* qw;        // [d] weights of the norm; null: no norm
  const void* kw;
  int w_bf16;
  float eps;
  float mscale;
  float2* dw;            // backward: partial weight gradients [rope_grad_ctas][2][d], in two words
  float* dqw;            // [d] or null
  float* dkw;
  // Set by the launcher: a warp takes a token as a whole, from token `whole` on
  // one of `parts` shares of its rows.
  long long whole;
  int parts;
};
cudaError_t launch_rope_forward(const RopeArgs& a, int d, bool bf16, cudaStream_t st);
// fp8: kc and vc are e4m3 with the scales ks and vs, else bf16.
cudaError_t launch_rope_append(const RopeArgs& a, int d, bool fp8, cudaStream_t st);
// CTAs of the backward launch, i.e. partial weight gradients it writes.
// Sets how they share the tokens.
int rope_grad_ctas(RopeArgs& a, int d);
cudaError_t launch_rope_backward(const RopeArgs& a, int ctas, int d, bool bf16, cudaStream_t st);
// dqw, dkw = the sums of the n partial weight gradients.
cudaError_t launch_rope_weight_grad(const RopeArgs& a, int n, int d, cudaStream_t st);

// ------------------------------------------------------------------ 8-bit pages read back
struct ReadArgs {
  const uint8_t* kc;  // pages [n_pages, page_size, kv_heads, d] e4m3
  const uint8_t* vc;
  const uint8_t* ks;  // their scales [n_pages, kv_heads, page_size] e8m0
  const uint8_t* vs;
  long long kc_page, vc_page, ks_page, vs_page;  // bytes from page to page
  void* ko;           // [tokens, kv_heads, d] bf16
  void* vo;
  const int* block_table;  // [n_req, max_pages]
  const int* lengths;      // [n_req]
  const int* cu;           // [n_req + 1]
  long long tokens;
  int n_req;
  int max_pages;
  int n_pages;
  int page_shift;
  int kv_heads;
  // Set by the launcher: rows that a warp takes together; outputs 32-byte aligned.
  int per_warp;
  int wide;
};
cudaError_t launch_paged_read(const ReadArgs& a, int d, cudaStream_t st);

// ------------------------------------------------------------------ paged decode
struct PagedArgs {
  const void* q;   // [T, heads, d] bf16
  const int* block_table;  // [n_req, max_pages]
  const int* lengths;      // [n_req], the new tokens included
  const int* cu_q;         // [n_req + 1], or null: n_q rows per request
  void* out;               // [T, heads, d] fp32, or bf16 (out_bf16)
  float* lse;              // [T, heads]
  long long T;
  long long n_q;           // rows per request; with cu_q those to expect
  long long window;        // 0: none
  int out_bf16;
  int n_req;
  int max_pages;
  int n_pages;
  int page_shift;
  int heads;
  int kv_heads;
  float scale_log2;        // log2(e) / sqrt(d)
  long long wait_limit;
  // Scratch: partial states of cut items, two slots per CTA (po [slot][row
  // tile][d]), and one record per CTA.
  float* po;
  float* pm;
  float* pl;
  void* cuts;
  // Pages in 8 bits: their scales, bytes from page to page.
  const uint8_t* ks;
  const uint8_t* vs;
  long long ks_page, vs_page;
  int item_heads;  // KV heads of an item: 1, or 2 of them, whose pairs kv_heads then counts
  // With a shared prefix.  Both launches leave states only: those of items that
  // are not cut at index whole + row of po, pm, pl, and in parts[row] where the
  // row's states are (paged_walk.cuh).
  long long whole;
  int2* parts;        // [T * heads]
  const int* cu_req;  // [n_groups + 1] the requests of each group
  int n_groups;
  int n_own;          // where the groups are among the requests, or all of them: requests
  // Where they follow the requests: n_req counts both, and of the groups
  const int* prefix_table;    // [n_groups, prefix_pages]
  const int* prefix_lengths;  // [n_groups]
  int prefix_pages;
};
// What the rows of a decode launch are: see paged_walk.cuh.
constexpr int kPagedPlain = 0, kPagedOwn = 1, kPagedShared = 2, kPagedBoth = 3;
// Query rows (of one request and KV head) that a CTA takes together: 8 or 16
// (paged_kernel.cu, two CTAs per SM) or 128 (paged_tc_kernel.cu, one).
int paged_row_tile(const PagedArgs& a, int d);
// Whether the own rows and those of groups go in one launch; group: the groups as requests.
bool paged_prefix_both(const PagedArgs& group);
size_t paged_cut_bytes(int ctas);
// tk, tv: maps over the pages, dims (d, kv_heads, page_size, n_pages), box
// 64 x 1 x min(page_size, 64) x 1, 128-byte swizzle.  kPagedShared goes right behind
// kPagedOwn, with no launch between them: it does not wait for what was before.
cudaError_t launch_paged_decode(const PagedArgs& a, int mode, int d, int ctas, int row_tile,
                                const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st);
cudaError_t launch_paged_combine(const PagedArgs& a, int d, int ctas, int row_tile, cudaStream_t st);
// out, lse = the states of both launches together (the row tiles are theirs).
cudaError_t launch_paged_join(const PagedArgs& own, const PagedArgs& shared, int d, int own_tile,
                              int shared_tile, cudaStream_t st);
cudaError_t launch_paged_tc(const PagedArgs& a, int mode, int d, int ctas, const CUtensorMap& tk,
                            const CUtensorMap& tv, cudaStream_t st);
// Over pages in 8 bits: row tiles of 8 or 16, two CTAs per SM, the same joining
// launch; tk, tv as above with a box of a whole row, page_size or
// paged_fp8_box_rows() rows.
int paged_fp8_row_tile(const PagedArgs& a);
int paged_fp8_item_heads(const PagedArgs& a, int d, int row_tile);
int paged_fp8_box_rows();
cudaError_t launch_paged_fp8(const PagedArgs& a, int d, int ctas, int row_tile, const CUtensorMap& tk,
                             const CUtensorMap& tv, cudaStream_t st);
cudaError_t take_paged_fp8_status(int* code);
// The shared launch on row tiles of 128 (the other launches: launch_paged_tc).
cudaError_t launch_paged_prefix(const PagedArgs& a, int d, int ctas, const CUtensorMap& tk, const CUtensorMap& tv,
                                cudaStream_t st);
cudaError_t take_paged_prefix_status(int* code);
cudaError_t take_paged_status(int* code);
cudaError_t take_paged_tc_status(int* code);

}  // namespace ra
