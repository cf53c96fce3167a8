// Internal interface of the serving and training operators around the
// attention kernels (page bookkeeping, q/k norm with rotary positions,
// paged decode) between serve_api.cu and the kernel units.
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>

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
cudaError_t launch_rope_append(const RopeArgs& a, int d, cudaStream_t st);
// CTAs of the backward launch, i.e. partial weight gradients it writes.
// Sets how they share the tokens.
int rope_grad_ctas(RopeArgs& a, int d);
cudaError_t launch_rope_backward(const RopeArgs& a, int ctas, int d, bool bf16, cudaStream_t st);
// dqw, dkw = the sums of the n partial weight gradients.
cudaError_t launch_rope_weight_grad(const RopeArgs& a, int n, int d, cudaStream_t st);

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
};
// Query rows (of one request and KV head) that a CTA takes together: 8 or 16
// (paged_kernel.cu, two CTAs per SM) or 128 (paged_tc_kernel.cu, one).
int paged_row_tile(const PagedArgs& a, int d);
size_t paged_cut_bytes(int ctas);
// tk, tv: maps over the pages, dims (d, kv_heads, page_size, n_pages), box
// 64 x 1 x min(page_size, 64) x 1, 128-byte swizzle.
cudaError_t launch_paged_decode(const PagedArgs& a, int d, int ctas, int row_tile,
                                const CUtensorMap& tk, const CUtensorMap& tv, cudaStream_t st);
cudaError_t launch_paged_combine(const PagedArgs& a, int d, int ctas, int row_tile, cudaStream_t st);
cudaError_t launch_paged_tc(const PagedArgs& a, int d, int ctas, const CUtensorMap& tk,
                            const CUtensorMap& tv, cudaStream_t st);
cudaError_t take_paged_status(int* code);
cudaError_t take_paged_tc_status(int* code);

}  // namespace ra
