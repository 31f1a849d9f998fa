// Host-side launchers of the paged-cache kernels (internal to libcca; the C ABI that calls them
// is in paged_api.cu, the layer's paged decode step in decode.cu).
#pragma once

#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "cca.h"

namespace cca {

// Rows of a [token, head, channel] tensor: element (sequence b, its token i, head h) starts at
// ptr + base * token_stride (packed) or ptr + b * seq_stride (uniform), + i * token_stride
// + h * head_stride, in elements of dtype (CCA_F32 / CCA_BF16 / CCA_F16).
struct Rows {
  void *ptr = nullptr;
  int dtype = 0;
  long long seq = 0, tok = 0, head = 0;
};

// Output type of the attention beyond the CCA_* element types: bfloat16 leading terms at
// Rows::ptr and remainders at PagedArgs::o_lo (the up-projection's operands).
constexpr int kRowsSplit = 100;

struct PagedArgs {
  void *k = nullptr, *v = nullptr;   // pages [n_pages, Hkv, page_size, row]
  void *scales = nullptr;            // 4 bits: [n_pages, Hkv, page_size, 4] float16
  const int *table = nullptr;        // [B, max_pages]
  const int *lengths = nullptr;      // [B]
  int *status = nullptr;
  const int *cu = nullptr;           // [B + 1] or null: tokens / B new tokens per sequence
  int B = 0, max_pages = 0, n_pages = 0, page_log2 = 0, Hkv = 0, D = 0;
  int bits = 16, page_f16 = 1;       // 16 or 4; element type of 16-bit pages
  int tokens = 0;
  int len_add = 0;                   // added to lengths[b] (1 where the step advances them later)
  int H = 0;                         // query heads
  Rows q, qo;                        // append: rotated copy (optional); attention: queries, output
  Rows nk, nv;                       // append: new keys and values; gather: the dense rows
  void *o_lo = nullptr;
  float rope_base = 0.f;             // append: 0 = no rotation
  float scale = 0.f;                 // attention
  void *workspace = nullptr;
};

cudaError_t paged_append(const PagedArgs &a, cudaStream_t st);
cudaError_t paged_gather(const PagedArgs &a, cudaStream_t st);
size_t paged_attention_workspace(const PagedArgs &a);
// Work units (key tiles of one head and row tile) the largest possible batch has; the scheduler
// counts them in 32 bits.
long long paged_attention_units(const PagedArgs &a);
cudaError_t paged_attention(const PagedArgs &a, cudaStream_t st);
// The kernel for many rows a sequence behind it (4 bits), on `ctas` CTAs; params: its AttnParams.
int paged_tc_rows();
int paged_tc_keys();
cudaError_t paged_attention_tc(const PagedArgs &a, const void *params, int ctas, cudaStream_t st);


// The layer's decode step over a paged cache (decode.cu): a holds x, y, the weights, the states,
// lengths and status; pa the pages (len_add 1).
int check_paged_cache(const cca_paged_cache_t *c, PagedArgs &a);   // paged_api.cu
struct Dims;
struct DecodeArgs;
struct StageMarker;
size_t paged_step_workspace(const Dims &d, const PagedArgs &pa);
cudaError_t decode_step_paged(const Dims &d, DecodeArgs a, PagedArgs pa, void *workspace,
                              cudaStream_t st, const StageMarker &mark);

}  // namespace cca
