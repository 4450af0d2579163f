// Argument blocks and launch wrappers of the routed-expert operations
// (clover_route, clover_quantize_fp4, clover_fp4_product,
// clover_moe_combine), shared by their host side and their kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "plan.h"

namespace clover {

constexpr int kRouteOpMaxExperts = 512;
constexpr int kRouteOpMaxTopK = 32;
// Tokens one CTA of the selection kernel takes, at most: one bit each in an
// expert's 64-bit token mask.
constexpr int kRouteOpCtaTokens = plan::kRouteCtaTokens;
static_assert(kRouteOpCtaTokens <= 64, "64-bit token masks");

struct RouteOpArgs {
  const void* logits;  // fp32 or bf16 [M], row t at element t * ld
  const float* bias;   // [E] or null
  int64_t ld;
  int bf16_logits;
  int M, E, K;
  int softmax, n_groups, top_groups, group_rank, renormalise;
  float scale;
  int32_t* idx;      // [M][K]
  float* w;          // [M][K]
  int32_t* offsets;  // [E + 1], null: no grouping
  int32_t* rows;     // [M * K]
  int32_t* pos;      // [M][K]
  int32_t* hist;     // [E][n_ctas] counts per expert and CTA (workspace)
  int32_t* totals;   // [E] (workspace)
  plan::RouteShape shape;
  int n_ctas;        // shape.ctas
  int cta_tokens;    // shape.cta_tokens, at most kRouteOpCtaTokens
  int vec;          // set by the launch: whole vectors of logits per lane
  int group_size;   // set by the launch: experts per group
  int group_shift;  // set by the launch: log2 of the lanes that hold one group, or -1
};

cudaError_t launch_route_op(const RouteOpArgs& a, cudaStream_t s);

struct CombineOpArgs {
  const __nv_bfloat16* y;       // [n_rows][H]
  const int32_t* pos;           // [M][K]
  const float* w;               // [M][K]
  const __nv_bfloat16* shared;  // [M][H] or null
  const float* x;               // [M][H] or null
  float* out;                   // [M][H]
  int n_rows, M, K, H;
};

cudaError_t launch_combine_op(const CombineOpArgs& a, cudaStream_t s);

struct Fp4QuantArgs {
  const void* x;            // fp32 or bf16 rows of cols, row i at element i * ldx
  int64_t ldx;
  int bf16_x;
  int64_t n_rows;           // rows of codes (n_mats * mat_rows, or the grouped rows)
  int mat_rows;             // rows per matrix (offsets == null)
  int cols;
  float mul;                // 2^-scale_exp (quantise), 2^scale_exp (dequantise)
  const int32_t* src_rows;  // grouped: source row of row i is src_rows[i] / src_div (null: i)
  int src_div;
  int src_shift;            // set by the launch: log2 of src_div, or -1
  int n_src;
  const int32_t* offsets;   // [n_groups + 1] or null
  int n_groups;
  uint8_t* codes;           // [n_rows][cols / 2]
  uint8_t* scales;          // tiles
  __nv_bfloat16* out;       // dequantise: [n_rows][cols]
  int wide;                 // set by the launch: 32-byte accesses to x (out) are aligned
};

cudaError_t launch_quantize_fp4(const Fp4QuantArgs& a, bool mx, cudaStream_t s);
cudaError_t launch_dequantize_fp4(const Fp4QuantArgs& a, bool mx, cudaStream_t s);

constexpr int kFp4MaxGroups = 512;

// Grouped product of 4-bit rows (csrc/product.cu).
struct Fp4ProductArgs {
  CUtensorMap tm_a;          // codes [n_rows][K / 2], boxes of 128 bytes x 128 rows
  CUtensorMap tm_a32;        // the same in boxes of 32 rows
  CUtensorMap tm_a_sf;       // scale tiles [row tiles][..], boxes of a stage's tiles x 1
  CUtensorMap tm_b;          // codes [mats][b_rows][K / 2], boxes of 128 bytes x 256 rows x 1 (SwiGLU: 128 x 2;
                             // CTA pairs: 128 x 1)
  CUtensorMap tm_b_sf;       // scale tiles [mats][b_rows / 128][..], boxes of a stage's tiles x 2 x 1 (SwiGLU: 1 x 2)
  const int32_t* offsets;    // [n_groups + 1] or null (one group of all rows)
  const float* group_alpha;  // [n_groups] or null
  float alpha;
  int n_rows, n_groups;
  int b_rows;                // rows of one B matrix: N, or N / 2 with SwiGLU
  int K;
  __nv_bfloat16* y;          // [n_rows][b_rows]
  int* err;
};

// The product's workspace in the library (256 bytes on the current device).
cudaError_t fp4_product_shared(void** p);

cudaError_t launch_fp4_product(const Fp4ProductArgs& a, bool mx, bool swiglu, bool pair, int sms, cudaStream_t s);

}  // namespace clover
