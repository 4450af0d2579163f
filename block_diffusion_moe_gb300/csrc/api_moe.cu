// Host side of the routed-expert operations declared in include/clover.h:
// argument checks, workspace layout and kernel launches.
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "../../include/clover.h"
#include "internal.h"
#include "moe_ops.cuh"

using namespace clover;

namespace {

int fail(int code, const char* fmt, ...) {
  char msg[400];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(msg, sizeof(msg), fmt, ap);
  va_end(ap);
  return set_last_error(code, msg);
}

int launched(cudaError_t e, const char* where) {
  const cudaError_t last = cudaGetLastError();
  if (e == cudaSuccess) e = last;
  if (e == cudaSuccess) return CLOVER_OK;
  return fail(CLOVER_ERR_CUDA, "%s: %s (%s)", where, cudaGetErrorName(e), cudaGetErrorString(e));
}

bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

constexpr int kMaxGroups = kFp4MaxGroups;
// Slots or rows of a call: 2^29 keeps every count of row tiles in 31 bits, even
// over offsets that do not ascend.
constexpr int kMaxSlots = 1 << 29;
constexpr size_t kCtrlBytes = 256;  // the status word that clover_workspace_status reads

int check_routing(const clover_routing* r) {
  if (r == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "routing is NULL");
  if (r->n_experts < 1 || r->n_experts > kRouteOpMaxExperts)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_experts=%d outside [1, %d]", r->n_experts, kRouteOpMaxExperts);
  if (r->top_k < 1 || r->top_k > kRouteOpMaxTopK || r->top_k > r->n_experts)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "top_k=%d: must be 1 to 32 and <= n_experts", r->top_k);
  if (r->score != CLOVER_SCORE_SOFTMAX && r->score != CLOVER_SCORE_SIGMOID)
    return fail(CLOVER_ERR_INVALID_ARG, "score=%d is neither softmax nor sigmoid", r->score);
  if (r->n_groups < 1 || r->n_groups > 32 || r->n_experts % r->n_groups != 0)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_groups=%d: must be 1 to 32 and divide n_experts", r->n_groups);
  if (r->top_groups < 1 || r->top_groups > r->n_groups)
    return fail(CLOVER_ERR_INVALID_ARG, "top_groups=%d outside [1, n_groups]", r->top_groups);
  if (r->group_rank != 1 && r->group_rank != 2)
    return fail(CLOVER_ERR_INVALID_ARG, "group_rank=%d is neither 1 nor 2", r->group_rank);
  if (!isfinite(r->scale)) return fail(CLOVER_ERR_INVALID_ARG, "scale is not finite");
  return CLOVER_OK;
}

size_t route_bytes(const clover_routing& r, int32_t M) {
  return kCtrlBytes + static_cast<size_t>(r.n_experts) * (static_cast<size_t>(plan::route_max_ctas(M)) + 1) * 4;
}

int fp4_block(int32_t format) { return format == CLOVER_FP4_MX ? 32 : 16; }

int check_fp4(int32_t format, int32_t cols) {
  if (format != CLOVER_FP4_NV && format != CLOVER_FP4_MX)
    return fail(CLOVER_ERR_INVALID_ARG, "format=%d is neither NV nor MX", format);
  if (cols < 64 || cols > (1 << 20) || cols % 64 != 0)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "cols=%d: must be a multiple of 64, 64 to 2^20", cols);
  return CLOVER_OK;
}

size_t scale_tile_bytes(int32_t format, int32_t cols) {
  return static_cast<size_t>((cols / fp4_block(format) + 3) / 4) * 512;
}

int check_input(const void* x, int32_t x_type, int64_t ldx, int32_t cols) {
  if (x_type != CLOVER_TYPE_F32 && x_type != CLOVER_TYPE_BF16)
    return fail(CLOVER_ERR_INVALID_ARG, "x_type=%d is neither fp32 nor bf16", x_type);
  if (x == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "x is NULL");
  const int64_t size = x_type == CLOVER_TYPE_F32 ? 4 : 2;
  if (ldx < cols || ldx > (INT64_C(1) << 40)) return fail(CLOVER_ERR_INVALID_ARG, "ldx smaller than cols (or past 2^40)");
  if (!aligned(x, 16) || (ldx * size) % 16 != 0) return fail(CLOVER_ERR_INVALID_ARG, "rows of x not 16-byte aligned");
  return CLOVER_OK;
}

int check_groups(int32_t n_rows, int32_t n_groups) {
  if (n_rows < 0 || n_rows > kMaxSlots) return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_rows=%d outside [0, 2^29]", n_rows);
  if (n_groups < 1 || n_groups > kMaxGroups)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_groups=%d outside [1, %d]", n_groups, kMaxGroups);
  return CLOVER_OK;
}

int check_matrices(int32_t n_mats, int32_t rows) {
  if (n_mats < 0 || rows < 0) return fail(CLOVER_ERR_INVALID_ARG, "n_mats=%d rows=%d: negative", n_mats, rows);
  if (static_cast<int64_t>(n_mats) * rows > kMaxSlots)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_mats=%d rows=%d: more than 2^29 rows", n_mats, rows);
  return CLOVER_OK;
}

int check_exp(int32_t scale_exp) {
  if (scale_exp < -64 || scale_exp > 64) return fail(CLOVER_ERR_INVALID_ARG, "scale_exp=%d outside [-64, 64]", scale_exp);
  return CLOVER_OK;
}

int check_codes(const void* codes, const void* scales) {
  if (codes == nullptr || scales == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "NULL codes/scales");
  if (!aligned(codes, 16) || !aligned(scales, 16))
    return fail(CLOVER_ERR_INVALID_ARG, "codes/scales not 16-byte aligned");
  return CLOVER_OK;
}

}  // namespace

extern "C" {

size_t clover_route_workspace_bytes(const clover_routing* routing, int32_t max_tokens) {
  if (check_routing(routing)) return 0;
  if (max_tokens < 0 || static_cast<int64_t>(max_tokens) * routing->top_k > kMaxSlots) {
    fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "max_tokens=%d: negative, or more than 2^29 slots", max_tokens);
    return 0;
  }
  return route_bytes(*routing, max_tokens);
}

int clover_route(const clover_routing* routing, const void* logits, int32_t logits_type, int64_t ld,
                 const float* bias, int32_t M, int32_t* topk_idx, float* topk_w, int32_t* offsets, int32_t* rows,
                 int32_t* pos, void* workspace, size_t workspace_bytes, clover_stream_t stream) {
  int rc;
  if ((rc = check_routing(routing))) return rc;
  const clover_routing& r = *routing;
  if (M < 0 || static_cast<int64_t>(M) * r.top_k > kMaxSlots)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "M=%d: negative, or more than 2^29 slots", M);
  if (logits_type != CLOVER_TYPE_F32 && logits_type != CLOVER_TYPE_BF16)
    return fail(CLOVER_ERR_INVALID_ARG, "logits_type=%d is neither fp32 nor bf16", logits_type);
  const bool grouping = offsets != nullptr;
  const size_t size = logits_type == CLOVER_TYPE_F32 ? 4 : 2;
  if (M > 0) {
    if (logits == nullptr || topk_idx == nullptr || topk_w == nullptr)
      return fail(CLOVER_ERR_INVALID_ARG, "NULL logits/topk_idx/topk_w");
    if ((rows != nullptr) != grouping || (pos != nullptr) != grouping)
      return fail(CLOVER_ERR_INVALID_ARG, "offsets, rows and pos must all be set or all be NULL");
    if (ld < r.n_experts || ld > (INT64_C(1) << 32))
      return fail(CLOVER_ERR_INVALID_ARG, "ld smaller than n_experts (or past 2^32)");
    if (!aligned(logits, size)) return fail(CLOVER_ERR_INVALID_ARG, "logits not aligned to their element size");
  }
  if (!aligned(bias, 4) || !aligned(topk_idx, 4) || !aligned(topk_w, 4) || !aligned(offsets, 4) || !aligned(rows, 4) ||
      !aligned(pos, 4))
    return fail(CLOVER_ERR_INVALID_ARG, "bias/topk_idx/topk_w/offsets/rows/pos not 4-byte aligned");
  if ((rc = check_workspace(workspace, workspace_bytes, route_bytes(r, M)))) return rc;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M == 0) {
    if (!grouping) return CLOVER_OK;
    return launched(cudaMemsetAsync(offsets, 0, static_cast<size_t>(r.n_experts + 1) * 4, s), "clearing the offsets");
  }
  RouteOpArgs a;
  a.logits = logits;
  a.bias = bias;
  a.ld = ld;
  a.bf16_logits = logits_type == CLOVER_TYPE_BF16;
  a.M = M;
  a.E = r.n_experts;
  a.K = r.top_k;
  a.softmax = r.score == CLOVER_SCORE_SOFTMAX;
  // with every group kept the groups change nothing
  a.n_groups = r.top_groups < r.n_groups ? r.n_groups : 1;
  a.top_groups = r.top_groups;
  a.group_rank = r.group_rank;
  a.renormalise = r.renormalise != 0;
  a.scale = r.scale;
  a.idx = topk_idx;
  a.w = topk_w;
  a.offsets = offsets;
  a.rows = rows;
  a.pos = pos;
  a.shape = plan::route_shape(M);
  a.n_ctas = a.shape.ctas;
  a.cta_tokens = a.shape.cta_tokens;
  if (!a.shape.cluster && a.n_ctas > plan::route_max_ctas(M))
    return fail(CLOVER_ERR_INVALID_ARG, "M=%d: launch of %d CTAs, the workspace holds %d", M, a.n_ctas,
                plan::route_max_ctas(M));
  a.totals = reinterpret_cast<int32_t*>(static_cast<uint8_t*>(workspace) + kCtrlBytes);
  a.hist = a.totals + a.E;
  return launched(launch_route_op(a, s), "launch route");
}

size_t clover_fp4_scale_bytes(int32_t format, int32_t n_mats, int32_t rows, int32_t cols) {
  if (check_fp4(format, cols) || check_matrices(n_mats, rows)) return 0;
  return static_cast<size_t>(n_mats) * ((static_cast<size_t>(rows) + 127) / 128) * scale_tile_bytes(format, cols);
}

size_t clover_fp4_grouped_scale_bytes(int32_t format, int32_t n_rows, int32_t n_groups, int32_t cols) {
  if (check_fp4(format, cols) || check_groups(n_rows, n_groups)) return 0;
  return (static_cast<size_t>(n_rows) / 128 + n_groups) * scale_tile_bytes(format, cols);
}

int clover_quantize_fp4(int32_t format, const void* x, int32_t x_type, int64_t ldx, int32_t n_mats, int32_t rows,
                        int32_t cols, int32_t scale_exp, uint8_t* codes, uint8_t* scales, clover_stream_t stream) {
  int rc;
  if ((rc = check_fp4(format, cols)) || (rc = check_matrices(n_mats, rows)) || (rc = check_exp(scale_exp))) return rc;
  if (n_mats == 0 || rows == 0) return CLOVER_OK;
  if ((rc = check_input(x, x_type, ldx, cols)) || (rc = check_codes(codes, scales))) return rc;
  Fp4QuantArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.ldx = ldx;
  a.bf16_x = x_type == CLOVER_TYPE_BF16;
  a.n_rows = static_cast<int64_t>(n_mats) * rows;
  a.mat_rows = rows;
  a.cols = cols;
  a.mul = ldexpf(1.f, -scale_exp);
  a.codes = codes;
  a.scales = scales;
  return launched(launch_quantize_fp4(a, format == CLOVER_FP4_MX, reinterpret_cast<cudaStream_t>(stream)),
                  "launch quantize fp4");
}

int clover_quantize_fp4_rows(int32_t format, const void* x, int32_t x_type, int64_t ldx, int32_t n_src, int32_t cols,
                             int32_t scale_exp, const int32_t* src_rows, int32_t src_div, int32_t n_rows,
                             const int32_t* offsets, int32_t n_groups, uint8_t* codes, uint8_t* scales,
                             clover_stream_t stream) {
  int rc;
  if ((rc = check_fp4(format, cols)) || (rc = check_groups(n_rows, n_groups)) || (rc = check_exp(scale_exp))) return rc;
  if (n_src < 0 || src_div < 1) return fail(CLOVER_ERR_INVALID_ARG, "n_src=%d src_div=%d: need >= 0 and >= 1", n_src, src_div);
  if (n_rows == 0) return CLOVER_OK;
  if ((rc = check_input(x, x_type, ldx, cols)) || (rc = check_codes(codes, scales))) return rc;
  if (offsets == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "offsets is NULL");
  if (!aligned(offsets, 4) || !aligned(src_rows, 4))
    return fail(CLOVER_ERR_INVALID_ARG, "offsets/src_rows not 4-byte aligned");
  Fp4QuantArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.ldx = ldx;
  a.bf16_x = x_type == CLOVER_TYPE_BF16;
  a.n_rows = n_rows;
  a.cols = cols;
  a.mul = ldexpf(1.f, -scale_exp);
  a.src_rows = src_rows;
  a.src_div = src_div;
  a.n_src = n_src;
  a.offsets = offsets;
  a.n_groups = n_groups;
  a.codes = codes;
  a.scales = scales;
  return launched(launch_quantize_fp4(a, format == CLOVER_FP4_MX, reinterpret_cast<cudaStream_t>(stream)),
                  "launch quantize fp4 rows");
}

int clover_dequantize_fp4(int32_t format, const uint8_t* codes, const uint8_t* scales, int32_t n_mats, int32_t rows,
                          int32_t cols, int32_t scale_exp, const int32_t* offsets, int32_t n_groups, uint16_t* out,
                          clover_stream_t stream) {
  int rc;
  if ((rc = check_fp4(format, cols)) || (rc = check_matrices(n_mats, rows)) || (rc = check_exp(scale_exp))) return rc;
  if (offsets != nullptr) {
    if ((rc = check_groups(rows, n_groups))) return rc;
    if (n_mats != 1) return fail(CLOVER_ERR_INVALID_ARG, "n_mats=%d: rows in groups form one matrix", n_mats);
    if (!aligned(offsets, 4)) return fail(CLOVER_ERR_INVALID_ARG, "offsets not 4-byte aligned");
  }
  if (n_mats == 0 || rows == 0) return CLOVER_OK;
  if ((rc = check_codes(codes, scales))) return rc;
  if (out == nullptr || !aligned(out, 16)) return fail(CLOVER_ERR_INVALID_ARG, "out is NULL or not 16-byte aligned");
  Fp4QuantArgs a;
  memset(&a, 0, sizeof(a));
  a.n_rows = static_cast<int64_t>(n_mats) * rows;
  a.mat_rows = rows;
  a.cols = cols;
  a.mul = ldexpf(1.f, scale_exp);
  a.offsets = offsets;
  a.n_groups = n_groups;
  a.codes = const_cast<uint8_t*>(codes);
  a.scales = const_cast<uint8_t*>(scales);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  return launched(launch_dequantize_fp4(a, format == CLOVER_FP4_MX, reinterpret_cast<cudaStream_t>(stream)),
                  "launch dequantize fp4");
}

size_t clover_fp4_product_workspace_bytes(void) { return kCtrlBytes; }

int clover_fp4_product_shared_workspace(void** workspace) {
  if (workspace == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "workspace is NULL");
  return launched(fp4_product_shared(workspace), "looking up the shared workspace");
}

int clover_fp4_product(int32_t format, const uint8_t* a_codes, const uint8_t* a_scales, int32_t n_rows,
                       const uint8_t* b_codes, const uint8_t* b_scales, const int32_t* offsets, int32_t n_groups,
                       int32_t N, int32_t K, float alpha, const float* group_alpha, int32_t epilogue, uint16_t* y,
                       void* workspace, size_t workspace_bytes, clover_stream_t stream) {
  int rc;
  if ((rc = check_fp4(format, K)) || (rc = check_groups(n_rows, n_groups))) return rc;
  if (epilogue != CLOVER_FP4_PLAIN && epilogue != CLOVER_FP4_SWIGLU)
    return fail(CLOVER_ERR_INVALID_ARG, "epilogue=%d is neither plain nor SwiGLU", epilogue);
  const bool swiglu = epilogue == CLOVER_FP4_SWIGLU;
  if (N < 1 || N > (1 << 24) || (swiglu && N % 2 != 0))
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "N=%d: must be 1 to 2^24, even with SwiGLU", N);
  if (!isfinite(alpha)) return fail(CLOVER_ERR_INVALID_ARG, "alpha is not finite");
  if (offsets == nullptr && n_groups != 1)
    return fail(CLOVER_ERR_INVALID_ARG, "offsets is NULL with n_groups=%d", n_groups);
  if ((rc = check_workspace(workspace, workspace_bytes, kCtrlBytes))) return rc;
  if (n_rows == 0) return CLOVER_OK;
  if ((rc = check_codes(a_codes, a_scales)) || (rc = check_codes(b_codes, b_scales))) return rc;
  if (y == nullptr || !aligned(y, 16)) return fail(CLOVER_ERR_INVALID_ARG, "y is NULL or not 16-byte aligned");
  if (!aligned(offsets, 4) || !aligned(group_alpha, 4))
    return fail(CLOVER_ERR_INVALID_ARG, "offsets/group_alpha not 4-byte aligned");
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  Fp4ProductArgs a;
  memset(&a, 0, sizeof(a));
  a.b_rows = swiglu ? N / 2 : N;
  const uint64_t mats = static_cast<uint64_t>(n_groups) * (swiglu ? 2 : 1);
  const uint32_t box_rows = swiglu ? 128 : 256, box_mats = swiglu ? 2 : 1;
  const bool pair = plan::fp4_pairs(n_rows, n_groups, K, swiglu);
  const uint64_t a_tiles = offsets != nullptr ? static_cast<uint64_t>(n_rows) / 128 + n_groups : (n_rows + 127) / 128;
  const uint32_t sf_bytes = 256 / (4 * fp4_block(format)) * 512;  // of a stage of 256 K elements
  if ((rc = encode_byte_boxes(&a.tm_a, a_codes, 0, n_rows, K / 2, 128, 128, 1, true, "rows' codes")) ||
      (rc = encode_byte_boxes(&a.tm_a32, a_codes, 0, n_rows, K / 2, 128, 32, 1, true, "rows' codes")) ||
      (rc = encode_byte_boxes(&a.tm_a_sf, a_scales, 0, a_tiles, scale_tile_bytes(format, K), sf_bytes, 1, 1, false,
                              "rows' scales")) ||
      (rc = encode_byte_boxes(&a.tm_b, b_codes, mats, a.b_rows, K / 2, 128, pair ? 128 : box_rows, pair ? 1 : box_mats,
                              true, "matrices' codes")) ||
      (rc = encode_byte_boxes(&a.tm_b_sf, b_scales, mats, (a.b_rows + 127) / 128, scale_tile_bytes(format, K), sf_bytes,
                              box_rows / 128, box_mats, false, "matrices' scales")))
    return rc;
  a.offsets = offsets;
  a.group_alpha = group_alpha;
  a.alpha = alpha;
  a.n_rows = n_rows;
  a.n_groups = n_groups;
  a.K = K;
  a.y = reinterpret_cast<__nv_bfloat16*>(y);
  a.err = static_cast<int*>(workspace);
  return launched(launch_fp4_product(a, format == CLOVER_FP4_MX, swiglu, pair, sms, reinterpret_cast<cudaStream_t>(stream)),
                  "launch fp4 product");
}

int clover_moe_combine(const uint16_t* y, int32_t n_rows, const int32_t* pos, const float* w, const uint16_t* shared,
                       const float* x, float* x_out, int32_t M, int32_t K, int32_t H, clover_stream_t stream) {
  if (n_rows < 0 || M < 0) return fail(CLOVER_ERR_INVALID_ARG, "n_rows=%d M=%d: negative", n_rows, M);
  if (K < 1 || K > kRouteOpMaxTopK || H < 8 || H % 8 != 0 || H > (1 << 20))
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "K=%d H=%d: need 1 <= K <= 32, H a multiple of 8, 8 to 2^20", K, H);
  if (static_cast<int64_t>(M) * K > kMaxSlots || static_cast<int64_t>(M) * (H / 8) > (INT64_C(1) << 38))
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "M=%d: too many slots or outputs", M);
  if (M == 0) return CLOVER_OK;
  if (pos == nullptr || w == nullptr || x_out == nullptr || (y == nullptr && n_rows > 0))
    return fail(CLOVER_ERR_INVALID_ARG, "NULL y/pos/w/x_out");
  if (!aligned(y, 16) || !aligned(shared, 16) || !aligned(x, 16) || !aligned(x_out, 16) || !aligned(pos, 4) ||
      !aligned(w, 4))
    return fail(CLOVER_ERR_INVALID_ARG, "y/shared/x/x_out not 16-byte aligned, or pos/w not 4-byte aligned");
  const uintptr_t xi = reinterpret_cast<uintptr_t>(x), xo = reinterpret_cast<uintptr_t>(x_out);
  const uintptr_t bytes = static_cast<uintptr_t>(M) * H * 4;
  if (x != nullptr && xi != xo && xi < xo + bytes && xo < xi + bytes)
    return fail(CLOVER_ERR_INVALID_ARG, "x and x_out overlap partially");
  CombineOpArgs a;
  a.y = reinterpret_cast<const __nv_bfloat16*>(y);
  a.pos = pos;
  a.w = w;
  a.shared = reinterpret_cast<const __nv_bfloat16*>(shared);
  a.x = x;
  a.out = x_out;
  a.n_rows = n_rows;
  a.M = M;
  a.K = K;
  a.H = H;
  return launched(launch_combine_op(a, reinterpret_cast<cudaStream_t>(stream)), "launch combine");
}

}  // extern "C"
