// Host side of the attention operations declared in include/clover.h: argument
// checks, workspace layout and kernel launches.
#include <float.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>
#include <string.h>

#include <algorithm>

#include "../../include/clover.h"
#include "attn_ops.cuh"
#include "internal.h"

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

constexpr int kMaxRows = 1 << 24;  // rows, key rows and positions of a call
constexpr int kMaxSeqs = plan::kMaxSeqs;
constexpr int kMaxKvHeads = 256;
constexpr int kMaxGroup = 64;
constexpr size_t kCtrlBytes = 256;  // the status word that clover_workspace_status reads

int check_heads(int32_t kv_heads, int32_t head_dim) {
  if (head_dim != 64 && head_dim != 128)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "head_dim=%d is neither 64 nor 128", head_dim);
  if (kv_heads < 1 || kv_heads > kMaxKvHeads)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "kv_heads=%d outside [1, %d]", kv_heads, kMaxKvHeads);
  return CLOVER_OK;
}

int check_q_heads(int32_t q_heads, int32_t kv_heads) {
  if (q_heads < 1 || q_heads % kv_heads != 0 || q_heads / kv_heads > kMaxGroup)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "q_heads=%d: must be 1 to %d times kv_heads=%d", q_heads, kMaxGroup, kv_heads);
  return CLOVER_OK;
}

int check_counts(int32_t n_rows, int32_t n_seqs) {
  if (n_rows < 0 || n_rows > kMaxRows) return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_rows=%d outside [0, 2^24]", n_rows);
  if (n_seqs < 1 || n_seqs > kMaxSeqs)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_seqs=%d outside [1, %d]", n_seqs, kMaxSeqs);
  return CLOVER_OK;
}

int check_page(int32_t page_tokens) {
  if (page_tokens < 16 || page_tokens > 65536 || page_tokens % 16 != 0)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "page_tokens=%d: must be a multiple of 16, 16 to 65536", page_tokens);
  return CLOVER_OK;
}

// The shapes of a cache and its sequences, without the pointers.
int check_cache(const clover_kv_cache* c, const clover_kv_seqs* s, int32_t n_rows) {
  int rc;
  if (c == nullptr || s == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "cache or seqs is NULL");
  if ((rc = check_heads(c->kv_heads, c->head_dim)) || (rc = check_page(c->page_tokens)) ||
      (rc = check_counts(n_rows, s->n_seqs)))
    return rc;
  if (c->n_pages < 1) return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_pages=%d: need at least one", c->n_pages);
  if (c->k_exp < -64 || c->k_exp > 64 || c->v_exp < -64 || c->v_exp > 64)
    return fail(CLOVER_ERR_INVALID_ARG, "k_exp=%d v_exp=%d outside [-64, 64]", c->k_exp, c->v_exp);
  if (s->max_pages < 0 || static_cast<int64_t>(s->max_pages) * c->page_tokens > kMaxRows)
    return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "max_pages=%d of %d tokens: negative, or more than 2^24 positions",
                s->max_pages, c->page_tokens);
  return CLOVER_OK;
}

int check_cache_pointers(const clover_kv_cache* c, const clover_kv_seqs* s) {
  if (c->pages == nullptr || s->offsets == nullptr || s->lens == nullptr || (s->table == nullptr && s->max_pages > 0))
    return fail(CLOVER_ERR_INVALID_ARG, "NULL pages/offsets/lens/table");
  if (!aligned(c->pages, 16)) return fail(CLOVER_ERR_INVALID_ARG, "pages not 16-byte aligned");
  if (!aligned(s->offsets, 4) || !aligned(s->lens, 4) || !aligned(s->table, 4))
    return fail(CLOVER_ERR_INVALID_ARG, "offsets/lens/table not 4-byte aligned");
  return CLOVER_OK;
}

int check_rows(const clover_rows* r, const char* what, int32_t rows, int32_t heads, int32_t dim, int size, AttnRows* out) {
  if (r == nullptr || r->data == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "%s is NULL", what);
  const int64_t most = INT64_C(1) << 36;
  if ((rows > 1 && (r->row_stride < dim || r->row_stride > most)) ||
      (heads > 1 && (r->head_stride < dim || r->head_stride > most)))
    return fail(CLOVER_ERR_INVALID_ARG, "%s: stride smaller than head_dim (or past 2^36)", what);
  out->data = static_cast<const uint8_t*>(r->data);
  out->row = rows > 1 ? r->row_stride * size : static_cast<int64_t>(dim) * size;
  out->head = heads > 1 ? r->head_stride * size : static_cast<int64_t>(dim) * size;
  if (!aligned(r->data, 16) || out->row % 16 != 0 || out->head % 16 != 0)
    return fail(CLOVER_ERR_INVALID_ARG, "%s: rows not 16-byte aligned", what);
  return CLOVER_OK;
}

int check_rule(float scale, int32_t block) {
  if (!(scale > 0.f) || !isfinite(scale)) return fail(CLOVER_ERR_INVALID_ARG, "scale must be finite and positive");
  if (block < 0) return fail(CLOVER_ERR_INVALID_ARG, "block=%d is negative", block);
  return CLOVER_OK;
}

int check_out(const void* out, const void* lse) {
  if (out == nullptr || !aligned(out, 16)) return fail(CLOVER_ERR_INVALID_ARG, "out is NULL or not 16-byte aligned");
  if (!aligned(lse, 4)) return fail(CLOVER_ERR_INVALID_ARG, "lse not 4-byte aligned");
  return CLOVER_OK;
}

int check_prompt(int32_t n_rows, int32_t n_keys, int32_t n_seqs, int32_t q_heads, int32_t kv_heads, int32_t head_dim) {
  int rc;
  if ((rc = check_heads(kv_heads, head_dim)) || (rc = check_q_heads(q_heads, kv_heads)) ||
      (rc = check_counts(n_rows, n_seqs)))
    return rc;
  if (n_keys < 0 || n_keys > kMaxRows) return fail(CLOVER_ERR_UNSUPPORTED_SHAPE, "n_keys=%d outside [0, 2^24]", n_keys);
  return CLOVER_OK;
}

void fill_cache(const clover_kv_cache& c, const clover_kv_seqs& s, int32_t n_rows, int sign, KvCache* kc, AttnSeqs* ks) {
  memset(ks, 0, sizeof(*ks));
  kc->pages = c.pages;
  kc->n_pages = c.n_pages;
  kc->page_tokens = c.page_tokens;
  kc->heads = c.kv_heads;
  kc->dim = c.head_dim;
  kc->k_mul = ldexpf(1.f, sign * c.k_exp);
  kc->v_mul = ldexpf(1.f, sign * c.v_exp);
  ks->offsets = s.offsets;
  ks->lens = s.lens;
  ks->table = s.table;
  ks->n = s.n_seqs;
  ks->max_pages = s.max_pages;
  ks->n_rows = n_rows;
  ks->n_keys = s.max_pages * c.page_tokens;
}

// The factor that takes q . k to the exponent of 2: kept a positive finite number
// where it would leave fp32's range.
float exponent_scale(float scale, float k_mul) {
  const double c = static_cast<double>(scale) * k_mul * 1.4426950408889634;
  return c > FLT_MAX ? FLT_MAX : (c < FLT_TRUE_MIN ? FLT_TRUE_MIN : static_cast<float>(c));
}

// The status words that a call's kernels set.
int fill_status(AttnArgs* a, void* workspace) {
  void* shared = nullptr;
  const int rc = launched(attention_shared_status(&shared), "looking up the attention status");
  a->err = static_cast<int*>(workspace);
  a->shared_err = static_cast<int*>(shared);
  return rc;
}

// A workspace: the control block, arrival counters that are zero between calls, and
// behind them what needs no value before a call. The counters have this place in a
// workspace of either kernel, whichever was the last to use it.
constexpr size_t kArrived = kCtrlBytes;
constexpr size_t kFreeBytes = kArrived + (plan::attend_few_pieces(8, true) * 4 + 255) / 256 * 256;

// The kernel for few rows.
struct FewLayout {
  size_t ml, part, bytes;
};

FewLayout few_layout(int32_t rows, bool alone, int32_t head_dim) {
  const size_t pieces = plan::attend_few_pieces(rows, alone);
  FewLayout l;
  l.ml = kFreeBytes;
  l.part = l.ml + 2 * pieces * kFewRows * 8;
  l.bytes = l.part + 2 * pieces * (alone ? rows : kFewRows) * head_dim * 4;
  return l;
}

// The kernel on tiles, where a call may be cut: what the pieces are, their maxima,
// sums of weights and exponents, their sums.
constexpr size_t kJoinBytes = (plan::kAttendMaxPieces * sizeof(AttendJoin) + 255) / 256 * 256;

size_t tile_bytes(int32_t head_dim) {
  return kFreeBytes + kJoinBytes + static_cast<size_t>(plan::kAttendMaxPieces) * 256 * (12 + head_dim * 4);
}

// Fills in what the kernel on tiles needs besides a.
int fill_tiles(AttendArgs* t, int32_t n_rows, int32_t n_seqs, int32_t head_dim, void* workspace) {
  const AttnArgs& a = t->a;
  t->tokens = 128 / a.group;
  t->n_slots = n_rows / (2 * t->tokens) + n_seqs;
  t->may_cut = plan::attend_may_cut(n_rows, a.group, a.c.heads);
  t->joins = reinterpret_cast<AttendJoin*>(static_cast<uint8_t*>(workspace) + kFreeBytes);
  t->part_ml = reinterpret_cast<float2*>(static_cast<uint8_t*>(workspace) + kFreeBytes + kJoinBytes);
  t->part_c = reinterpret_cast<float*>(t->part_ml + plan::kAttendMaxPieces * 256);
  t->part = t->part_c + plan::kAttendMaxPieces * 256;
  return encode_head_boxes(&t->tm_q, a.q.data, n_rows, a.q_heads, head_dim, a.q.row, a.q.head, a.group, t->tokens, "q");
}

// (for up to n_rows rows: calls of fewer may take tiles of 8 rows instead of 16)
size_t cached_bytes(const clover_kv_cache& c, int32_t n_rows, int32_t q_heads, int32_t n_seqs, int32_t max_pages) {
  const int group = q_heads / c.kv_heads;
  const bool alone = plan::attend_few_alone(n_seqs, c.kv_heads);
  size_t most = kFreeBytes;
  if (group <= 8) most = std::max(most, few_layout(8, alone, c.head_dim).bytes);
  if (group <= 16 && plan::attend_few_rows(n_rows, group, n_seqs, c.kv_heads) == 16)
    most = std::max(most, few_layout(16, alone, c.head_dim).bytes);
  if (!plan::attend_few(n_rows, group, n_seqs)) most = std::max(most, tile_bytes(c.head_dim));
  return most;
}

size_t prompt_bytes(int32_t head_dim) { return tile_bytes(head_dim); }

}  // namespace

extern "C" {

int clover_attention_shared_status(void** status) {
  if (status == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "status is NULL");
  return launched(attention_shared_status(status), "looking up the attention status");
}

size_t clover_kv_page_bytes(int32_t page_tokens, int32_t kv_heads, int32_t head_dim) {
  if (check_page(page_tokens) || check_heads(kv_heads, head_dim)) return 0;
  return static_cast<size_t>(page_tokens / 16) * kv_heads * 18 * head_dim;
}

int clover_kv_write(const clover_kv_cache* cache, const clover_kv_seqs* seqs, const clover_rows* k, const clover_rows* v,
                    int32_t type, int32_t n_rows, clover_stream_t stream) {
  int rc;
  if ((rc = check_cache(cache, seqs, n_rows))) return rc;
  if (type != CLOVER_TYPE_F32 && type != CLOVER_TYPE_BF16)
    return fail(CLOVER_ERR_INVALID_ARG, "type=%d is neither fp32 nor bf16", type);
  if (n_rows == 0) return CLOVER_OK;
  if ((rc = check_cache_pointers(cache, seqs))) return rc;
  KvCopyArgs a;
  memset(&a, 0, sizeof(a));
  const int size = type == CLOVER_TYPE_F32 ? 4 : 2;
  if ((rc = check_rows(k, "k", n_rows, cache->kv_heads, cache->head_dim, size, &a.k)) ||
      (rc = check_rows(v, "v", n_rows, cache->kv_heads, cache->head_dim, size, &a.v)))
    return rc;
  fill_cache(*cache, *seqs, n_rows, -1, &a.c, &a.s);
  return launched(launch_kv_write(a, type == CLOVER_TYPE_BF16, reinterpret_cast<cudaStream_t>(stream)), "launch kv write");
}

int clover_kv_read(const clover_kv_cache* cache, const clover_kv_seqs* seqs, uint16_t* k_out, uint16_t* v_out,
                   int32_t n_rows, clover_stream_t stream) {
  int rc;
  if ((rc = check_cache(cache, seqs, n_rows))) return rc;
  if (n_rows == 0) return CLOVER_OK;
  if ((rc = check_cache_pointers(cache, seqs))) return rc;
  if (k_out == nullptr || v_out == nullptr || !aligned(k_out, 16) || !aligned(v_out, 16))
    return fail(CLOVER_ERR_INVALID_ARG, "k_out/v_out is NULL or not 16-byte aligned");
  KvCopyArgs a;
  memset(&a, 0, sizeof(a));
  fill_cache(*cache, *seqs, n_rows, 1, &a.c, &a.s);
  a.k_out = reinterpret_cast<__nv_bfloat16*>(k_out);
  a.v_out = reinterpret_cast<__nv_bfloat16*>(v_out);
  return launched(launch_kv_read(a, reinterpret_cast<cudaStream_t>(stream)), "launch kv read");
}

size_t clover_kv_attention_workspace_bytes(const clover_kv_cache* cache, int32_t n_rows, int32_t q_heads, int32_t n_seqs,
                                           int32_t max_pages) {
  clover_kv_seqs seqs;
  memset(&seqs, 0, sizeof(seqs));
  seqs.n_seqs = n_seqs;
  seqs.max_pages = max_pages;
  if (check_cache(cache, &seqs, n_rows) || check_q_heads(q_heads, cache->kv_heads)) return 0;
  return cached_bytes(*cache, n_rows, q_heads, n_seqs, max_pages);
}

int clover_kv_attention(const clover_kv_cache* cache, const clover_kv_seqs* seqs, const clover_rows* q, int32_t n_rows,
                        int32_t q_heads, float scale, int32_t block, uint16_t* out, float* lse, void* workspace,
                        size_t workspace_bytes, clover_stream_t stream) {
  int rc;
  if ((rc = check_cache(cache, seqs, n_rows)) || (rc = check_q_heads(q_heads, cache->kv_heads)) ||
      (rc = check_rule(scale, block)) ||
      (rc = check_workspace(workspace, workspace_bytes,
                            cached_bytes(*cache, n_rows, q_heads, seqs->n_seqs, seqs->max_pages))))
    return rc;
  if (n_rows == 0) return CLOVER_OK;
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  if ((rc = check_cache_pointers(cache, seqs)) ||
      (rc = check_rows(q, "q", n_rows, q_heads, cache->head_dim, 2, &a.q)) || (rc = check_out(out, lse)))
    return rc;
  fill_cache(*cache, *seqs, n_rows, 1, &a.c, &a.s);
  a.q_heads = q_heads;
  a.group = q_heads / cache->kv_heads;
  a.block = block;
  a.scale_log2 = exponent_scale(scale, a.c.k_mul);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  if ((rc = fill_status(&a, workspace))) return rc;
  if (plan::attend_few(n_rows, a.group, seqs->n_seqs)) {
    int sms = 0;
    if ((rc = device_sms(&sms))) return rc;
    AttendFewArgs f;
    f.a = a;
    const int rows = plan::attend_few_rows(n_rows, a.group, seqs->n_seqs, cache->kv_heads);
    const bool alone = plan::attend_few_alone(seqs->n_seqs, cache->kv_heads);
    const FewLayout l = few_layout(rows, alone, cache->head_dim);
    uint8_t* at = static_cast<uint8_t*>(workspace);
    f.tokens = rows / a.group;
    f.arrived = reinterpret_cast<uint32_t*>(at + kArrived);
    f.part_ml = reinterpret_cast<float2*>(at + l.ml);
    f.part = reinterpret_cast<float*>(at + l.part);
    return launched(launch_attend_few(f, sms < plan::kAttendSms ? sms : plan::kAttendSms, alone,
                                      reinterpret_cast<cudaStream_t>(stream)),
                    "launch kv attention");
  }
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  AttendArgs t;
  memset(&t, 0, sizeof(t));
  t.a = a;
  if ((rc = fill_tiles(&t, n_rows, seqs->n_seqs, cache->head_dim, workspace))) return rc;
  return launched(launch_attend(t, true, std::min(sms, plan::kAttendSms), reinterpret_cast<cudaStream_t>(stream)),
                  "launch kv attention");
}

size_t clover_prompt_attention_workspace_bytes(int32_t n_rows, int32_t n_keys, int32_t n_seqs, int32_t q_heads,
                                               int32_t kv_heads, int32_t head_dim) {
  if (check_prompt(n_rows, n_keys, n_seqs, q_heads, kv_heads, head_dim)) return 0;
  return prompt_bytes(head_dim);
}

int clover_prompt_attention(const clover_prompt_seqs* seqs, const clover_rows* q, const clover_rows* k,
                            const clover_rows* v, int32_t n_rows, int32_t n_keys, int32_t q_heads, int32_t kv_heads,
                            int32_t head_dim, float scale, int32_t block, uint16_t* out, float* lse, void* workspace,
                            size_t workspace_bytes, clover_stream_t stream) {
  int rc;
  if (seqs == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "seqs is NULL");
  if ((rc = check_prompt(n_rows, n_keys, seqs->n_seqs, q_heads, kv_heads, head_dim)) || (rc = check_rule(scale, block)) ||
      (rc = check_workspace(workspace, workspace_bytes,
                            prompt_bytes(head_dim))))
    return rc;
  if (n_rows == 0) return CLOVER_OK;
  AttnArgs a;
  memset(&a, 0, sizeof(a));
  if (seqs->offsets == nullptr || seqs->k_offsets == nullptr) return fail(CLOVER_ERR_INVALID_ARG, "NULL offsets/k_offsets");
  if (!aligned(seqs->offsets, 4) || !aligned(seqs->k_offsets, 4))
    return fail(CLOVER_ERR_INVALID_ARG, "offsets/k_offsets not 4-byte aligned");
  if ((rc = check_rows(q, "q", n_rows, q_heads, head_dim, 2, &a.q)) || (rc = check_out(out, lse))) return rc;
  if (n_keys > 0 && ((rc = check_rows(k, "k", n_keys, kv_heads, head_dim, 2, &a.k)) ||
                     (rc = check_rows(v, "v", n_keys, kv_heads, head_dim, 2, &a.v))))
    return rc;
  a.c.heads = kv_heads;
  a.c.dim = head_dim;
  a.c.v_mul = 1.f;
  a.s.offsets = seqs->offsets;
  a.s.k_offsets = seqs->k_offsets;
  a.s.n = seqs->n_seqs;
  a.s.n_rows = n_rows;
  a.s.n_keys = n_keys;
  a.q_heads = q_heads;
  a.group = q_heads / kv_heads;
  a.block = block;
  a.scale_log2 = exponent_scale(scale, 1.f);
  a.out = reinterpret_cast<__nv_bfloat16*>(out);
  a.lse = lse;
  if ((rc = fill_status(&a, workspace))) return rc;
  AttendArgs t;
  memset(&t, 0, sizeof(t));
  t.a = a;
  if ((rc = fill_tiles(&t, n_rows, seqs->n_seqs, head_dim, workspace))) return rc;
  t.tm_k = t.tm_v = t.tm_q;  // without keys nothing is loaded through them
  if (n_keys > 0 &&
      ((rc = encode_head_boxes(&t.tm_k, a.k.data, n_keys, kv_heads, head_dim, a.k.row, a.k.head, 1, 128, "k")) ||
      (rc = encode_head_boxes(&t.tm_v, a.v.data, n_keys, kv_heads, head_dim, a.v.row, a.v.head, 1, 128, "v"))))
    return rc;
  int sms = 0;
  if ((rc = device_sms(&sms))) return rc;
  return launched(launch_attend(t, false, std::min(sms, plan::kAttendSms), reinterpret_cast<cudaStream_t>(stream)),
                  "launch prompt attention");
}

}  // extern "C"
