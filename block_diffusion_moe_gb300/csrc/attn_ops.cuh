// Argument blocks, device helpers and launch wrappers of the attention
// operations (clover_kv_write, clover_kv_read, clover_kv_attention,
// clover_prompt_attention), shared by their host side and their kernels.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "fp4.cuh"
#include "plan.h"
#include "sm100.cuh"

namespace clover {

// A paged cache (include/clover.h, clover_kv_cache) and its sequences.
struct KvCache {
  uint8_t* pages;
  int n_pages, page_tokens, heads, dim;
  float k_mul, v_mul;  // 2^k_exp, 2^v_exp (writing: 2^-k_exp, 2^-v_exp)
};

struct AttnSeqs {
  const int32_t* offsets;  // [n + 1] rows of the call
  const int32_t* lens;     // [n] (cache)
  const int32_t* table;    // [n][max_pages] (cache)
  const int32_t* k_offsets;  // [n + 1] (prompt)
  int n, max_pages;
  int n_rows, n_keys;      // rows of the call; key rows (prompt), table capacity (cache)
};

// Strided rows of heads, strides in bytes.
struct AttnRows {
  const uint8_t* data;
  int64_t row, head;
};

struct KvCopyArgs {  // write: k, v -> cache; read: cache -> k_out, v_out
  KvCache c;
  AttnSeqs s;
  AttnRows k, v;
  __nv_bfloat16* k_out;
  __nv_bfloat16* v_out;
  int wide;            // set by the launch: 32-byte accesses to the rows are aligned
  int cta_rows;        // set by the launch: rows of a CTA
  uint32_t row_magic;  // set by the launch: 2^32 / blocks of a row, rounded up (0: divide)
};

cudaError_t launch_kv_write(const KvCopyArgs& a, bool bf16, cudaStream_t s);
cudaError_t launch_kv_read(const KvCopyArgs& a, cudaStream_t s);

struct AttnArgs {
  KvCache c;  // heads and dim are set for prompts too
  AttnSeqs s;
  AttnRows q, k, v;
  int q_heads, group;  // group: query heads per key/value head
  int block;
  float scale_log2;  // scale * log2(e) * 2^k_exp
  __nv_bfloat16* out;
  float* lse;  // or null
  int wide_out;  // set by the launch: 32-byte stores to out are aligned
  int* err;         // status words of the workspace
  int* shared_err;  // and of the library
};

// A piece of a cut item: which of how many (at most one: nothing to join), and the
// item's rows.
struct AttendJoin {
  int parts, part, head, row0, tokens;
};

// Attention on tensor-core tiles (csrc/attend.cu). A tile is 128 rows: the
// group's query heads of `tokens` = 128 / group consecutive tokens, row
// token * group + head.
struct AttendArgs {
  CUtensorMap tm_q;  // q [n_rows][q_heads][dim], boxes of 64 elements x group x tokens
  CUtensorMap tm_k;  // prompt: k [n_keys][heads][dim], boxes of 64 elements x 1 x 128
  CUtensorMap tm_v;
  AttnArgs a;
  int tokens;
  int n_slots;         // pairs of tiles: n_rows / (2 tokens) + the number of sequences
  int may_cut;         // few items are cut into pieces
  float* part;         // [CTAs][2][dim / 4][128][4] sums of pieces, or flushed (workspace)
  float2* part_ml;     // [pieces][256] their maxima (of S) and sums of weights
  float* part_c;       // [pieces][256] exponent of 2 per unit of their scores
  AttendJoin* joins;   // [pieces]
  uint32_t per_magic;  // set by the launch: 2^32 / sixteens of a page, rounded up (0: one)
};

cudaError_t launch_attend(const AttendArgs& a, bool cached, int sms, cudaStream_t s);

// The library's own status block on the current device.
cudaError_t attention_shared_status(void** p);

// Attention of few query rows over a cache (csrc/attend_few.cu): tiles of at most
// 8 or 16 rows, the group's query heads of `tokens` tokens.
constexpr int kFewRows = 16;

struct AttendFewArgs {
  AttnArgs a;
  int tokens;
  float* part;        // [2 pieces][16 (8)][dim] sums of parts of a tile's keys (workspace)
  float2* part_ml;    // [2 pieces][16] their maxima and sums of weights
  uint32_t* arrived;  // [pieces], zero between calls
  uint32_t per_magic;  // set by the launch: 2^32 / sixteens of a page, rounded up (0: one)
};

// alone: a piece of the work to each warp, else to an SM.
cudaError_t launch_attend_few(const AttendFewArgs& a, int sms, bool alone, cudaStream_t s);

// ------------------------------------------------------------ device helpers

// A wait ran out.
__device__ __forceinline__ void record_timeout(const AttnArgs& a) {
  atomicOr(a.err, kErrMbarTimeout);
  atomicOr(a.shared_err, kErrMbarTimeout);
}

// One sequence of a call: its rows, and how many positions it has.
struct SeqSpan {
  int row0, rows, len;
  int key0;  // first key row (prompt)
};

__device__ __forceinline__ SeqSpan seq_span(const AttnSeqs& s, int i) {
  SeqSpan r;
  r.row0 = group_offset(s.offsets, i, s.n_rows);
  r.rows = max(group_offset(s.offsets, i + 1, s.n_rows) - r.row0, 0);
  if (s.k_offsets != nullptr) {
    r.key0 = group_offset(s.k_offsets, i, s.n_keys);
    r.len = max(group_offset(s.k_offsets, i + 1, s.n_keys) - r.key0, 0);
  } else {
    r.key0 = 0;
    r.len = min(max(s.lens[i], 0), s.n_keys);
  }
  return r;
}

// The last sequence that begins at or before this row (-1: none does).
__device__ __forceinline__ int seq_of_row(const AttnSeqs& s, int row) {
  int lo = -1, hi = s.n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (s.offsets[m] <= row)
      lo = m;
    else
      hi = m;
  }
  return lo;
}

// Positions below this are seen by the query at position p of len.
__device__ __forceinline__ int seen(int p, int len, int block) {
  if (block == 0) return len;
  if (p < 0) return 0;
  const int64_t end = (static_cast<int64_t>(p / block) + 1) * block;
  return end < len ? static_cast<int>(end) : len;
}

// The sixteen that holds position j of sequence i and head h: 16 rows of key codes, their
// scales, the same of the values. Null where there is no page.
__device__ __forceinline__ uint8_t* kv_sixteen(const KvCache& c, const AttnSeqs& s, int i, int h, int j) {
  const int slot = j / c.page_tokens;
  const int page = s.table[static_cast<int64_t>(i) * s.max_pages + slot];
  if (page < 0 || page >= c.n_pages) return nullptr;
  const int per = c.page_tokens / 16;
  return c.pages + ((static_cast<int64_t>(page) * c.heads + h) * per + (j - slot * c.page_tokens) / 16) * (18 * c.dim);
}

}  // namespace clover
