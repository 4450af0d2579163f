// Attention on tensor-core tiles: clover_prompt_attention, and
// clover_kv_attention where a sequence has more than a few rows.
//
// An item is two tiles of 128 query rows (the group's heads of consecutive tokens
// of one sequence) over the keys they see, 128 at a time:
//   S = Q K^T          tcgen05.mma, both operands from shared memory
//   P = 2^(c (S - m))  one thread per row: m a running maximum, l the sum of P
//   O = O + P V        tcgen05.mma, P (16 bits) from tensor memory
// and in the end O / l. m moves only where the row's maximum has grown by more
// than a limit (O and l are scaled then): numerators and sums are floating point,
// and a P above 1 is rounded like any other. (Were m always the maximum itself, the largest P
// would be 1 and lose nothing, for a rescaling in most steps.)
//
// Roles: warps 0-3 and 4-7 the softmax of tile 0 and 1, warp 8 loads, warp 9
// issues the MMAs, warp 10 watches the ring for it. While one tile's softmax runs,
// the tensor core works for the other: two tiles fill tensor memory's time, and their
// scores and sums its 512 columns; numerators take the place of their scores. They
// are handed over in halves, so that the product begins while the other half is
// worked out (723 -> 700 us for 16,384 tokens). Prompt: keys and values come as they
// are (TMA), and warp 10 looks after the values that not every row may see. Cache:
// warp 8 copies pages' codes and scales, and warps 12-15 expand them to fp16 tiles
// (exact); queries become fp16 too, each row scaled by a power of two so that its
// largest element is about 2^14.
//
// CTAs are persistent, one per SM. Where a call has at most half as many items as SMs,
// an item's keys are cut into pieces, whose sums a second kernel joins.
//
// Measured on a GB300 (kernels alone, in a graph): one prompt of 16,384 tokens, causal,
// 16 heads of 128: 669 to 700 us, 1.6 PFLOP/s; 2 x 1,000 rows over 13,000 keys: 150 us, 1.37
// PFLOP/s; 4 prompts of up to 6,000 tokens in blocks of 32, 32 heads of 64: 152 us, 0.79
// PFLOP/s. With 128 elements a tile's chain of scores, softmax and products bounds it:
// the tensor pipe is busy 69% of the second of these. With 64 there are half the products
// to the same exponentials, and the softmax's chain is what is left (tensor pipe 36%,
// exponentials 36%, issue slots 44%). 32 rows of 16 heads over 131,072
// cached: 50 us, 14 steps of 1.7 us on each SM (the warps that expand share the issue
// slots with the softmax; a prompt's step takes 1.4), 9 us before the first and 9 for
// writing and joining the pieces' sums, 20 MB.
#include <math.h>

#include "attn_ops.cuh"
#include "launch.cuh"

namespace clover {

namespace {

constexpr int kKeys = 128;  // keys per step
constexpr uint32_t kTmemCols = 512;
// Columns of tile t's scores and sums: + 128 t. Its numerators lie where the scores
// were, which are in registers by then.
constexpr uint32_t kTmemS = 0, kTmemO = 256;
constexpr int kMinSteps = 4;                   // of a piece

template <int kDim, bool kCached>
struct Layout {
  static constexpr int kThreads = kCached ? 512 : 384;
  static constexpr int kTileBytes = 128 * kDim * 2;  // of Q, of K, of V
  static constexpr int kSlab = 128 * 128;            // 64 elements of 128 rows
  static constexpr int kStages = (kCached ? 4 : 5) * (128 / kDim);
  static constexpr int kSixteen = 18 * kDim;  // bytes of 16 tokens in the cache
  static constexpr int kHalf = 9 * kDim;      // of their keys, or of their values: codes, then scales
  static constexpr int kRawBytes = 8 * kHalf;  // a tile's
  static constexpr int kRaw = kCached ? 3 * (128 / kDim) : 0;
  // Numerators are about 2^(c (S - m) + kLift), m up to 2^kGrowth behind. Cache: at most
  // 2^15, and what fp16 rounds by more than half a step, or to 0, is 2^-36 of the largest.
  static constexpr float kGrowth = kCached ? 4.f : 8.f, kLift = kCached ? 11.f : 0.f;
};

// A row's numerators are 2^(c (S - base) + lift): base 0 and lift kLift - c m, rounded once,
// which all of them share, where c m is at most this. Where it is larger that rounding
// would be as large as the room above the lift in fp16 (from scores of 9e7 on; in fp32
// from 2e9 on): then base is m, and the difference, exact near the maximum, comes before
// the factor. (4 prompts in blocks of 32, heads of 64: 148 us without, 150 so, 153 to 162 with
// the difference for every row; what was added since makes them 152.)
constexpr float kFar = 1048576.f;
__device__ __forceinline__ float base_of(float m, float c) { return m == -INFINITY || fabsf(m * c) <= kFar ? 0.f : m; }

// Steps after which a tile's sums go to the workspace, where they are added in fp32, and
// begin again. The tensor core cuts off what its accumulators do not hold, each time it
// adds 16 keys: after so many steps (32,768 keys) that has taken 2^-14 of a sum of values of
// one sign, and without an end 0.5% of 1,048,576 and 10% of 2^24. (3 us each, 0.8%.)
constexpr int kFlush = 256;

constexpr int kItems = 16;  // of a CTA that are worked out at its beginning

// What a CTA works on.
struct Item {
  SeqSpan sp;
  int seq, head;
  int tok0;       // first token of tile 0 in the sequence; tile t: + t * tokens
  int n[2];       // steps of each tile
  int all, any;   // positions below `all` are seen by every row, none from `any` on
  int j0, j1;     // the steps of this piece
  int part, parts;  // parts 0: nothing
  __device__ __forceinline__ int steps(int t) const { return max(min(j1, n[t]) - j0, 0); }
  __device__ __forceinline__ int steps() const { return max(steps(0), steps(1)); }
};

struct Shared {
  uint64_t q_full[2], q_empty[2], q_ready[2];  // ready: converted (cache)
  uint64_t full[10], empty[10];
  uint64_t raw_full[6], raw_empty[6];
  uint64_t s_full[2], p_half[2], p_full[2], o_full[2], o_empty[2];
  uint64_t drain;
  uint32_t tmem, abort;
  int poison[16];  // of item k: [k % 16]
  uint32_t there[16];  // of step k: sixteens that have a page (cache)
  int sums[3][16];
  Item items[kItems];  // this CTA's first
};

// How a call is cut: every item whole, its slots counted from the offsets alone; or
// in pieces of at most `chunk` steps.
struct Cut {
  int chunk;   // 0: whole
  int pieces;  // (whole: slots, some of them empty)
};

__device__ __forceinline__ int seen_by(const AttendArgs& p, const SeqSpan& sp, int tok) {
  return seen(sp.len - sp.rows + tok, sp.len, p.a.block);
}

__device__ __forceinline__ void fill_item(const AttendArgs& p, Item* it) {
  it->any = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(it->tok0 + (t + 1) * p.tokens, it->sp.rows) - 1;
    const int lim = last < it->tok0 + t * p.tokens ? 0 : seen_by(p, it->sp, last);
    it->n[t] = (lim + kKeys - 1) / kKeys;
    it->any = max(it->any, lim);
  }
  it->all = seen_by(p, it->sp, it->tok0);
  it->j0 = 0;
  it->j1 = max(it->n[0], it->n[1]);
  it->part = 0;
  it->parts = 1;
}

// Pieces of an item of this many steps.
__device__ __forceinline__ int pieces_of(int steps, int chunk) { return max(1, (steps + chunk - 1) / chunk); }

__device__ __forceinline__ int steps_of_tile(const AttendArgs& p, const SeqSpan& sp, int tile) {
  const int last = min((tile + 1) * 2 * p.tokens, sp.rows) - 1;
  return (seen_by(p, sp, last) + kKeys - 1) / kKeys;
}

// Piece k, by a whole warp. False: an empty slot.
__device__ __forceinline__ bool locate(const AttendArgs& p, const Cut& cut, int k, Item* it) {
  const int pair = 2 * p.tokens, n = p.a.s.n_rows;
  if (cut.chunk == 0) {
    // the last tiles of a sequence see the most: they come first
    const int idx = cut.pieces - 1 - k, slot = idx / p.a.c.heads;
    it->head = idx - slot * p.a.c.heads;
    const int s = warp_search(p.a.s.n, slot, [&](int i) { return group_offset(p.a.s.offsets, i, n) / pair + i; });
    it->seq = s;
    it->sp = seq_span(p.a.s, s);
    it->tok0 = (slot - (it->sp.row0 / pair + s)) * pair;
    if (it->tok0 < 0 || it->tok0 >= it->sp.rows) return false;
    fill_item(p, it);
    return true;
  }
  const int lane = threadIdx.x & 31;
  for (int s0 = 0; s0 < p.a.s.n; s0 += 32) {
    int own = 0;
    if (s0 + lane < p.a.s.n) {
      const SeqSpan sp = seq_span(p.a.s, s0 + lane);
      for (int t = 0; t * pair < sp.rows; ++t) own += pieces_of(steps_of_tile(p, sp, t), cut.chunk);
      own *= p.a.c.heads;
    }
    int upto = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const int all = __shfl_sync(0xffffffffu, upto, 31);
    if (k >= all) {
      k -= all;
      continue;
    }
    const int l = __ffs(__ballot_sync(0xffffffffu, upto > k)) - 1;
    const int per_head = __shfl_sync(0xffffffffu, own, l) / p.a.c.heads;
    k -= __shfl_sync(0xffffffffu, upto - own, l);
    it->seq = s0 + l;
    it->sp = seq_span(p.a.s, it->seq);
    it->head = k / per_head;
    k -= it->head * per_head;
    for (int t = 0;; ++t) {
      const int steps = steps_of_tile(p, it->sp, t), parts = pieces_of(steps, cut.chunk);
      if (k < parts) {
        it->tok0 = t * pair;
        fill_item(p, it);
        it->part = k;
        it->parts = parts;
        it->j0 = static_cast<int>(static_cast<int64_t>(steps) * k / parts);
        it->j1 = static_cast<int>(static_cast<int64_t>(steps) * (k + 1) / parts);
        return true;
      }
      k -= parts;
    }
  }
  return false;
}

// How the call is cut, by all threads of a CTA; the same in every CTA. The pieces are
// at most as many as SMs, and as short as that allows: of a chunk between steps / SMs
// and steps / (SMs - items), where it is certain, each warp tries one length. (Of
// more items than half the SMs, none is cut: 126 items of 98 steps in two rounds of
// pieces took 324 us, whole 165.)
__device__ Cut cut_call(const AttendArgs& p, int (&sums)[3][16]) {
  const Cut whole = {0, p.n_slots * p.a.c.heads};
  if (!p.may_cut) return whole;
  const int pair = 2 * p.tokens, ctas = gridDim.x, warps = blockDim.x / 32, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int items = 0;
  uint32_t own = 0;  // steps (what overflows belongs to too many items)
  for (int i = threadIdx.x; i < p.a.s.n; i += blockDim.x) {
    const SeqSpan sp = seq_span(p.a.s, i);
    const int tiles = (sp.rows + pair - 1) / pair;
    items += min(tiles, ctas) * p.a.c.heads;
    if (tiles < ctas)
      for (int t = 0; t < tiles; ++t) own += steps_of_tile(p, sp, t) * p.a.c.heads;
  }
  items = warp_sum_i(items);
  int steps = warp_sum_i(static_cast<int>(own));
  if (lane == 0) sums[0][warp] = items, sums[1][warp] = steps;
  __syncthreads();
  items = steps = 0;
  for (int w = 0; w < warps; ++w) items += sums[0][w], steps += sums[1][w];
  if (2 * items > ctas) return whole;
  const int lo = max(kMinSteps, (steps + ctas - 1) / ctas), hi = max(kMinSteps, (steps + ctas - items - 1) / (ctas - items));
  auto chunk = [&](int w) { return lo + (hi - lo) * w / (warps - 1); };
  int pieces = 0;
  for (int i = lane; i < p.a.s.n; i += 32) {
    const SeqSpan sp = seq_span(p.a.s, i);
    for (int t = 0; t * pair < sp.rows; ++t) pieces += pieces_of(steps_of_tile(p, sp, t), chunk(warp)) * p.a.c.heads;
  }
  pieces = warp_sum_i(pieces);
  if (lane == 0) sums[2][warp] = pieces;
  __syncthreads();
  int w = 0;
  while (w < warps - 1 && sums[2][w] > ctas) ++w;
  return {chunk(w), sums[2][w]};
}

// This CTA's i-th piece: forth and back over the CTAs, so that no CTA always has the
// longest.
__device__ __forceinline__ int piece_at(int i) {
  const int b = blockIdx.x, g = gridDim.x;
  return i * g + (i & 1 ? g - 1 - b : b);
}

// A role's way through the CTA's pieces, by a whole warp.
struct Work {
  int i = -1;
  // The next one that is not empty; false: there is none left.
  __device__ __forceinline__ bool next(const AttendArgs& p, const Shared* sh, const Cut& cut, Item* it) {
    while (piece_at(++i) < cut.pieces) {
      if (i < kItems) {
        *it = sh->items[i];
        if (it->parts != 0) return true;
      } else if (locate(p, cut, piece_at(i), it)) {
        return true;
      }
    }
    return false;
  }
};

__device__ __forceinline__ bool warp_wait(const AttendArgs& p, Shared* sh, uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_wait(bar, parity, &sh->abort))) return true;
  if (elect_one()) {
    record_timeout(p.a);
    *reinterpret_cast<volatile uint32_t*>(&sh->abort) = 1u;
  }
  __syncwarp();
  return false;
}

// A ring's stages in turn. K and V ring: K of step 0, V of step 0, K of step 1, ...
template <int kStages>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int by = 1) {
    st += by;
    if (st >= kStages) {
      st -= kStages;
      ph ^= 1u;
    }
  }
};

// Copies of barriers that may be in flight when a role gives up.
struct Flight {
  uint32_t issued = 0, parity = 0;
  __device__ __forceinline__ void add(int st, uint32_t ph) {
    issued |= 1u << st;
    parity = (parity & ~(1u << st)) | (ph << st);
  }
  __device__ __forceinline__ void land(uint64_t* bars) {
    for (int i = 0; i < 32; ++i)
      if (issued >> i & 1u) mbar_wait_for(&bars[i], parity >> i & 1u, 200000000ull);
  }
};

template <int kDim, bool kCached>
__device__ void load_role(const AttendArgs& p, Shared* sh, const Cut& cut, uint32_t q, uint32_t ring, uint32_t raw) {
  using L = Layout<kDim, kCached>;
  const int lane = threadIdx.x & 31;
  const uint64_t keep = l2_policy_evict_last();
  Ring<kCached ? L::kRaw : L::kStages> r;
  Flight flight, q_flight;
  uint32_t q_count[2] = {0, 0};
  int k_step = 0;  // steps so far, of all items
  bool ok = true;
  Work work;
  Item it;
  while (ok && work.next(p, sh, cut, &it)) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (ok && it.steps(t) > 0) {
        ok = warp_wait(p, sh, &sh->q_empty[t], (q_count[t] & 1) ^ 1u);
        if (ok && elect_one()) {
          mbar_arrive_expect_tx(&sh->q_full[t], kDim / 64 * p.a.group * p.tokens * 128);
#pragma unroll
          for (int d = 0; d < kDim / 64; ++d)
            tma_load_3d(q + t * L::kTileBytes + d * L::kSlab, &p.tm_q, &sh->q_full[t], d * 64, it.head * p.a.group,
                        it.sp.row0 + it.tok0 + t * p.tokens, keep);
        }
        __syncwarp();
        if (ok) q_flight.add(t, q_count[t] & 1);
        ++q_count[t];
      }
    }
    const int steps = it.steps();
    if constexpr (!kCached) {
      for (int i = 0; i < 2 * steps && ok; ++i, r.next()) {
        if (!(ok = warp_wait(p, sh, &sh->empty[r.st], r.ph ^ 1u))) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(&sh->full[r.st], L::kTileBytes);
#pragma unroll
          for (int d = 0; d < kDim / 64; ++d)
            tma_load_3d(ring + r.st * L::kTileBytes + d * L::kSlab, i & 1 ? &p.tm_v : &p.tm_k, &sh->full[r.st], d * 64, it.head,
                        it.sp.key0 + (it.j0 + (i >> 1)) * kKeys, keep);
        }
        __syncwarp();
        flight.add(r.st, r.ph);
      }
    } else {
      // keys, then values of each step; lane i looks up the sixteen i % 8 of step i / 8 on,
      // four steps at a time
      const int per = p.a.c.page_tokens / 16;
      int from = -1;
      uint32_t all = 0;
      for (int i = 0; i < 2 * steps && ok; ++i, r.next()) {
        if ((i & 7) == 0) {
          const int x = (it.j0 + (i >> 1)) * 8 + lane;
          from = -1;
          if (x * 16 < it.any && (i >> 1) + (lane >> 3) < steps) {
            const int entry = p.per_magic != 0 ? static_cast<int>(__umulhi(x, p.per_magic)) : x;
            const int page = p.a.s.table[static_cast<int64_t>(it.seq) * p.a.s.max_pages + entry];
            if (page >= 0 && page < p.a.c.n_pages) from = (page * p.a.c.heads + it.head) * per + (x - entry * per);
          }
          all = __ballot_sync(0xffffffffu, from >= 0);
        }
        const int at = __shfl_sync(0xffffffffu, from, (i & 6) * 4 + (lane & 7));
        const uint32_t has = all >> ((i & 6) * 4) & 0xFFu;
        if (!(ok = warp_wait(p, sh, &sh->raw_empty[r.st], r.ph ^ 1u))) break;
        if (lane == 0) {
          if ((i & 1) == 0) *reinterpret_cast<volatile uint32_t*>(&sh->there[k_step & 15]) = has;
          mbar_arrive_expect_tx(&sh->raw_full[r.st], __popc(has) * L::kHalf);
        }
        k_step += i & 1;
        __syncwarp();
        if (lane < 8 && at >= 0)
          bulk_load(raw + r.st * L::kRawBytes + lane * L::kHalf,
                    p.a.c.pages + static_cast<int64_t>(at) * L::kSixteen + (i & 1) * L::kHalf, L::kHalf, &sh->raw_full[r.st]);
        __syncwarp();
        flight.add(r.st, r.ph);
      }
    }
  }
  // the copies in flight must land before the CTA leaves
  if (*reinterpret_cast<volatile uint32_t*>(&sh->abort)) {
    flight.land(kCached ? sh->raw_full : sh->full);
    q_flight.land(sh->q_full);
  }
}

// Run by a whole warp whose control flow is uniform: what it depends on is put in
// uniform registers, where the MMAs' descriptors stay. (With the piece count and the
// steps left in ordinary ones the issue of an MMA took longer than the 64 cycles
// that the tensor core needs for it.) False: gave up.
template <int kDim, bool kCached>
__device__ __forceinline__ bool issue_all(const AttendArgs& p, Shared* sh, const Cut& cut_in, uint32_t q, uint32_t ring) {
  using L = Layout<kDim, kCached>;
  constexpr uint32_t kIdS = kCached ? umma_idesc_f16(128, kKeys) : umma_idesc_bf16(128, kKeys);
  constexpr uint32_t kIdO = (kCached ? umma_idesc_f16(128, kDim) : umma_idesc_bf16(128, kDim)) | kUmmaBMnMajor;
  const Cut cut = {warp_uniform(cut_in.chunk), warp_uniform(cut_in.pieces)};
  const uint32_t tmem = static_cast<uint32_t>(warp_uniform(static_cast<int>(sh->tmem)));
  Ring<L::kStages> rk, rv;
  uint32_t items0 = 0, items1 = 0, steps0 = 0, steps1 = 0;
  // a descriptor whose address (in units of 16 bytes) is `at` further on than that of
  // the first Q tile or stage
  const uint64_t q_desc = umma_desc_sw128(q), k_desc = umma_desc_sw128(ring), v_desc = umma_desc_sw128_mn(ring, L::kSlab);
  auto at = [](uint64_t desc, uint32_t by) {
    return desc & ~0xFFFFFFFFull | static_cast<uint32_t>(desc) + by;
  };
  // (by one lane) tile t's scores of a step, whose keys lie in the ring at rk's stage
  auto scores = [&](int t, uint32_t k_at, bool last) {
#pragma unroll
    for (int s = 0; s < kDim / 16; ++s) {
      const uint32_t o = (s / 4) * (L::kSlab >> 4) + (s % 4) * 2;
      umma_bf16(tmem + kTmemS + t * 128, at(q_desc, t * (L::kTileBytes >> 4) + o), at(k_desc, k_at + o), kIdS, s > 0);
    }
    umma_commit(&sh->s_full[t]);
    if (last) umma_commit(&sh->q_empty[t]);
  };
  // (by one lane) half of its numerators times the values that rv holds: the upper 64
  // keys' come first
  auto sums = [&](int t, int h, uint32_t v_at, bool first) {
#pragma unroll
    for (int s = h * 4; s < h * 4 + 4; ++s)
      umma_bf16_ta(tmem + kTmemO + t * 128, tmem + kTmemS + t * 128 + s * 8, at(v_desc, v_at + s * 128), kIdO,
                   s != 4 ? 1u : !first);
  };
  auto stage = [](int st) { return static_cast<uint32_t>(warp_uniform(st * (L::kTileBytes >> 4))); };
  Work work;
  Item it;
  while (__any_sync(0xffffffffu, work.next(p, sh, cut, &it))) {
    const int n0 = warp_uniform(it.steps(0)), n1 = warp_uniform(it.steps(1)), steps = max(n0, n1);
    if (steps == 0) continue;
    rv = rk;
    rv.next();
    if (n0 > 0 && !warp_wait(p, sh, kCached ? &sh->q_ready[0] : &sh->q_full[0], items0 & 1)) return false;
    if (n1 > 0 && !warp_wait(p, sh, kCached ? &sh->q_ready[1] : &sh->q_full[1], items1 & 1)) return false;
    if (!warp_wait(p, sh, &sh->full[rk.st], rk.ph)) return false;
    tc_fence_after();
    const uint32_t k_first = stage(rk.st);
    if (elect_one()) {
      if (n0 > 0) scores(0, k_first, n0 == 1);
      if (n1 > 0) scores(1, k_first, n1 == 1);
      umma_commit(&sh->empty[rk.st]);
    }
    __syncwarp();
    for (int j = 0; j < steps; ++j) {
      rk.next(2);
      const uint32_t k_at = stage(rk.st), v_at = stage(rv.st);
      // p_half: half the numerators are in place, and the values of this step and the
      // keys of the next one; o_empty: the sums of the item before are read
      if (j < n0) {
        if (j == 0 && !warp_wait(p, sh, &sh->o_empty[0], (items0 & 1) ^ 1u)) return false;
        if (!warp_wait(p, sh, &sh->p_half[0], steps0 & 1)) return false;
        tc_fence_after();
        if (elect_one()) sums(0, 1, v_at, j == 0);
        __syncwarp();
        if (!warp_wait(p, sh, &sh->p_full[0], steps0++ & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          sums(0, 0, v_at, false);
          if (j + 1 == n0) umma_commit(&sh->o_full[0]);
          if (j + 1 < n0) scores(0, k_at, j + 2 == n0);
          if (j >= n1) {
            umma_commit(&sh->empty[rv.st]);
            if (j + 1 < steps) umma_commit(&sh->empty[rk.st]);
          }
        }
        __syncwarp();
      }
      if (j < n1) {
        if (j == 0 && !warp_wait(p, sh, &sh->o_empty[1], (items1 & 1) ^ 1u)) return false;
        if (!warp_wait(p, sh, &sh->p_half[1], steps1 & 1)) return false;
        tc_fence_after();
        if (elect_one()) sums(1, 1, v_at, j == 0);
        __syncwarp();
        if (!warp_wait(p, sh, &sh->p_full[1], steps1++ & 1)) return false;
        tc_fence_after();
        if (elect_one()) {
          sums(1, 0, v_at, false);
          if (j + 1 == n1) umma_commit(&sh->o_full[1]);
          if (j + 1 < n1) scores(1, k_at, j + 2 == n1);
          umma_commit(&sh->empty[rv.st]);
          if (j + 1 < steps) umma_commit(&sh->empty[rk.st]);
        }
        __syncwarp();
      }
      rv.next(2);
    }
    items0 += n0 > 0;
    items1 += n1 > 0;
  }
  return true;
}

template <int kDim, bool kCached>
__device__ void mma_role(const AttendArgs& p, Shared* sh, const Cut& cut, uint32_t q, uint32_t ring) {
  issue_all<kDim, kCached>(p, sh, cut, q, ring);
  if (elect_one()) umma_commit(&sh->drain);
  __syncwarp();
  mbar_wait_for(&sh->drain, 0, 200000000ull);
}

// Values that not every row sees: a weight of 0 does not keep an infinity or a
// NaN out of a sum. Rows of V past every row's sight become zeros, and so do
// infinities and NaN among the others, which the end of the softmax role adds
// to the rows that do see them (true: there were some). Step j of an item, by a warp.
template <int kDim>
__device__ __forceinline__ bool look_after(const Item& it, uint8_t* v, int j) {
  using L = Layout<kDim, false>;
  const int lane = threadIdx.x & 31, lo = max(it.all - j * kKeys, 0), hi = min(it.any - j * kKeys, kKeys);
  constexpr int kPer = kDim / 8;  // 16-byte pieces of a row
  uint32_t top = 0;
#pragma unroll 4
  for (int e = lane; e < (hi - lo) * kPer; e += 32) {
    const int row = lo + e / kPer, c = e % kPer;
    const uint4 x = *reinterpret_cast<const uint4*>(v + (c / 8) * L::kSlab + row * 128 + (c % 8) * 16);
    top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
  }
  const bool odd = __any_sync(0xffffffffu, (top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u);
  if (odd) {
    for (int e = lane; e < (hi - lo) * kDim; e += 32) {
      const int row = lo + e / kDim, d = e % kDim;
      uint16_t* x = reinterpret_cast<uint16_t*>(v + (d / 64) * L::kSlab + row * 128 + ((d % 64 / 8) ^ (row & 7)) * 16) + d % 8;
      if ((*x & 0x7F80u) == 0x7F80u) *x = 0;
    }
  }
  for (int e = lane; e < (kKeys - hi) * kPer; e += 32) {
    const int row = hi + e / kPer, c = e % kPer;
    *reinterpret_cast<uint4*>(v + (c / 8) * L::kSlab + row * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_shared();
  __syncwarp();
  return odd;
}

// Waits for the ring in place of the MMA role, which then has one barrier to wait
// for per tile and step (with all of them it left the tensor core idle for a
// quarter of the time), and looks after the prompt's values.
template <int kDim, bool kCached>
__device__ void watch_role(const AttendArgs& p, Shared* sh, const Cut& cut, uint8_t* ring) {
  using L = Layout<kDim, kCached>;
  const int lane = threadIdx.x & 31;
  Ring<L::kStages> r;
  uint32_t count[2] = {0, 0};
  Work work;
  Item it;
  for (int item = -1; work.next(p, sh, cut, &it);) {
    if (it.steps() == 0) continue;
    // (items with steps are counted; of a ring of 16, eight on, or back, is out of
    // everyone's reach)
    ++item;
    if (!kCached && lane == 0) *reinterpret_cast<volatile int*>(&sh->poison[(item + 8) & 15]) = 0;
    __syncwarp();
    const int steps = it.steps();
    for (int j = -1; j < steps; ++j) {
      if (j >= 0) {  // values of step j
        if (!warp_wait(p, sh, &sh->full[r.st], r.ph)) return;
        if (!kCached && (it.j0 + j + 1) * kKeys > it.all && look_after<kDim>(it, ring + r.st * L::kTileBytes, it.j0 + j) && lane == 0)
          *reinterpret_cast<volatile int*>(&sh->poison[item & 15]) = 1;
        if (lane == 0) mbar_arrive(&sh->empty[r.st]);
        r.next();
      }
      if (j + 1 < steps) {  // keys of the next one
        if (!warp_wait(p, sh, &sh->full[r.st], r.ph)) return;
        if (lane == 0) mbar_arrive(&sh->empty[r.st]);
        r.next();
      }
      if (j < 0) continue;
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        if (j >= it.steps(t)) continue;
        // (not before the step before has been through)
        if (!warp_wait(p, sh, &sh->p_half[t], (count[t] & 1) ^ 1u)) return;
        ++count[t];
        if (lane == 0) mbar_arrive(&sh->p_half[t]);
      }
    }
  }
}

// A tile of 128 rows from its codes: 4 warps, 32 rows each; a lane takes 16 codes (one
// scale) of a key at a time. Neighbouring lanes take one key's codes, so that reads
// do not meet in a bank; of the two 16-byte pieces a lane writes, the upper half of
// a 128-element key swaps the order, so that writes do not either.
// kGuard: the scales of positions pos + .. that are not to count are replaced; true:
// there were NaN among them.
template <int kDim, bool kGuard>
__device__ __forceinline__ bool expand_tile(const uint8_t* raw, uint8_t* tile, int warp, uint32_t there, int all, int any, int pos) {
  using L = Layout<kDim, true>;
  constexpr int kPer = kDim / 16;            // lanes of a key
  constexpr int kRows = 32 / kPer;           // keys of a warp at a time
  const int lane = threadIdx.x & 31, c = lane % kPer, key = lane / kPer;
  const bool swap = kDim == 128 && c >= 4;
  // (row = warp 32 + i kRows + key; what follows from i is known when this is compiled)
  const uint8_t* codes = raw + warp * 2 * L::kHalf + key * (kDim / 2) + c * 8;
  const uint8_t* scales = raw + warp * 2 * L::kHalf + 8 * kDim + key * kPer + c;
  uint8_t* to[2][2];  // first and second piece of rows whose number mod 8 is below and from 4 on (64 elements: one kind)
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int chunk = 2 * c + (h ^ static_cast<int>(swap));
    uint8_t* at = tile + (chunk / 8) * L::kSlab + (warp * 32 + key) * 128;
    to[h][0] = at + ((chunk & 7) ^ key) * 16;
    to[h][1] = at + ((chunk & 7) ^ key ^ 4) * 16;
  }
  bool poison = false;
#pragma unroll
  for (int i = 0; i < 32 / kRows; ++i) {
    const int in = i * kRows;  // of the warp's rows, less key
    const uint2 w = *reinterpret_cast<const uint2*>(codes + (in / 16) * L::kHalf + (in % 16) * (kDim / 2));
    uint32_t b = scales[(in / 16) * L::kHalf + (in % 16) * kPer];
    if (kGuard) {
      const int row = warp * 32 + in + key;
      if (pos + row >= any || !(there >> (row >> 4) & 1u)) b = 0;
      if (pos + row >= all && (b & 0x7Fu) == 0x7Fu) {
        poison = true;
        b = 0;
      }
    }
    const __half2 s = __low2half2(scales2(b));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      __half2 v[4];
      expand_word((h == 1) != swap ? w.y : w.x, v);
      uint4 o;
      o.x = half2_word(__hmul2(v[0], s));
      o.y = half2_word(__hmul2(v[1], s));
      o.z = half2_word(__hmul2(v[2], s));
      o.w = half2_word(__hmul2(v[3], s));
      *reinterpret_cast<uint4*>(to[h][kRows == 4 ? i & 1 : 0] + in * 128) = o;
    }
  }
  return poison;
}

template <int kDim>
__device__ void expand_role(const AttendArgs& p, Shared* sh, const Cut& cut, uint8_t* ring, const uint8_t* raw) {
  using L = Layout<kDim, true>;
  const int warp = (threadIdx.x >> 5) - 12, lane = threadIdx.x & 31;
  Ring<L::kStages> r;
  Ring<L::kRaw> rr;
  int k_step = 0;
  Work work;
  Item it;
  for (int item = -1; work.next(p, sh, cut, &it);) {
    if (it.steps() == 0) continue;
    ++item;
    if (warp == 0 && lane == 0) *reinterpret_cast<volatile int*>(&sh->poison[(item + 8) & 15]) = 0;
    __syncwarp();
    for (int i = 0; i < it.steps(); ++i, ++k_step) {
      const int pos = (it.j0 + i) * kKeys;
#pragma unroll
      for (int v = 0; v < 2; ++v, r.next(), rr.next()) {
        if (!warp_wait(p, sh, &sh->raw_full[rr.st], rr.ph) || !warp_wait(p, sh, &sh->empty[r.st], r.ph ^ 1u)) return;
        const uint8_t* from = raw + rr.st * L::kRawBytes;
        uint8_t* tile = ring + r.st * L::kTileBytes;
        const uint32_t there = *reinterpret_cast<volatile uint32_t*>(&sh->there[k_step & 15]);
        if (v == 0 || (there == 0xFFu && pos + kKeys <= it.all)) {
          expand_tile<kDim, false>(from, tile, warp, there, 0, 0, 0);
        } else if (__any_sync(0xffffffffu, expand_tile<kDim, true>(from, tile, warp, there, it.all, it.any, pos))) {
          if (lane == 0) *reinterpret_cast<volatile int*>(&sh->poison[item & 15]) = 1;
        }
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sh->full[r.st]);
          mbar_arrive(&sh->raw_empty[rr.st]);
        }
      }
    }
  }
}

// The row of Q that a thread of the softmax owns to fp16, scaled by a power of two;
// returns the factor's inverse exponent. Neighbouring threads begin at different
// pieces of 16 bytes: rows are 128 bytes apart, where the same piece of eight rows lies
// in the same banks (6.5 us a tile of 128 elements, of which 32 rows over 131,072
// cached then took 55).
template <int kDim>
__device__ __forceinline__ int convert_row(uint8_t* q, int r) {
  using L = Layout<kDim, true>;
  uint8_t* row = q + r * 128;
  uint32_t top = 0;  // the largest finite magnitude, as bits
#pragma unroll 4
  for (int c = 0; c < kDim / 8; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(row + (c / 8) * L::kSlab + ((c ^ r) % 8) * 16);
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t lo = w[i] << 16 & 0x7FFF0000u, hi = w[i] & 0x7FFF0000u;
      top = max(top, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
    }
  }
  const int e = top != 0 ? ilogbf(__uint_as_float(top)) - 14 : 0;
  const float f0 = scalbnf(1.f, -e / 2), f1 = scalbnf(1.f, -e - -e / 2);  // (2^-e itself may leave fp32's range)
#pragma unroll 4
  for (int c = 0; c < kDim / 8; ++c) {
    uint4* at = reinterpret_cast<uint4*>(row + (c / 8) * L::kSlab + ((c ^ r) % 8) * 16);
    const uint4 x = *at;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = half2_word(__floats2half2_rn(__uint_as_float(w[i] << 16) * f0 * f1, __uint_as_float(w[i] & 0xFFFF0000u) * f0 * f1));
    *at = make_uint4(o[0], o[1], o[2], o[3]);
  }
  return e;
}

// Numerators of 64 scores to tensor memory as 32 columns of pairs; returns their sum.
template <bool kHalf>
__device__ __forceinline__ float numerators(const uint32_t (&s)[2][32], float c, float lift, uint32_t to) {
  uint64_t sum[2] = {0, 0};
  const uint64_t c2 = pack2(c, c), lift2 = pack2(lift, lift);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t w[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      float a, b;
      unpack2(fma2(pack2(__uint_as_float(s[h][2 * k]), __uint_as_float(s[h][2 * k + 1])), c2, lift2), &a, &b);
      a = exp2_fast(a);
      b = exp2_fast(b);
      sum[k & 1] = add2(sum[k & 1], pack2(a, b));
      if (kHalf) {
        w[k] = half2_word(__floats2half2_rn(a, b));
      } else {
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
        w[k] = *reinterpret_cast<const uint32_t*>(&x);
      }
    }
    tmem_st16(to + h * 16, w);
  }
  float a, b;
  unpack2(add2(sum[0], sum[1]), &a, &b);
  return a + b;
}

// Scores of 64 keys from key `at` of the step on that the row does not see: -inf.
__device__ __forceinline__ void mask(uint32_t (&s)[2][32], int at, int left, uint32_t there) {
  asm volatile("");  // a branch, not 64 predicated instructions in every step
#pragma unroll
  for (int i = 0; i < 64; ++i)
    if (at + i >= left || !(there >> ((at + i) / 16) & 1u)) s[i / 32][i % 32] = 0xFF800000u;
}

// The same less the row's base.
__device__ __forceinline__ void rebase(uint32_t (&s)[2][32], float base) {
  asm volatile("");
#pragma unroll
  for (int i = 0; i < 64; ++i) s[i / 32][i % 32] = __float_as_uint(__uint_as_float(s[i / 32][i % 32]) - base);
}

__device__ __forceinline__ float largest(const uint32_t (&s)[2][32]) {
  float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < 32; ++i) top[i & 3] = max3(top[i & 3], __uint_as_float(s[i / 16][2 * i % 32]), __uint_as_float(s[i / 16][2 * i % 32 + 1]));
  return fmaxf(max3(top[0], top[1], top[2]), top[3]);
}

// What look_after (expand_tile) has taken out of V, added to the sums of the rows that
// see it: infinities and NaN. By a whole warp, each lane for its row, whose sums
// begin at o_at. (They stay in tensor memory: an array that a call changes would lie
// in memory for every item, which took 3 us of each.) 32 positions at a time, which the
// lanes share: large blocks leave as many positions as a block has to be gone through, and
// the roles that wait meanwhile give up after two seconds.
template <int kDim, bool kCached>
__device__ __noinline__ void add_odd_values(const AttendArgs& p, const Cut& cut, int k, int lim, uint32_t o_at) {
  const int lane = threadIdx.x & 31;
  Item it;
  locate(p, cut, k, &it);
  const int mine = min(lim, it.j1 * kKeys), begin = max(it.all, it.j0 * kKeys), end = warp_uniform(mine);
#pragma unroll 1
  for (int i = 0; i < kDim / 32; ++i) {
    uint32_t o[1][32];
    tmem_ld32_async(o_at + i * 32, o[0]);
    tmem_wait_ld(o);
    for (int j = begin; j < end; j += 32) {
      const int n = min(32, end - j);
      if (kCached) {
        // a lane looks at a position's scales: which positions have a NaN among these 32 elements
        const uint8_t* six = lane < n ? kv_sixteen(p.a.c, p.a.s, it.seq, it.head, j + lane) : nullptr;
        uint32_t two = 0;
        if (six != nullptr) two = *reinterpret_cast<const uint16_t*>(six + 17 * kDim + (j + lane) % 16 * (kDim / 16) + i * 2);
        const uint32_t see = mine - j >= 32 ? 0xffffffffu : (1u << max(mine - j, 0)) - 1u;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t odd = __ballot_sync(0xffffffffu, (two >> (8 * h) & 0x7F) == 0x7F) & see;
#pragma unroll
          for (int x = 0; x < 16; ++x)
            if (odd != 0) o[0][16 * h + x] = 0x7FC00000u;
        }
      } else {
        // a lane adds up an element's of all these positions, or of those that its row sees
        const uint16_t* v = reinterpret_cast<const uint16_t*>(p.a.v.data + (it.sp.key0 + j) * p.a.v.row + it.head * p.a.v.head) + i * 32;
        auto odd = [&](int y, int x) {
          const uint32_t b = *reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(v + x) + y * p.a.v.row);
          return (b & 0x7F80u) == 0x7F80u ? __uint_as_float(b << 16) : 0.f;
        };
        float sum = 0.f;
#pragma unroll 8
        for (int y = 0; y < n; ++y) sum += odd(y, lane);
        if (!__any_sync(0xffffffffu, sum != 0.f)) continue;
        const bool some = mine > j && mine < j + n, all = mine >= j + n;
#pragma unroll
        for (int x = 0; x < 32; ++x) {
          float add = __shfl_sync(0xffffffffu, sum, x);
          if (some) {
            add = 0.f;
            for (int y = 0; y < mine - j; ++y) add += odd(y, x);
          }
          if (all || some) o[0][x] = __float_as_uint(__uint_as_float(o[0][x]) + add);
        }
      }
    }
    __syncwarp();
    tmem_st32(o_at + i * 32, o[0]);
  }
  tmem_wait_st();
}

// A tile's lift is that of its maximum.
template <int kDim, bool kCached>
__device__ __forceinline__ float lift_of(float m, float c) {
  constexpr float kLift = Layout<kDim, kCached>::kLift;
  return m == -INFINITY || base_of(m, c) != 0.f ? kLift : fmaf(-m, c, kLift);
}

// What sums whose maximum was m are to be multiplied by where it is `to` now.
template <int kDim, bool kCached>
__device__ __forceinline__ float rescaled(float m, float to, float c) {
  if (m == to) return 1.f;
  if (m == -INFINITY) return 0.f;
  return exp2_fast(fmaf(base_of(m, c) - base_of(to, c), c, lift_of<kDim, kCached>(to, c) - lift_of<kDim, kCached>(m, c)));
}

// Where this CTA's tile t keeps row r's sums (four columns of all rows next to one another, as
// the lanes have them), its maximum and sum of weights: of a piece, and those flushed.
__device__ __forceinline__ float4* part_at(const AttendArgs& p, int t, int r, int dim) {
  return reinterpret_cast<float4*>(p.part + (static_cast<int64_t>(blockIdx.x) * 2 + t) * 128 * dim) + r;
}
__device__ __forceinline__ float2* part_ml_at(const AttendArgs& p, int t, int r) { return p.part_ml + (blockIdx.x * 2 + t) * 128 + r; }

// A row's sums to the workspace, where the steps before have left theirs (`more`), and
// zeros in their place.
template <int kDim, bool kCached>
__device__ __noinline__ void flush(const AttendArgs& p, uint32_t o_at, bool more, float m, float l, float c) {
  const uint32_t zeros[16] = {};
  const int t = threadIdx.x >> 7, r = threadIdx.x & 127;
  float4* to = part_at(p, t, r, kDim);
  float2* ml = part_ml_at(p, t, r);
  const float2 before = more ? __ldcg(ml) : make_float2(m, 0.f);
  const float scale = rescaled<kDim, kCached>(before.x, m, c);
  __stcg(ml, make_float2(m, l + before.y * scale));
#pragma unroll 1
  for (int d = 0; d < kDim / 16; ++d) {
    float o[16];
    tmem_ld16(o_at + d * 16, o);
    tmem_st16(o_at + d * 16, zeros);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float4* at = to + (d * 4 + x) * 128;
      const float4 b = more ? __ldcg(at) : make_float4(0.f, 0.f, 0.f, 0.f);
      __stcg(at, make_float4(fmaf(b.x, scale, o[4 * x]), fmaf(b.y, scale, o[4 * x + 1]), fmaf(b.z, scale, o[4 * x + 2]),
                             fmaf(b.w, scale, o[4 * x + 3])));
    }
  }
  tmem_wait_st();
}

// The other way, at the end: what was flushed is added to a row's sums. Returns its sum of weights.
template <int kDim, bool kCached>
__device__ __noinline__ float add_flushed(const AttendArgs& p, uint32_t o_at, float m, float c) {
  const int t = threadIdx.x >> 7, r = threadIdx.x & 127;
  const float4* from = part_at(p, t, r, kDim);
  const float2 before = __ldcg(part_ml_at(p, t, r));
  const float scale = rescaled<kDim, kCached>(before.x, m, c);
#pragma unroll 1
  for (int d = 0; d < kDim / 16; ++d) {
    float o[16];
    uint32_t w[16];
    tmem_ld16(o_at + d * 16, o);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float4 b = __ldcg(from + (d * 4 + x) * 128);
      w[4 * x] = __float_as_uint(fmaf(b.x, scale, o[4 * x]));
      w[4 * x + 1] = __float_as_uint(fmaf(b.y, scale, o[4 * x + 1]));
      w[4 * x + 2] = __float_as_uint(fmaf(b.z, scale, o[4 * x + 2]));
      w[4 * x + 3] = __float_as_uint(fmaf(b.w, scale, o[4 * x + 3]));
    }
    tmem_st16(o_at + d * 16, w);
  }
  tmem_wait_st();
  return before.y * scale;
}

template <int kDim, bool kCached>
__device__ void softmax_role(const AttendArgs& p, Shared* sh, const Cut& cut, int t, uint8_t* q) {
  using L = Layout<kDim, kCached>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x & 127;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t s_at = sh->tmem + kTmemS + t * 128 + lanes, o_at = sh->tmem + kTmemO + t * 128 + lanes;
  const int tok_in = r / p.a.group, head_in = r - tok_in * p.a.group;
  uint32_t s_count = 0, q_count = 0;
  int k_step = 0;
  Work work;
  for (int item = -1;;) {
    // what outlives this block lives in registers beside the scores
    int lim, whole, n, steps, j0;
    bool mine, part;
    int64_t at;  // the row in out and lse
    {
      Item it;
      if (!work.next(p, sh, cut, &it)) break;
      const int tok = it.tok0 + t * p.tokens + tok_in;
      mine = tok_in < p.tokens && tok < it.sp.rows;
      lim = mine ? seen_by(p, it.sp, tok) : 0;
      n = t == 0 ? it.steps(0) : it.steps(1);
      steps = it.steps();
      j0 = it.j0;
      part = it.parts > 1;
      at = static_cast<int64_t>(it.sp.row0 + tok) * p.a.q_heads + it.head * p.a.group + head_in;
    }
    whole = mine ? lim : 0x7fffffff;  // every row of the warp sees the positions below
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) whole = min(whole, __shfl_xor_sync(0xffffffffu, whole, o));
    float c = p.a.scale_log2;
    float m = -INFINITY, l = 0.f;  // m: of S
    // A row's maximum moves by what that row sees alone: a warp scales its rows together, by 1
    // where it does not. (Lanes without a query never ask for it, rows with a base in
    // every step.)
    float lift = L::kLift, gate = mine ? L::kGrowth : INFINITY;
    item += steps > 0;
    if (kCached && n > 0) {
      if (!warp_wait(p, sh, &sh->q_full[t], q_count & 1)) return;
      const int e = convert_row<kDim>(q + t * L::kTileBytes, r);
      c = fminf(fmaxf(scalbnf(c, e), 1.4e-45f), 3.4028234e38f);
      fence_proxy_async_shared();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->q_ready[t]);
    }
    for (int i = 0; i < n; ++i) {
      if (!warp_wait(p, sh, &sh->s_full[t], s_count & 1)) return;
      ++s_count;
      tc_fence_after();
      if (i != 0 && i % kFlush == 0) {
        flush<kDim, kCached>(p, o_at, i != kFlush, m, l, c);
        l = 0.f;
      }
      const int j = j0 + i, left = lim - j * kKeys;
      const uint32_t there = kCached ? *reinterpret_cast<volatile uint32_t*>(&sh->there[(k_step + i) & 15]) : 0xFFu;
      const bool masked = (j + 1) * kKeys > whole || (kCached && there != 0xFFu);
      uint32_t lo[2][32], hi[2][32];
      tmem_ld32_async(s_at, lo[0]);
      tmem_ld32_async(s_at + 32, lo[1]);
      tmem_ld32_async(s_at + 64, hi[0]);
      tmem_ld32_async(s_at + 96, hi[1]);
      tmem_wait_ld(lo);
      if (masked) mask(lo, 0, left, there);
      float top = largest(lo);
      tmem_wait_ld(hi);
      if (masked) mask(hi, 64, left, there);
      top = fmaxf(top, largest(hi));
      const bool grown = (top - m) * c > gate;
      if (__any_sync(0xffffffffu, grown)) {
        const float up = grown ? fmaxf(m, top) : m;
        const float base = base_of(up, c), lift_to = base != 0.f || up == -INFINITY ? L::kLift : fmaf(-up, c, L::kLift);
        const float f = m == up ? 1.f : m == -INFINITY ? 0.f : exp2_fast(fmaf(base_of(m, c) - base, c, lift_to - lift));
        m = up;
        lift = lift_to;
        if (base != 0.f) gate = -INFINITY;
        l *= f;
        if (__any_sync(0xffffffffu, base != 0.f)) {
          rebase(lo, base);
          rebase(hi, base);
        }
        if (i > 0) {
          // (16 columns at a time: 32 beside all the scores leave the registers, cached
          // steps took 3 us instead of 1.7)
#pragma unroll 1
          for (int d = 0; d < kDim / 16; ++d) {
            float o[16];
            uint32_t w[16];
            tmem_ld16(o_at + d * 16, o);
#pragma unroll
            for (int x = 0; x < 16; ++x) w[x] = __float_as_uint(o[x] * f);
            tmem_st16(o_at + d * 16, w);
          }
        }
      }
      l += numerators<kCached>(hi, c, lift, s_at + 32);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_half[t]);
      l += numerators<kCached>(lo, c, lift, s_at);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->p_full[t]);
    }
    k_step += steps;
    if (n > 0) {
      if (!warp_wait(p, sh, &sh->o_full[t], q_count & 1)) return;
      ++q_count;
    }
    tc_fence_after();
    if (n > kFlush) l += add_flushed<kDim, kCached>(p, o_at, m, c);
    const float base = base_of(m, c);
    // (pieces are joined by their m: as if numerators were 2^(c (S - m)))
    const float f = l == 0.f ? 0.f : part ? exp2_fast(fmaf(base - m, c, -lift)) : p.a.c.v_mul / l;
    const int k = piece_at(work.i);
    if (n > 0 && *reinterpret_cast<volatile int*>(&sh->poison[item & 15]) != 0) {
      __syncwarp();
      add_odd_values<kDim, kCached>(p, cut, k, lim, o_at);
    }
    float4* to_part = part_at(p, t, r, kDim);
#pragma unroll 1
    for (int i = 0; i < kDim / 32; ++i) {
      uint32_t o[1][32];
      __syncwarp();
      if (n > 0) {
        tmem_ld32_async(o_at + i * 32, o[0]);
        tmem_wait_ld(o);
      }
#pragma unroll
      for (int x = 0; x < 32; ++x) o[0][x] = n > 0 && f != 0.f ? __float_as_uint(__uint_as_float(o[0][x]) * f) : 0u;
      if (!mine) continue;
      if (part) {
#pragma unroll
        for (int x = 0; x < 8; ++x)
          __stcg(to_part + (i * 8 + x) * 128, make_float4(__uint_as_float(o[0][4 * x]), __uint_as_float(o[0][4 * x + 1]),
                                                          __uint_as_float(o[0][4 * x + 2]), __uint_as_float(o[0][4 * x + 3])));
        continue;
      }
      uint32_t w[2][8];
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        const __nv_bfloat162 y = __floats2bfloat162_rn(__uint_as_float(o[0][2 * x]), __uint_as_float(o[0][2 * x + 1]));
        w[x / 8][x % 8] = *reinterpret_cast<const uint32_t*>(&y);
      }
      store32b(p.a.out + at * kDim + i * 32, p.a.wide_out, w[0]);
      store32b(p.a.out + at * kDim + i * 32 + 16, p.a.wide_out, w[1]);
    }
    __syncwarp();
    if (n > 0) {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->o_empty[t]);
    }
    if (part) {
      __stcg(part_ml_at(p, t, r), make_float2(m, l * f));
      __stcg(&p.part_c[(blockIdx.x * 2 + t) * 128 + r], c);
    } else if (mine && p.a.lse != nullptr) {
      p.a.lse[at] = l == 0.f ? -INFINITY : fmaf(base, c, log2f(l) - lift) * 0.6931471805599453f;
    }
    __syncwarp();
  }
}

}  // namespace

template <int kDim, bool kCached>
__global__ void __launch_bounds__(Layout<kDim, kCached>::kThreads, 1) k_attend(const __grid_constant__ AttendArgs p) {
  using L = Layout<kDim, kCached>;
  extern __shared__ uint8_t smem[];
  uint8_t* q = smem + ((1024u - (smem_u32(smem) & 1023u)) & 1023u);
  uint8_t* ring = q + 2 * L::kTileBytes;
  uint8_t* raw = ring + L::kStages * L::kTileBytes;
  Shared* sh = reinterpret_cast<Shared*>(raw + L::kRaw * L::kRawBytes);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh->q_full[t], 1);
      mbar_init(&sh->q_empty[t], 1);
      mbar_init(&sh->q_ready[t], 4);
      mbar_init(&sh->s_full[t], 1);
      mbar_init(&sh->p_half[t], 5);  // the softmax's warps, and the watch
      mbar_init(&sh->p_full[t], 4);
      mbar_init(&sh->o_full[t], 1);
      mbar_init(&sh->o_empty[t], 4);
    }
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&sh->full[i], kCached ? 4 : 1);   // expanding warps, or the copy
      mbar_init(&sh->empty[i], 2);               // the MMAs that read it, and the watch
    }
    for (int i = 0; i < L::kRaw; ++i) {
      mbar_init(&sh->raw_full[i], 1);
      mbar_init(&sh->raw_empty[i], 4);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    for (int i = 0; i < 16; ++i) sh->poison[i] = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    if (elect_one()) {
      tma_prefetch_desc(&p.tm_q);
      if (!kCached) {
        tma_prefetch_desc(&p.tm_k);
        tma_prefetch_desc(&p.tm_v);
      }
    }
    __syncwarp();
  }
  pdl_wait();
  pdl_trigger();
  const Cut cut = cut_call(p, sh->sums);
  for (int i = warp; i < kItems && piece_at(i) < cut.pieces; i += L::kThreads / 32) {
    Item it;
    if (!locate(p, cut, piece_at(i), &it)) it.parts = 0;
    if (elect_one()) {
      sh->items[i] = it;
      if (i == 0 && cut.chunk != 0)
        p.joins[blockIdx.x] = {it.parts, it.part, it.head, it.sp.row0 + it.tok0, min(2 * p.tokens, it.sp.rows - it.tok0)};
    }
    __syncwarp();
  }
  if (p.may_cut && threadIdx.x == 0 && (cut.chunk == 0 || blockIdx.x >= cut.pieces)) p.joins[blockIdx.x].parts = 0;
  if (blockIdx.x >= cut.pieces) return;  // the whole CTA
  if (warp == 9) {
    tmem_alloc(&sh->tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp < 8) {
    regs_inc<kCached ? 192 : 216>();  // (a warpgroup's share; 8 x 192 + 8 x 64 and 8 x 216 + 4 x 72 are what a CTA has)
    softmax_role<kDim, kCached>(p, sh, cut, warp >> 2, q);
  } else {
    regs_dec<kCached ? 64 : 72>();
    if (warp == 8)
      load_role<kDim, kCached>(p, sh, cut, smem_u32(q), smem_u32(ring), smem_u32(raw));
    else if (warp == 9)
      mma_role<kDim, kCached>(p, sh, cut, smem_u32(q), smem_u32(ring));
    else if (warp == 10)
      watch_role<kDim, kCached>(p, sh, cut, ring);
    else if (kCached && warp >= 12)
      expand_role<kDim>(p, sh, cut, ring, raw);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(sh->tmem, kTmemCols);
  }
}

// The pieces' sums of cut items, joined. Each piece has kJoinCtas CTAs, which with
// those of the item's other pieces share its outputs: four columns of 32 rows to a
// unit of one to eight warps, a row to a lane. The more pieces, the more warps to a
// unit: at most 16 pieces to a warp as a rule, eight of whose loads are in flight
// together; then there are hardly more units than warps for them. (74 pieces of 256
// rows of 128, two items: 20 MB in 5.5 us. Two warps for every unit, 16 loads at a
// time, left most warps without one: 6.8 us.)
constexpr int kJoinCtas = 4, kJoinBatch = 8;

template <int kDim>
__global__ void __launch_bounds__(256, 4) k_attend_join(const __grid_constant__ AttendArgs p) {
  __shared__ float4 s_o[8][32];
  __shared__ float2 s_ml[8][32];
  pdl_wait();
  pdl_trigger();
  const int k = blockIdx.x / kJoinCtas;
  const AttendJoin it = p.joins[k];
  if (it.parts <= 1) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, k0 = k - it.part;
  const int wide = it.parts <= 16 ? 1 : it.parts <= 32 ? 2 : it.parts <= 64 ? 4 : 8;
  const int own = warp & (wide - 1), per = 8 / wide, b0 = it.parts * own / wide, b1 = it.parts * (own + 1) / wide;
  constexpr int kUnits = 8 * (kDim / 4);
  for (int u0 = (it.part * kJoinCtas + blockIdx.x % kJoinCtas) * per; u0 < kUnits; u0 += it.parts * kJoinCtas * per) {
    const int u = u0 + warp / wide;  // (the same number of rounds for all warps of the CTA)
    const int r = (u & 7) * 32 + lane, t = r >> 7, tok_in = (r & 127) / p.a.group, tok = t * p.tokens + tok_in, d4 = u >> 3;
    const bool mine = u < kUnits && tok_in < p.tokens && tok < it.tokens;
    float m = -INFINITY, l = 0.f;
    const float c = mine ? __ldcg(&p.part_c[static_cast<int64_t>(k0) * 256 + r]) : 0.f;  // (of any of them)
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int b = b0; b < b1 && mine; b += kJoinBatch) {
      float2 ml[kJoinBatch];
      float4 v[kJoinBatch];
      float top = m;
#pragma unroll
      for (int x = 0; x < kJoinBatch; ++x) {
        if (b + x >= b1) {
          ml[x] = make_float2(-INFINITY, 0.f);
          v[x] = make_float4(0.f, 0.f, 0.f, 0.f);
          continue;
        }
        const int64_t at = k0 + b + x;
        ml[x] = __ldcg(&p.part_ml[at * 256 + r]);
        v[x] = __ldcg(reinterpret_cast<const float4*>(p.part + (at * 2 + t) * 128 * kDim) + d4 * 128 + (r & 127));
      }
#pragma unroll
      for (int x = 0; x < kJoinBatch; ++x) top = fmaxf(top, ml[x].x);
      const float f = m == top ? 1.f : exp2_fast((m - top) * c);
      m = top;
      l *= f;
      o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
      for (int x = 0; x < kJoinBatch; ++x) {
        const float w = ml[x].x == m ? 1.f : exp2_fast((ml[x].x - m) * c);
        l += w * ml[x].y;
        o.x += w * v[x].x, o.y += w * v[x].y, o.z += w * v[x].z, o.w += w * v[x].w;
      }
    }
    if (wide > 1) {
      s_o[warp][lane] = o;
      s_ml[warp][lane] = make_float2(m, l);
      __syncthreads();
      if (own == 0) {
        for (int x = 1; x < wide; ++x) {
          const float2 other = s_ml[warp + x][lane];
          const float4 v = s_o[warp + x][lane];
          const float top = fmaxf(m, other.x);
          const float f = m == top ? 1.f : exp2_fast((m - top) * c), w = other.x == top ? 1.f : exp2_fast((other.x - top) * c);
          m = top;
          l = l * f + other.y * w;
          o = make_float4(o.x * f + v.x * w, o.y * f + v.y * w, o.z * f + v.z * w, o.w * f + v.w * w);
        }
      }
      __syncthreads();
    }
    if (own == 0 && mine) {
      const int64_t at = static_cast<int64_t>(it.row0 + tok) * p.a.q_heads + it.head * p.a.group + (r & 127) - tok_in * p.a.group;
      if (l == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);
      const float inv = l == 0.f ? 0.f : p.a.c.v_mul / l;
      const __nv_bfloat162 lo = __floats2bfloat162_rn(o.x * inv, o.y * inv), hi = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2*>(p.a.out + at * kDim + d4 * 4) =
          make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
      if (d4 == 0 && p.a.lse != nullptr) p.a.lse[at] = l == 0.f ? -INFINITY : fmaf(m, c, log2f(l)) * 0.6931471805599453f;
    }
  }
}

// Looked up on every call: the address belongs to the current context.
static __device__ __align__(256) uint32_t g_attention_status[64];

cudaError_t attention_shared_status(void** p) { return cudaGetSymbolAddress(p, g_attention_status); }

template <int kDim, bool kCached>
static cudaError_t launch(const AttendArgs& a, int grid, cudaStream_t s) {
  using L = Layout<kDim, kCached>;
  const size_t smem = 1024 + (2 + L::kStages) * static_cast<size_t>(L::kTileBytes) + L::kRaw * L::kRawBytes + sizeof(Shared);
  cudaError_t e = cudaFuncSetAttribute(k_attend<kDim, kCached>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  e = launch_kernel(k_attend<kDim, kCached>, dim3(grid), dim3(L::kThreads), smem, s, true, a);
  if (e != cudaSuccess || !a.may_cut) return e;
  return launch_kernel(k_attend_join<kDim>, dim3(grid * kJoinCtas), dim3(256), 0, s, true, a);
}

cudaError_t launch_attend(const AttendArgs& args, bool cached, int sms, cudaStream_t s) {
  AttendArgs a = args;
  a.a.wide_out = reinterpret_cast<uintptr_t>(a.a.out) % 32 == 0;
  const unsigned per = a.a.c.page_tokens / 16;
  a.per_magic = per <= 1 ? 0u : static_cast<unsigned>(((1ull << 32) + per - 1) / per);
  const int64_t slots = static_cast<int64_t>(a.n_slots) * a.a.c.heads;
  const int grid = a.may_cut || slots > sms ? sms : static_cast<int>(slots);
  if (a.a.c.dim == 64) return cached ? launch<64, true>(a, grid, s) : launch<64, false>(a, grid, s);
  return cached ? launch<128, true>(a, grid, s) : launch<128, false>(a, grid, s);
}

}  // namespace clover
