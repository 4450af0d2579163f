// Attention of few query rows over the paged 4-bit cache (clover_kv_attention of
// single tokens and short runs).
//
// A tile is up to 16 rows: the group's query heads of one or more tokens. Each
// warp expands codes to fp16 in registers (exact: e2m1 times e4m3 has 6
// significant bits and stays below 2^12) and multiplies with mma.sync m16n8k16,
// whose 16 rows the few queries half fill: the tensor core is not what bounds
// this, and no operand passes through shared memory a second time. Queries are
// scaled to fp16 by a power of two per row (the largest element to 2^14, so that
// what falls below fp16's range is 2^-38 of it).
//
// The call's work is one line of units of 384 keys of one tile (32 for each of 12
// warps); every CTA takes an equal piece of it, whatever the lengths are. A
// piece that begins or ends inside a tile leaves its sums in the workspace; the
// last CTA to finish with a tile adds them up, in the order of the keys. Each warp
// streams its own keys through its own ring (one copy per 16 tokens, of codes and
// scales together), on past the ends of tiles.
#include <math.h>

#include "attn_ops.cuh"
#include "launch.cuh"
#include "sm100.cuh"

namespace clover {

namespace {

constexpr int kWarps = 12;
constexpr int kThreads = kWarps * 32;
constexpr int kWarpKeys = 32;  // of a unit: two sixteens
constexpr int kUnit = kWarps * kWarpKeys;
// Numerators are 2^(c S - m + 11), m the row's maximum or up to 2^4 below it: at most
// 2^15, and what fp16 cannot tell from 0 or rounds by more than half a step is
// 2^-36 of the largest.
constexpr float kGrowth = 4.f, kLift = 11.f;

template <int kDim>
struct Layout {
  static constexpr int kSixteen = 18 * kDim;  // bytes: key codes, key scales, value codes, value scales
  static constexpr int kKs = 8 * kDim, kV = 9 * kDim, kVs = 17 * kDim;
  static constexpr int kStage = 2 * kSixteen;
  static constexpr int kStages = kDim == 128 ? 3 : 6;
  static constexpr int kFrag = kDim / 2;  // accumulator registers of a lane
  static constexpr int kPitch = kDim + 4;  // of a row of sums in shared memory: element d at d + d / (kDim / 4)
};

template <int kDim>
struct Shared {
  uint8_t ring[kWarps][Layout<kDim>::kStages][Layout<kDim>::kStage];
  float sums[kWarps / 2][Layout<kDim>::kFrag * 32];
  float2 ml[kWarps][kFewRows];
  float2 row_ml[kFewRows];
  int64_t before[kFewMaxSeqs + 1];  // units of the sequences before
  int64_t scan[kWarps];
  uint64_t full[kWarps][Layout<kDim>::kStages];
  int poison, last;
  uint32_t abort;
};

// Where a warp is in the line of units.
struct Cursor {
  int64_t u;
  int seq, head, tile, unit, units;
  int lim;  // positions from here on are seen by no row of the tile
};

__device__ __forceinline__ int last_seen(const AttendFewArgs& p, const SeqSpan& sp, int tile) {
  const int last = min((tile + 1) * p.tokens, sp.rows) - 1;
  return seen(sp.len - sp.rows + last, sp.len, p.a.block);
}

// Units of a tile: at least one, which writes the rows that see nothing.
__device__ __forceinline__ int units_of(int lim) { return max(1, (lim + kUnit - 1) / kUnit); }

__device__ __forceinline__ int64_t units_of_seq(const AttendFewArgs& p, int i) {
  const SeqSpan sp = seq_span(p.a.s, i);
  int64_t n = 0;
  for (int t = 0; t * p.tokens < sp.rows; ++t) n += units_of(last_seen(p, sp, t));
  return n * p.a.c.heads;
}

template <int kDim>
__device__ void place(const AttendFewArgs& p, const Shared<kDim>& sh, Cursor* c) {
  int lo = 0, hi = p.a.s.n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (sh.before[m] <= c->u)
      lo = m;
    else
      hi = m;
  }
  c->seq = lo;
  const int64_t per_head = (sh.before[lo + 1] - sh.before[lo]) / p.a.c.heads, r = c->u - sh.before[lo];
  c->head = static_cast<int>(r / per_head);
  int left = static_cast<int>(r - c->head * per_head);
  const SeqSpan sp = seq_span(p.a.s, lo);
  for (c->tile = 0;; ++c->tile) {
    c->lim = last_seen(p, sp, c->tile);
    c->units = units_of(c->lim);
    if (left < c->units) break;
    left -= c->units;
  }
  c->unit = left;
}

// The page of lane i's sixteen (i < 2) of the cursor's unit, -1: none.
__device__ __forceinline__ int page_of(const AttendFewArgs& p, const Cursor& c, int pos) {
  if (pos >= c.lim) return -1;
  const int page = p.a.s.table[static_cast<int64_t>(c.seq) * p.a.s.max_pages + pos / p.a.c.page_tokens];
  return page < p.a.c.n_pages ? page : -1;
}

// Four pairs of values of eight codes.
__device__ __forceinline__ void expand(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

__device__ __forceinline__ uint32_t mul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A scale byte, twice, in fp16.
__device__ __forceinline__ uint32_t scale2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b16 x;\n\tcvt.u16.u32 x, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, x;\n\t}" : "=r"(r) : "r"(byte * 0x101u));
  return r;
}

__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// The rows of a tile that a lane holds: g and g + 8.
template <int kDim>
struct Rows {
  uint32_t q[kDim / 16][4];  // elements kDim / 4 * t .. of both rows, four to a step
  float c[2];                // exponent of 2 per unit of the rows' scores
  int lim[2];
  int all;                   // positions below are seen by every row
};

template <int kDim>
__device__ __forceinline__ void load_rows(const AttendFewArgs& p, const Cursor& cu, Rows<kDim>* r) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const SeqSpan sp = seq_span(p.a.s, cu.seq);
  r->all = seen(sp.len - sp.rows + cu.tile * p.tokens, sp.len, p.a.block);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = g + 8 * h, tok_in = row / p.a.group, tok = cu.tile * p.tokens + tok_in;
    const bool mine = tok_in < p.tokens && tok < sp.rows;
    r->lim[h] = mine ? seen(sp.len - sp.rows + tok, sp.len, p.a.block) : 0;
    float v[kDim / 4], top = 0.f;
    if (mine) {
      const uint4* src = reinterpret_cast<const uint4*>(
          p.a.q.data + (sp.row0 + tok) * p.a.q.row + (cu.head * p.a.group + row - tok_in * p.a.group) * p.a.q.head +
          t * (kDim / 2));
#pragma unroll
      for (int i = 0; i < kDim / 32; ++i) {
        const uint4 x = src[i];
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          v[8 * i + 2 * k] = __uint_as_float(w[k] << 16);
          v[8 * i + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kDim / 4; ++i) v[i] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kDim / 4; ++i) {
      const float x = fabsf(v[i]);
      top = fmaxf(top, x < INFINITY ? x : 0.f);
    }
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
    // top 2^-e in [2^14, 2^15)
    const int e = top > 0.f ? ilogbf(top) - 14 : 0;
    r->c[h] = fminf(fmaxf(scalbnf(p.a.scale_log2, e), 1.4e-45f), 3.4028234e38f);
    const float f0 = scalbnf(1.f, -e / 2), f1 = scalbnf(1.f, -e - -e / 2);  // (2^-e itself may leave fp32's range)
#pragma unroll
    for (int i = 0; i < kDim / 4; ++i) v[i] = v[i] * f0 * f1;
#pragma unroll
    for (int i = 0; i < kDim / 16; ++i) {
      r->q[i][h] = half2_bits(v[4 * i], v[4 * i + 1]);
      r->q[i][2 + h] = half2_bits(v[4 * i + 2], v[4 * i + 3]);
    }
  }
}

// Softmax state of a lane's two rows, and its share of their sums: accumulator j
// holds columns 2t and 2t + 1 of the 8 elements j, j + kDim / 8, ...
template <int kDim>
struct State {
  float o[kDim / 8][4];
  float m[2], l[2];
};

// One step of a warp: 32 keys from position pos, whose sixteens with a page are
// `there`. Returns whether a value that some but not all rows see is NaN (it counts
// as 0 here).
template <int kDim, bool kMasked>
__device__ __forceinline__ bool step(const AttendFewArgs& p, const uint8_t* stage, const Rows<kDim>& r, int pos, int any,
                                     uint32_t there, State<kDim>* st) {
  using L = Layout<kDim>;
  constexpr int kWordsK = kDim / 32;  // words of codes of a lane's share of a key
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float s[2][2][4];
#pragma unroll
  for (int x = 0; x < 2; ++x) {
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      const uint8_t* k = stage + x * L::kSixteen;
      const int key = 8 * n + g;
      uint32_t w[kWordsK];
      uint32_t sc[kWordsK];
      if (kDim == 128) {
        const uint4 v = *reinterpret_cast<const uint4*>(k + key * 64 + t * 16);
        w[0] = v.x, w[1] = v.y, w[2 % kWordsK] = v.z, w[3 % kWordsK] = v.w;
        const uint32_t b = *reinterpret_cast<const uint16_t*>(k + L::kKs + key * 8 + 2 * t);
        sc[0] = sc[1] = scale2(b & 0xFFu);
        sc[2 % kWordsK] = sc[3 % kWordsK] = scale2(b >> 8);
      } else {
        const uint2 v = *reinterpret_cast<const uint2*>(k + key * 32 + t * 8);
        w[0] = v.x, w[1] = v.y;
        sc[0] = sc[1] = scale2(k[L::kKs + key * 4 + t]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) s[x][n][i] = 0.f;
#pragma unroll
      for (int i = 0; i < kWordsK; ++i) {
        uint32_t h[4];
        expand(w[i], h);
        mma(s[x][n], r.q[2 * i], mul2(h[0], sc[i]), mul2(h[1], sc[i]));
        mma(s[x][n], r.q[2 * i + 1], mul2(h[2], sc[i]), mul2(h[3], sc[i]));
      }
    }
  }
  if (kMasked) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = pos + 16 * x + 8 * n + 2 * t + (i & 1);
          if (at >= r.lim[i >> 1] || !(there >> x & 1u)) s[x][n][i] = -INFINITY;
        }
  }
  float top[2], base[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float v = -INFINITY;
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < 2; ++n) v = fmaxf(v, fmaxf(s[x][n][2 * h], s[x][n][2 * h + 1]));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
    v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
    top[h] = v * r.c[h];
  }
  if (__any_sync(0xffffffffu, top[0] - st->m[0] > kGrowth || top[1] - st->m[1] > kGrowth)) {
    float f[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float up = fmaxf(st->m[h], top[h]);
      f[h] = st->m[h] == up ? 1.f : exp2_fast(st->m[h] - up);
      st->m[h] = up;
      st->l[h] *= f[h];
    }
#pragma unroll
    for (int j = 0; j < kDim / 8; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) st->o[j][i] *= f[i >> 1];
  }
  base[0] = (st->m[0] == -INFINITY ? 0.f : st->m[0]) - kLift;
  base[1] = (st->m[1] == -INFINITY ? 0.f : st->m[1]) - kLift;
  bool poison = false;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint32_t a[4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float e0 = exp2_fast(fmaf(s[x][n][2 * h], r.c[h], -base[h]));
        const float e1 = exp2_fast(fmaf(s[x][n][2 * h + 1], r.c[h], -base[h]));
        st->l[h] += e0 + e1;
        a[2 * n + h] = half2_bits(e0, e1);
      }
    const uint8_t* v = stage + x * L::kSixteen + L::kV;
    const uint8_t* vs = stage + x * L::kSixteen + L::kVs;
    uint32_t w[4][kDim / 64], sc[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int key = 2 * t + (k & 1) + (k >> 1) * 8;
      uint32_t b;
      if (kDim == 128) {
        const uint2 c = *reinterpret_cast<const uint2*>(v + key * 64 + g * 8);
        w[k][0] = c.x, w[k][kDim / 64 - 1] = c.y;
        b = vs[key * 8 + g];
      } else {
        w[k][0] = *reinterpret_cast<const uint32_t*>(v + key * 32 + g * 4);
        b = vs[key * 4 + g / 2];
      }
      if (kMasked) {
        const int at = pos + 16 * x + key;
        if (at >= any || !(there >> x & 1u)) b = 0;
        if (at >= r.all && (b & 0x7Fu) == 0x7Fu) {
          poison = true;
          b = 0;
        }
      }
      sc[k] = scale2(b);
    }
#pragma unroll
    for (int i = 0; i < kDim / 64; ++i) {
      uint32_t h[4][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        expand(w[k][i], h[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) h[k][e] = mul2(h[k][e], sc[k]);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        mma(st->o[8 * i + 2 * e], a, __byte_perm(h[0][e], h[1][e], 0x5410), __byte_perm(h[2][e], h[3][e], 0x5410));
        mma(st->o[8 * i + 2 * e + 1], a, __byte_perm(h[0][e], h[1][e], 0x7632), __byte_perm(h[2][e], h[3][e], 0x7632));
      }
    }
  }
  return poison;
}

// First unit of CTA c's piece, and the CTA whose piece holds unit u. No more CTAs
// than units have a piece.
__device__ __forceinline__ int64_t pieces(int64_t total) { return min(total, static_cast<int64_t>(gridDim.x)); }
__device__ __forceinline__ int64_t piece(int64_t total, int c) { return total * c / pieces(total); }
__device__ __forceinline__ int piece_of(int64_t total, int64_t u) {
  return static_cast<int>(((u + 1) * pieces(total) - 1) / total);
}

// A row's result from its sum, maximum and weight.
__device__ __forceinline__ void write_row(const AttendFewArgs& p, int64_t at, int dim, int d, float4 o, float inv) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.a.out + at * dim + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void write_lse(const AttendFewArgs& p, int64_t at, float m, float l) {
  if (p.a.lse != nullptr) p.a.lse[at] = l == 0.f ? -INFINITY : (m - kLift + log2f(l)) * 0.6931471805599453f;
}

// The end of a tile's keys in this CTA, by all its threads: the warps' sums
// become one, which is the result or goes to the workspace. units u0 .. u1 - 1 of
// the tile lie here.
template <int kDim>
__device__ void finish(const AttendFewArgs& p, Shared<kDim>* sh, const Cursor& c, int64_t total, int u0, int u1, State<kDim>* st) {
  using L = Layout<kDim>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    st->l[h] += __shfl_xor_sync(0xffffffffu, st->l[h], 1);
    st->l[h] += __shfl_xor_sync(0xffffffffu, st->l[h], 2);
    if (t == 0) sh->ml[warp][g + 8 * h] = make_float2(st->m[h], st->l[h]);
  }
  __syncthreads();
  float f[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    float m = -INFINITY, l = 0.f;
    for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh->ml[w][g + 8 * h].x);
    f[h] = st->m[h] == m ? 1.f : exp2_fast(st->m[h] - m);
    if (warp == 0 && t == 0) {
      for (int w = 0; w < kWarps; ++w) {
        const float2 v = sh->ml[w][g + 8 * h];
        l += v.y * (v.x == m ? 1.f : exp2_fast(v.x - m));
      }
      sh->row_ml[g + 8 * h] = make_float2(m, l);
    }
  }
#pragma unroll
  for (int j = 0; j < kDim / 8; ++j)
#pragma unroll
    for (int i = 0; i < 4; ++i) st->o[j][i] *= f[i >> 1];
  // 12 warps' sums to 6, to 3, to 1: `from` warps from `to` on hand theirs over
  constexpr int kSteps[3][2] = {{6, 6}, {3, 3}, {1, 2}};
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int to = kSteps[k][0], from = kSteps[k][1];
    if (warp >= to && warp < to + from)
#pragma unroll
      for (int i = 0; i < L::kFrag; ++i) sh->sums[warp - to][i * 32 + lane] = st->o[i / 4][i % 4];
    __syncthreads();
    if (k < 2 ? warp < to : warp == 0)
      for (int w = k < 2 ? warp : 0; w < from; w += k < 2 ? from : 1)
#pragma unroll
        for (int i = 0; i < L::kFrag; ++i) st->o[i / 4][i % 4] += sh->sums[w][i * 32 + lane];
    __syncthreads();
  }
  float* rows = sh->sums[0];
  if (warp == 0) {
#pragma unroll
    for (int i = 0; i < L::kFrag; ++i) {
      const int d = (2 * t + (i & 1)) * (kDim / 8) + i / 4;
      rows[(g + (i & 2) * 4) * L::kPitch + d + d / (kDim / 4)] = st->o[i / 4][i % 4];
    }
  }
  __syncthreads();
  const SeqSpan sp = seq_span(p.a.s, c.seq);
  const int n_rows = min(p.tokens, sp.rows - c.tile * p.tokens) * p.a.group;
  const bool whole = u0 == 0 && u1 == c.units;
  const bool poison = sh->poison != 0;
  // (a piece that begins inside a tile keeps that tile's sums in the first of
  // the CTA's two places, one that ends inside a later tile in the second)
  const int64_t first = c.u - c.unit;  // unit 0 of the tile
  const int place0 = 2 * blockIdx.x + (first + u0 == piece(total, blockIdx.x) ? 0 : 1);
  auto row_at = [&](int r) {
    const int tok = r / p.a.group;
    return (static_cast<int64_t>(sp.row0) + c.tile * p.tokens + tok) * p.a.q_heads + c.head * p.a.group + (r - tok * p.a.group);
  };
  for (int i = threadIdx.x; i < n_rows * (kDim / 4); i += kThreads) {
    const int r = i / (kDim / 4), d = i % (kDim / 4) * 4;
    const float* s = rows + r * L::kPitch + d + d / (kDim / 4);
    float4 o = make_float4(s[0], s[1], s[2], s[3]);
    const float2 ml = sh->row_ml[r];
    if (poison) {
      const int tok = c.tile * p.tokens + r / p.a.group, p0 = sp.len - sp.rows;
      const int lo = max(seen(p0 + c.tile * p.tokens, sp.len, p.a.block), u0 * kUnit);
      const int hi = min(seen(p0 + tok, sp.len, p.a.block), u1 * kUnit);
      for (int j = lo; j < hi; ++j) {
        const uint8_t* six = kv_sixteen(p.a.c, p.a.s, c.seq, c.head, j);
        if (six != nullptr && (six[L::kVs + j % 16 * (kDim / 16) + d / 16] & 0x7F) == 0x7F)
          o = make_float4(NAN, NAN, NAN, NAN);
      }
    }
    if (whole) {
      write_row(p, row_at(r), kDim, d, o, ml.y == 0.f ? 0.f : p.a.c.v_mul / ml.y);
      if (d == 0) write_lse(p, row_at(r), ml.x, ml.y);
    } else {
      *reinterpret_cast<float4*>(p.part + (static_cast<int64_t>(place0) * kFewRows + r) * kDim + d) = o;
      if (d == 0) p.part_ml[place0 * kFewRows + r] = ml;
    }
  }
  if (!whole) {
    const int c0 = piece_of(total, first), c1 = piece_of(total, first + c.units - 1);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) sh->last = atomicInc(p.arrived + c0, c1 - c0) == static_cast<uint32_t>(c1 - c0);
    __syncthreads();
    if (sh->last) {
      __threadfence();
      auto place_of = [&](int k) { return 2 * k + (k == c0 && first != piece(total, k) ? 1 : 0); };
      for (int i = threadIdx.x; i < n_rows * (kDim / 4); i += kThreads) {
        const int r = i / (kDim / 4), d = i % (kDim / 4) * 4;
        float m = -INFINITY, l = 0.f;
        for (int k = c0; k <= c1; ++k) m = fmaxf(m, __ldcg(&p.part_ml[place_of(k) * kFewRows + r].x));
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
        for (int k = c0; k <= c1; ++k) {
          const float2 ml = __ldcg(&p.part_ml[place_of(k) * kFewRows + r]);
          const float4 v = __ldcg(reinterpret_cast<const float4*>(
              p.part + (static_cast<int64_t>(place_of(k)) * kFewRows + r) * kDim + d));
          const float w = ml.x == m ? 1.f : exp2_fast(ml.x - m);
          l += w * ml.y;
          o.x += w * v.x, o.y += w * v.y, o.z += w * v.z, o.w += w * v.w;
        }
        write_row(p, row_at(r), kDim, d, o, l == 0.f ? 0.f : p.a.c.v_mul / l);
        if (d == 0) write_lse(p, row_at(r), m, l);
      }
    }
  }
  __syncthreads();  // the buffers are free again
}

}  // namespace

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1) k_attend_few(const __grid_constant__ AttendFewArgs p) {
  using L = Layout<kDim>;
  extern __shared__ __align__(128) uint8_t raw[];
  Shared<kDim>* sh = reinterpret_cast<Shared<kDim>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kWarps * L::kStages) mbar_init(&sh->full[0][0] + threadIdx.x, 1);
  if (threadIdx.x == 0) {
    sh->poison = 0;
    sh->abort = 0;
  }
  fence_mbar_init();
  pdl_wait();
  pdl_trigger();
  // the line of units: three sequences to a thread
  static_assert(3 * kThreads >= kFewMaxSeqs, "every sequence needs a thread");
  int64_t own[3], sum = 0;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int i = 3 * threadIdx.x + k;
    own[k] = i < p.a.s.n ? units_of_seq(p, i) : 0;
    sum += own[k];
  }
  int64_t incl = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) sh->scan[warp] = incl;
  __syncthreads();
  int64_t at = incl - sum, total = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) at += sh->scan[w];
    total += sh->scan[w];
  }
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    const int i = 3 * threadIdx.x + k;
    if (i < p.a.s.n) sh->before[i] = at;
    at += own[k];
    if (i == p.a.s.n - 1) sh->before[i + 1] = at;
  }
  __syncthreads();
  if (blockIdx.x >= pieces(total)) return;
  const int64_t u_begin = piece(total, blockIdx.x), u_end = piece(total, blockIdx.x + 1);

  // the ring: what is fetched next, its page looked up one step ahead
  Cursor f;
  f.u = u_begin;
  place<kDim>(p, *sh, &f);
  Cursor c = f;
  auto pos_of = [&](const Cursor& x) { return x.unit * kUnit + warp * kWarpKeys + (lane & 1) * 16; };
  int page = lane < 2 ? page_of(p, f, pos_of(f)) : -1;
  uint32_t there = 0;  // two bits per stage: sixteens that have a page
  int fs = 0;
  uint32_t fph = 0;  // parity of each stage's last fetch
  bool dead = false;
  auto fetch = [&]() {
    if (f.u >= u_end) return;
    const uint32_t has = __ballot_sync(0xffffffffu, page >= 0) & 3u;
    there = (there & ~(3u << (2 * fs))) | has << (2 * fs);
    fph ^= 1u << fs;
    uint64_t* bar = &sh->full[warp][fs];
    if (lane == 0) mbar_arrive_expect_tx(bar, __popc(has) * L::kSixteen);
    __syncwarp();
    if (page >= 0) {
      const int pos = pos_of(f), per = p.a.c.page_tokens / 16;
      const uint8_t* src = p.a.c.pages + ((static_cast<int64_t>(page) * p.a.c.heads + f.head) * per +
                                          pos % p.a.c.page_tokens / 16) * L::kSixteen;
      bulk_load(smem_u32(sh->ring[warp][fs]) + lane * L::kSixteen, src, L::kSixteen, bar);
    }
    fs = fs + 1 == L::kStages ? 0 : fs + 1;
    if (++f.u < u_end) {
      if (++f.unit == f.units) place<kDim>(p, *sh, &f);
      page = lane < 2 ? page_of(p, f, pos_of(f)) : -1;
    }
  };
  for (int i = 0; i < L::kStages; ++i) fetch();

  State<kDim> st;
  Rows<kDim> rows;
  int s = 0;
  uint32_t ph = 0;
  int u0 = c.unit;
  bool begin = true;
  while (true) {
    if (begin) {
      begin = false;
      u0 = c.unit;
      load_rows<kDim>(p, c, &rows);
#pragma unroll
      for (int j = 0; j < kDim / 8; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) st.o[j][i] = 0.f;
      st.m[0] = st.m[1] = -INFINITY;
      st.l[0] = st.l[1] = 0.f;
    }
    const int pos = c.unit * kUnit + warp * kWarpKeys;
    const uint32_t has = there >> (2 * s) & 3u;
    if (!dead && !__all_sync(0xffffffffu, mbar_wait(&sh->full[warp][s], ph, &sh->abort))) {
      dead = true;
      if (lane == 0) {
        atomicOr(p.a.err, kErrMbarTimeout);
        *reinterpret_cast<volatile uint32_t*>(&sh->abort) = 1u;
      }
    }
    if (pos < c.lim) {
      const uint8_t* stage = sh->ring[warp][s];
      if (has == 3u && pos + kWarpKeys <= rows.all) {
        step<kDim, false>(p, stage, rows, pos, c.lim, has, &st);
      } else if (step<kDim, true>(p, stage, rows, pos, c.lim, has, &st)) {
        *reinterpret_cast<volatile int*>(&sh->poison) = 1;
      }
    }
    __syncwarp();
    if (++s == L::kStages) {
      s = 0;
      ph ^= 1u;
    }
    if (!dead) fetch();
    const bool end = c.u + 1 == u_end;
    if (end || c.unit + 1 == c.units) {
      finish<kDim>(p, sh, c, total, u0, c.unit + 1, &st);
      if (threadIdx.x == 0) sh->poison = 0;
      __syncthreads();
      begin = true;
    }
    if (end) break;
    ++c.u;
    if (++c.unit == c.units) place<kDim>(p, *sh, &c);
  }
  // (the copies in flight must land before the CTA leaves)
  if (dead)
    for (int i = 0; i < L::kStages; ++i) mbar_wait_for(&sh->full[warp][i], (fph >> i & 1u) ^ 1u, 200000000ull);
}

template <int kDim>
static cudaError_t launch(const AttendFewArgs& a, int grid, cudaStream_t s) {
  const cudaError_t e = cudaFuncSetAttribute(k_attend_few<kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             static_cast<int>(sizeof(Shared<kDim>)));
  if (e != cudaSuccess) return e;
  return launch_kernel(k_attend_few<kDim>, dim3(grid), dim3(kThreads), sizeof(Shared<kDim>), s, true, a);
}

cudaError_t launch_attend_few(const AttendFewArgs& a, int grid, cudaStream_t s) {
  return a.a.c.dim == 64 ? launch<64>(a, grid, s) : launch<128>(a, grid, s);
}

}  // namespace clover
