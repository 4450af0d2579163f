// Attention of few query rows over the paged 4-bit cache (clover_kv_attention of
// single tokens and short runs).
//
// A tile is up to 8 or 16 rows: the group's query heads of one or more tokens. Each
// warp expands codes to fp16 in registers (exact: e2m1 times e4m3 has 6
// significant bits and stays below 2^12) and multiplies with mma.sync m16n8k16,
// keys and values on its side of 16 and queries on that of 8: the tensor core is
// not what bounds this, and no operand passes through shared memory a second time.
// Scores come out transposed (a lane holds keys g and g + 8 of rows 2t and 2t + 1),
// and so do the sums; movmatrix turns the numerators between. Queries are scaled to
// fp16 by a power of two per row (the largest element to 2^14, so that what falls
// below fp16's range is 2^-38 of it).
//
// The call's work is one line of units of keys of one tile; every team of warps
// takes an equal piece of it, whatever the lengths are. A team is one warp (units of
// 32 keys) where there are many tiles: nothing waits for another warp. Few tiles
// would then be in too many pieces, so a team is all warps of an SM (32 keys of a
// unit each), whose sums meet in shared memory. A piece that begins or ends inside a
// tile leaves its sums in the workspace; the last team to finish with a tile adds
// them up, in the order of the keys. Each warp streams its own keys through its own
// ring (one copy per 16 tokens, of codes and scales together), on past the ends of
// tiles.
//
// Measured on a GB300 (the kernel alone, in a graph): 64 sequences of 8,192 keys, 32
// heads over 8 of 128: 122 us, 4.9 TB/s of 6.7; of up to 16,384: 123 us. No unit is
// saturated (issue slots 61% busy, ALU 51%, tensor pipe 23%; 315 instructions to a warp for
// 16 tokens, of which expansion takes about half), and warps do not end together: at 107 us
// on average, the last of an SM at 113 and the last of all at 125, when the whole took that.
// One token over 1,021 keys of 2 heads: 13.4 us: 2 to place the work, 2 for the queries and the first keys, 1.5 for
// the step, 6 for the sums of 16 warps and 4 pieces, most of it code that runs once.
#include <math.h>

#include "attn_ops.cuh"
#include "launch.cuh"

namespace clover {

namespace {

constexpr int kWarpKeys = 32;  // of a unit: two sixteens
// Warps of a CTA, one on an SM: what registers allow. (CTAs of four warps that work
// alone, as many on an SM: the later ones are served last and end 20 us after the
// first; 64 sequences of 8,192 keys, 8 heads, took 129 us instead of 123.)
constexpr int few_warps(int cols) { return cols == 1 ? 16 : 12; }
// Numerators are 2^(c (S - m) + 11), m the row's largest S or one that is up to 2^4 less in
// weight: at most 2^15, and what fp16 cannot tell from 0 or rounds by more than half a step
// is 2^-36 of the largest. (The difference comes before the factor: it is exact near the
// maximum however large the scores are. c S - c m is off by the roundings of c m, which
// from scores of 9e7 on are more than fp16 has room for.)
constexpr float kGrowth = 4.f, kLift = 11.f;
// Units of a tile after which its sums go to the workspace, where they are added in fp32, and
// begin again: the tensor core cuts off what its accumulators do not hold, each time it
// adds 16 keys, which after so many (32,768 keys of a warp) has taken 2^-14 of a sum of values
// of one sign, and without an end several % of 2^24.
constexpr int kFlush = 1024;

// kCols: groups of 8 rows.
template <int kDim, int kCols>
struct Layout {
  static constexpr int kSixteen = 18 * kDim;  // bytes: key codes, key scales, value codes, value scales
  static constexpr int kKs = 8 * kDim, kV = 9 * kDim, kVs = 17 * kDim;
  static constexpr int kStage = 2 * kSixteen;
  static constexpr int kStages = (kCols == 1 ? 2 : 3) * (128 / kDim);
  static constexpr int kFrag = kCols * kDim / 4;  // accumulator registers of a lane
  // of a row of sums in shared memory, element d at d + d / (kDim / 8): no bank twice
  static constexpr int kPitch = kDim + 36;
};

template <int kDim, int kCols, int kWarps, int kTeam>
struct Shared {
  uint8_t ring[kWarps][Layout<kDim, kCols>::kStages][Layout<kDim, kCols>::kStage];
  float sums[kTeam > 1 ? kTeam / 2 : 1][kTeam > 1 ? Layout<kDim, kCols>::kFrag * 32 : 1];
  float2 ml[kWarps][kFewRows];
  float2 row_ml[kFewRows];
  float row_c[kFewRows];
  float2 row_f[kFewRows];
  int64_t scan[kWarps];
  uint64_t full[kWarps][Layout<kDim, kCols>::kStages];
  int poison, last;
  uint32_t abort;
  alignas(8) int64_t before[1];  // [sequences + 1] units of the sequences before
};

// Where a warp is in the line of units.
struct Cursor {
  int64_t u;
  int seq, head, tile, unit, units;
  int lim;  // positions from here on are seen by no row of the tile
  SeqSpan sp;
};

__device__ __forceinline__ int last_seen(const AttendFewArgs& p, const SeqSpan& sp, int tile) {
  const int last = min((tile + 1) * p.tokens, sp.rows) - 1;
  return seen(sp.len - sp.rows + last, sp.len, p.a.block);
}

// Units of a tile: at least one, which writes the rows that see nothing.
template <int kTeam>
__device__ __forceinline__ int units_of(int lim) {
  return max(1, (lim + kTeam * kWarpKeys - 1) / (kTeam * kWarpKeys));
}

template <int kTeam>
__device__ __forceinline__ int64_t units_of_seq(const AttendFewArgs& p, int i) {
  const SeqSpan sp = seq_span(p.a.s, i);
  int64_t n = 0;
  for (int t = 0; t * p.tokens < sp.rows; ++t) n += units_of<kTeam>(last_seen(p, sp, t));
  return n * p.a.c.heads;
}

template <int kTeam>
__device__ void place(const AttendFewArgs& p, const int64_t* before, Cursor* c) {
  int lo = 0, hi = p.a.s.n;
  while (hi - lo > 1) {
    const int m = (lo + hi) >> 1;
    if (before[m] <= c->u)
      lo = m;
    else
      hi = m;
  }
  c->seq = lo;
  const int64_t per_head = (before[lo + 1] - before[lo]) / p.a.c.heads, r = c->u - before[lo];
  c->head = static_cast<int>(r / per_head);
  int left = static_cast<int>(r - c->head * per_head);
  c->sp = seq_span(p.a.s, lo);
  for (c->tile = 0;; ++c->tile) {
    c->lim = last_seen(p, c->sp, c->tile);
    c->units = units_of<kTeam>(c->lim);
    if (left < c->units) break;
    left -= c->units;
  }
  c->unit = left;
}

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit values, two of a row to a lane, transposed.
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ uint32_t half2_bits(float a, float b) { return half2_word(__floats2half2_rn(a, b)); }

// What a lane keeps of a tile's rows. As a factor: elements kDim / 4 * t .. of
// rows g and g + 8, four to a step. As results: rows 2t, 2t + 1 (and 8 further).
template <int kDim, int kCols>
struct Rows {
  uint32_t q[kCols][kDim / 16][2];
  float c[kCols][2];  // exponent of 2 per unit of the rows' scores
  int lim[kCols][2];
  int all;            // positions below are seen by every row
};

template <int kDim, int kCols>
__device__ __forceinline__ void load_rows(const AttendFewArgs& p, const Cursor& cu, Rows<kDim, kCols>* r) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const SeqSpan& sp = cu.sp;
  r->all = seen(sp.len - sp.rows + cu.tile * p.tokens, sp.len, p.a.block);
  // the token (of the sequence) of a row, or -1
  auto token = [&](int row) {
    const int in = row / p.a.group, tok = cu.tile * p.tokens + in;
    return in < p.tokens && tok < sp.rows ? tok : -1;
  };
#pragma unroll
  for (int h = 0; h < kCols; ++h) {
    const int row = g + 8 * h, tok = token(row);
    float v[kDim / 4], top = 0.f;
    if (tok >= 0) {
      const uint4* src = reinterpret_cast<const uint4*>(p.a.q.data + (sp.row0 + tok) * p.a.q.row +
                                                        (cu.head * p.a.group + row % p.a.group) * p.a.q.head + t * (kDim / 2));
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
    const float c = fminf(fmaxf(scalbnf(p.a.scale_log2, e), 1.4e-45f), 3.4028234e38f);
    const float f0 = scalbnf(1.f, -e / 2), f1 = scalbnf(1.f, -e - -e / 2);  // (2^-e itself may leave fp32's range)
#pragma unroll
    for (int i = 0; i < kDim / 4; ++i) v[i] = v[i] * f0 * f1;
#pragma unroll
    for (int i = 0; i < kDim / 16; ++i) {
      r->q[h][i][0] = half2_bits(v[4 * i], v[4 * i + 1]);
      r->q[h][i][1] = half2_bits(v[4 * i + 2], v[4 * i + 3]);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      r->c[h][i] = __shfl_sync(0xffffffffu, c, 4 * (2 * t + i));
      const int at = token(8 * h + 2 * t + i);
      r->lim[h][i] = at >= 0 ? seen(sp.len - sp.rows + at, sp.len, p.a.block) : 0;
    }
  }
}

// Softmax state of a lane's rows (m: of S), and its share of their sums: accumulator j holds
// elements kDim / 8 * g + 2 j (registers 0 and 1) and the next (2 and 3).
template <int kDim, int kCols>
struct State {
  float o[kCols][kDim / 16][4];
  float m[kCols][2], l[kCols][2];
};

// One step of a warp: 32 keys from position pos, whose sixteens with a page are
// `there`. Returns whether a value that some but not all rows see is NaN (it counts
// as 0 here).
template <int kDim, int kCols, bool kMasked>
__device__ __forceinline__ bool step(const uint8_t* stage, const Rows<kDim, kCols>& r, int pos, int any, uint32_t there,
                                     State<kDim, kCols>* st) {
  using L = Layout<kDim, kCols>;
  constexpr int kWords = kDim / 32;  // words of codes of a lane's share of a key
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  float s[2][kCols][4];
#pragma unroll
  for (int x = 0; x < 2; ++x)
#pragma unroll
    for (int h = 0; h < kCols; ++h)
#pragma unroll
      for (int i = 0; i < 4; ++i) s[x][h][i] = 0.f;
  {
    uint32_t w[2][2][kWords];
    __half2 sc[2][2];
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int n = 0; n < 2; ++n) {
        const uint8_t* k = stage + x * L::kSixteen;
        const int key = 8 * n + g;
        if constexpr (kDim == 128) {
          const uint4 v = *reinterpret_cast<const uint4*>(k + key * 64 + t * 16);
          w[x][n][0] = v.x, w[x][n][1] = v.y, w[x][n][2] = v.z, w[x][n][3] = v.w;
          sc[x][n] = scales2(*reinterpret_cast<const uint16_t*>(k + L::kKs + key * 8 + 2 * t));
        } else {
          const uint2 v = *reinterpret_cast<const uint2*>(k + key * 32 + t * 8);
          w[x][n][0] = v.x, w[x][n][1] = v.y;
          sc[x][n] = scales2(k[L::kKs + key * 4 + t]);
        }
      }
#pragma unroll
    for (int i = 0; i < kWords; ++i)
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        __half2 h[2][4];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          expand_word(w[x][n][i], h[n]);
          const __half2 f = kDim == 128 && i >= 2 ? __high2half2(sc[x][n]) : __low2half2(sc[x][n]);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[n][e] = __hmul2(h[n][e], f);
        }
#pragma unroll
        for (int c = 0; c < kCols; ++c)
#pragma unroll
          for (int e = 0; e < 2; ++e)
            mma(s[x][c], half2_word(h[0][2 * e]), half2_word(h[1][2 * e]), half2_word(h[0][2 * e + 1]), half2_word(h[1][2 * e + 1]),
                r.q[c][2 * i + e][0], r.q[c][2 * i + e][1]);
      }
  }
  if (kMasked) {
#pragma unroll
    for (int x = 0; x < 2; ++x)
#pragma unroll
      for (int c = 0; c < kCols; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = pos + 16 * x + g + (i >> 1) * 8;
          if (at >= r.lim[c][i & 1] || !(there >> x & 1u)) s[x][c][i] = -INFINITY;
        }
  }
  // each lane's own keys say whether a row's maximum may have grown; only then is it worked
  // out, and moves where it has (what a row gets depends on nothing that other rows see)
  float top[kCols][2], base[kCols][2];
  bool grown = false;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      top[c][i] = fmaxf(fmaxf(s[0][c][i], s[0][c][i + 2]), fmaxf(s[1][c][i], s[1][c][i + 2]));
      grown |= (top[c][i] - st->m[c][i]) * r.c[c][i] > kGrowth;
    }
  if (__any_sync(0xffffffffu, grown)) {
#pragma unroll
    for (int c = 0; c < kCols; ++c)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float up = fmaxf(top[c][i], st->m[c][i]);
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) up = fmaxf(up, __shfl_xor_sync(0xffffffffu, up, o));
        if (!((up - st->m[c][i]) * r.c[c][i] > kGrowth)) up = st->m[c][i];
        const float f = st->m[c][i] == up ? 1.f : exp2_fast((st->m[c][i] - up) * r.c[c][i]);
        st->m[c][i] = up;
        st->l[c][i] *= f;
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j) st->o[c][j][i] *= f, st->o[c][j][i + 2] *= f;
      }
  }
#pragma unroll
  for (int c = 0; c < kCols; ++c)
#pragma unroll
    for (int i = 0; i < 2; ++i) base[c][i] = st->m[c][i] == -INFINITY ? 0.f : st->m[c][i];
  bool poison = false;
#pragma unroll
  for (int x = 0; x < 2; ++x) {
    uint32_t b[kCols][2];
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      float e[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        e[i] = exp2_fast(fmaf(s[x][c][i] - base[c][i & 1], r.c[c][i & 1], kLift));
        st->l[c][i & 1] += e[i];
      }
      b[c][0] = transposed(half2_bits(e[0], e[1]));
      b[c][1] = transposed(half2_bits(e[2], e[3]));
    }
    const uint8_t* v = stage + x * L::kSixteen + L::kV;
    const uint8_t* vs = stage + x * L::kSixteen + L::kVs;
    // two keys' codes side by side in a byte: the pairs that the product takes
    uint32_t w[2][kDim / 64][2];
    __half2 sc[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t u[2][kDim / 64], byte[2];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int key = 2 * t + e + 8 * k;
        if constexpr (kDim == 128) {
          const uint2 x2 = *reinterpret_cast<const uint2*>(v + key * 64 + g * 8);
          u[e][0] = x2.x, u[e][1] = x2.y;
          byte[e] = vs[key * 8 + g];
        } else {
          u[e][0] = *reinterpret_cast<const uint32_t*>(v + key * 32 + g * 4);
          byte[e] = vs[key * 4 + g / 2];
        }
        if (kMasked) {
          const int at = pos + 16 * x + key;
          if (at >= any || !(there >> x & 1u)) byte[e] = 0;
          if (at >= r.all && (byte[e] & 0x7Fu) == 0x7Fu) {
            poison = true;
            byte[e] = 0;
          }
        }
      }
      sc[k] = scales2(byte[0] + byte[1] * 256u);
#pragma unroll
      for (int i = 0; i < kDim / 64; ++i) {
        w[k][i][0] = (u[0][i] & 0x0F0F0F0Fu) | (u[1][i] * 16u & 0xF0F0F0F0u);
        w[k][i][1] = (u[0][i] >> 4 & 0x0F0F0F0Fu) | (u[1][i] & 0xF0F0F0F0u);
      }
    }
#pragma unroll
    for (int i = 0; i < kDim / 64; ++i) {
      __half2 h[2][2][4];
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          expand_word(w[k][i][n], h[k][n]);
#pragma unroll
          for (int e = 0; e < 4; ++e) h[k][n][e] = __hmul2(h[k][n][e], sc[k]);
        }
#pragma unroll
      for (int e = 0; e < 4; ++e)
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          mma(st->o[c][4 * i + e], half2_word(h[0][0][e]), half2_word(h[0][1][e]), half2_word(h[1][0][e]), half2_word(h[1][1][e]), b[c][0], b[c][1]);
    }
  }
  return poison;
}

// The line is cut into as many pieces as there are teams (or units, if those are
// fewer): the first unit of piece k, and the piece that holds unit u.
struct Line {
  int64_t total, pieces;
  __device__ __forceinline__ int64_t first(int k) const { return total * k / pieces; }
  __device__ __forceinline__ int piece_of(int64_t u) const { return static_cast<int>(((u + 1) * pieces - 1) / total); }
};

// Where piece k keeps its sums of the tile that begins at unit `first`: a piece has
// two places, for a tile that began before it and for one that goes on behind it.
__device__ __forceinline__ int place_of(const Line& line, int k, int64_t first) {
  return 2 * k + (first > line.first(k) ? 1 : 0);
}

// Says that this team's sums of the tile of units first .. first + units - 1 are in
// place; true for the last team of them.
__device__ __forceinline__ bool arrive_last(const AttendFewArgs& p, int c0, int c1) {
  __threadfence();
  return atomicInc(p.arrived + c0, c1 - c0) == static_cast<uint32_t>(c1 - c0);
}

// A row's result from its sum, maximum and weight.
__device__ __forceinline__ void write_row(const AttendFewArgs& p, int64_t at, int dim, int d, float4 o, float inv) {
  if (inv == 0.f) o = make_float4(0.f, 0.f, 0.f, 0.f);  // (nothing seen: not even 0 times a NaN)
  const __nv_bfloat162 a = __floats2bfloat162_rn(o.x * inv, o.y * inv), b = __floats2bfloat162_rn(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(p.a.out + at * dim + d) =
      make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}
__device__ __forceinline__ void write_lse(const AttendFewArgs& p, int64_t at, float m, float l, float c) {
  if (p.a.lse != nullptr) p.a.lse[at] = l == 0.f ? -INFINITY : fmaf(m, c, log2f(l) - kLift) * 0.6931471805599453f;
}

// The end of a tile's keys in this CTA, by all its threads: the warps' sums
// become one, which is the result or goes to the workspace. Units u0 .. u1 - 1 of
// the tile lie here, those before v0 in the workspace already; done: it does not go on here. (All sums added up in one step, with two barriers instead of a dozen,
// spilled registers of the loop: one token over 131,072 keys, 8 heads, 50 -> 56 us,
// one over 1,021 13.1 -> 13.0.)
template <int kDim, int kCols, int kWarps>
__device__ void finish_team(const AttendFewArgs& p, Shared<kDim, kCols, kWarps, kWarps>* sh, const Cursor& c, const Line& line,
                            int u0, int v0, int u1, bool done, const Rows<kDim, kCols>& rw, State<kDim, kCols>* st) {
  using L = Layout<kDim, kCols>;
  constexpr int kThreads = kWarps * 32, kUnit = kWarps * kWarpKeys;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
#pragma unroll
  for (int h = 0; h < kCols; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = st->l[h][i];
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
      if (g == 0) sh->ml[warp][8 * h + 2 * t + i] = make_float2(st->m[h][i], l);
    }
  __syncthreads();
#pragma unroll
  for (int h = 0; h < kCols; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 8 * h + 2 * t + i;
      float m = -INFINITY, l = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, sh->ml[w][row].x);
      const float f = st->m[h][i] == m ? 1.f : exp2_fast((st->m[h][i] - m) * rw.c[h][i]);
      if (warp == 0 && g == 0) {
        for (int w = 0; w < kWarps; ++w) {
          const float2 v = sh->ml[w][row];
          l += v.y * (v.x == m ? 1.f : exp2_fast((v.x - m) * rw.c[h][i]));
        }
        sh->row_ml[row] = make_float2(m, l);
        sh->row_c[row] = rw.c[h][i];
      }
#pragma unroll
      for (int j = 0; j < kDim / 16; ++j) st->o[h][j][i] *= f, st->o[h][j][i + 2] *= f;
    }
  // the warps' sums to half as many, and so on (12: 6, 3, 1): those from `to` on hand
  // theirs over, the others add one each, in the last step the first adds all
  float (&acc)[L::kFrag] = *reinterpret_cast<float(*)[L::kFrag]>(&st->o[0][0][0]);
#pragma unroll
  for (int from = kWarps; from > 1; from = from > 3 ? from / 2 : 1) {
    const int to = from > 3 ? from / 2 : 1;
    if (warp >= to && warp < from)
#pragma unroll
      for (int i = 0; i < L::kFrag; ++i) sh->sums[warp - to][i * 32 + lane] = acc[i];
    __syncthreads();
    if (warp < to)
      for (int w = warp; w < from - to; w += to)
#pragma unroll
        for (int i = 0; i < L::kFrag; ++i) acc[i] += sh->sums[w][i * 32 + lane];
    __syncthreads();
  }
  float* rows = sh->sums[0];
  static_assert(8 * kCols * L::kPitch <= kWarps / 2 * L::kFrag * 32, "a tile's rows must fit");
  if (warp == 0) {
#pragma unroll
    for (int h = 0; h < kCols; ++h)
#pragma unroll
      for (int j = 0; j < kDim / 16; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int d = g * (kDim / 8) + 2 * j + (i >> 1);
          rows[(8 * h + 2 * t + (i & 1)) * L::kPitch + d + g] = st->o[h][j][i];
        }
  }
  __syncthreads();
  const SeqSpan& sp = c.sp;
  const int n_rows = min(p.tokens, sp.rows - c.tile * p.tokens) * p.a.group;
  const bool whole = done && u0 == 0 && u1 == c.units, poison = sh->poison != 0;
  const int64_t first = c.u - c.unit;  // unit 0 of the tile
  const int place0 = place_of(line, blockIdx.x, first);
  auto row_at = [&](int r) {
    const int tok = r / p.a.group;
    return (static_cast<int64_t>(sp.row0) + c.tile * p.tokens + tok) * p.a.q_heads + c.head * p.a.group + (r - tok * p.a.group);
  };
  if (v0 != u0) {
    if (threadIdx.x < n_rows) {
      const int r = threadIdx.x;
      const float2 a = sh->row_ml[r], b = __ldcg(&p.part_ml[place0 * kFewRows + r]);
      const float m = fmaxf(a.x, b.x), c = sh->row_c[r];
      const float f = a.x == m ? 1.f : exp2_fast((a.x - m) * c), w = b.x == m ? 1.f : exp2_fast((b.x - m) * c);
      sh->row_ml[r] = make_float2(m, a.y * f + b.y * w);
      sh->row_f[r] = make_float2(f, w);
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < n_rows * (kDim / 4); i += kThreads) {
    const int r = i / (kDim / 4), d = i % (kDim / 4) * 4;
    const float* s = rows + r * L::kPitch + d + d / (kDim / 8);
    float4 o = make_float4(s[0], s[1], s[2], s[3]);
    const float2 ml = sh->row_ml[r];
    if (poison) {
      const int tok = c.tile * p.tokens + r / p.a.group, p0 = sp.len - sp.rows;
      const int lo = max(seen(p0 + c.tile * p.tokens, sp.len, p.a.block), v0 * kUnit);
      const int hi = min(seen(p0 + tok, sp.len, p.a.block), u1 * kUnit);
      for (int j = lo; j < hi; ++j) {
        const uint8_t* six = kv_sixteen(p.a.c, p.a.s, c.seq, c.head, j);
        if (six != nullptr && (six[L::kVs + j % 16 * (kDim / 16) + d / 16] & 0x7F) == 0x7F)
          o = make_float4(NAN, NAN, NAN, NAN);
      }
    }
    if (v0 != u0) {
      const float2 f = sh->row_f[r];
      const float4 b = __ldcg(reinterpret_cast<const float4*>(p.part + (static_cast<int64_t>(place0) * kFewRows + r) * kDim + d));
      o = make_float4(o.x * f.x + b.x * f.y, o.y * f.x + b.y * f.y, o.z * f.x + b.z * f.y, o.w * f.x + b.w * f.y);
    }
    if (whole) {
      write_row(p, row_at(r), kDim, d, o, ml.y == 0.f ? 0.f : p.a.c.v_mul / ml.y);
      if (d == 0) write_lse(p, row_at(r), ml.x, ml.y, sh->row_c[r]);
    } else {
      *reinterpret_cast<float4*>(p.part + (static_cast<int64_t>(place0) * kFewRows + r) * kDim + d) = o;
      if (d == 0) p.part_ml[place0 * kFewRows + r] = ml;
    }
  }
  if (done && !whole) {
    const int c0 = line.piece_of(first), c1 = line.piece_of(first + c.units - 1);
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) sh->last = arrive_last(p, c0, c1);
    __syncthreads();
    if (sh->last) {
      __threadfence();
      const int skip = place_of(line, c0, first) - 2 * c0;
      for (int i = threadIdx.x; i < n_rows * (kDim / 4); i += kThreads) {
        const int r = i / (kDim / 4), d = i % (kDim / 4) * 4;
        float m = -INFINITY, l = 0.f;
        const float c = sh->row_c[r];
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        // kBatch parts at a time, so that their loads are in flight together
        constexpr int kBatch = 8;
        for (int k0 = c0; k0 <= c1; k0 += kBatch) {
          float2 ml[kBatch];
          float4 v[kBatch];
          float top = m;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            const int j = min(k0 + k, c1), at = (2 * j + (j == c0 ? skip : 0)) * kFewRows + r;
            ml[k] = __ldcg(&p.part_ml[at]);
            v[k] = __ldcg(reinterpret_cast<const float4*>(p.part + static_cast<int64_t>(at) * kDim + d));
          }
#pragma unroll
          for (int k = 0; k < kBatch; ++k) top = fmaxf(top, ml[k].x);
          const float f = m == top ? 1.f : exp2_fast((m - top) * c);
          m = top;
          l *= f;
          o.x *= f, o.y *= f, o.z *= f, o.w *= f;
#pragma unroll
          for (int k = 0; k < kBatch; ++k) {
            if (k0 + k > c1) continue;
            const float w = ml[k].x == m ? 1.f : exp2_fast((ml[k].x - m) * c);
            l += w * ml[k].y;
            o.x += w * v[k].x, o.y += w * v[k].y, o.z += w * v[k].z, o.w += w * v[k].w;
          }
        }
        write_row(p, row_at(r), kDim, d, o, l == 0.f ? 0.f : p.a.c.v_mul / l);
        if (d == 0) write_lse(p, row_at(r), m, l, c);
      }
    }
  }
  __syncthreads();  // the buffers are free again
}

// The same for a team of one warp, whose lanes keep their own elements throughout:
// in the workspace a part lies as the lanes hold it.
template <int kDim, int kCols>
__device__ void finish_warp(const AttendFewArgs& p, const Cursor& c, const Line& line, int piece, int u0, int v0, int u1, bool done, bool poison,
                            const Rows<kDim, kCols>& rw, State<kDim, kCols>* st) {
  constexpr int kFrag = Layout<kDim, kCols>::kFrag;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const SeqSpan& sp = c.sp;
  const int n_rows = min(p.tokens, sp.rows - c.tile * p.tokens) * p.a.group;
#pragma unroll
  for (int h = 0; h < kCols; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int o = 4; o < 32; o <<= 1) st->l[h][i] += __shfl_xor_sync(0xffffffffu, st->l[h][i], o);
  if (__any_sync(0xffffffffu, poison)) {
    const int p0 = sp.len - sp.rows, at0 = max(seen(p0 + c.tile * p.tokens, sp.len, p.a.block), v0 * kWarpKeys);
#pragma unroll
    for (int h = 0; h < kCols; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int row = 8 * h + 2 * t + i, tok = c.tile * p.tokens + row / p.a.group;
        const int hi = row < n_rows ? min(seen(p0 + tok, sp.len, p.a.block), u1 * kWarpKeys) : 0;
        for (int j = at0; j < hi; ++j) {
          const uint8_t* six = kv_sixteen(p.a.c, p.a.s, c.seq, c.head, j);
          if (six != nullptr && (six[Layout<kDim, kCols>::kVs + j % 16 * (kDim / 16) + g * (kDim / 8) / 16] & 0x7F) == 0x7F)
#pragma unroll
            for (int k = 0; k < kDim / 16; ++k) st->o[h][k][i] = st->o[h][k][i + 2] = NAN;
        }
      }
    __syncwarp();
  }
  float (&acc)[kFrag] = *reinterpret_cast<float(*)[kFrag]>(&st->o[0][0][0]);
  auto add_part = [&](int at) {
    const float* from = p.part + static_cast<int64_t>(at) * (kFrag * 32) + lane;
    float v[kFrag];
#pragma unroll
    for (int i = 0; i < kFrag; ++i) v[i] = __ldcg(from + i * 32);
#pragma unroll
    for (int h = 0; h < kCols; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float2 ml = __ldcg(&p.part_ml[at * kFewRows + 8 * h + 2 * t + i]);
        const float m = fmaxf(st->m[h][i], ml.x);
        const float f = st->m[h][i] == m ? 1.f : exp2_fast((st->m[h][i] - m) * rw.c[h][i]);
        const float w = ml.x == m ? 1.f : exp2_fast((ml.x - m) * rw.c[h][i]);
        st->m[h][i] = m;
        st->l[h][i] = st->l[h][i] * f + ml.y * w;
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j)
#pragma unroll
          for (int e = i; e < 4; e += 2) st->o[h][j][e] = st->o[h][j][e] * f + v[(h * (kDim / 16) + j) * 4 + e] * w;
      }
  };
  const int64_t first = c.u - c.unit;
  const int mine = place_of(line, piece, first);
  int at0 = mine, parts = v0 != u0, skip = 0;  // what is to be added: its own sums before, then those of all pieces
  for (bool join = false;; join = true) {
#pragma unroll 1
    for (int k = 0; k < parts; ++k) add_part(at0 + 2 * k + (k == 0 ? skip : 0));
    if (join || (done && u0 == 0 && u1 == c.units)) break;
    float* part = p.part + static_cast<int64_t>(mine) * (kFrag * 32) + lane;
#pragma unroll
    for (int i = 0; i < kFrag; ++i) __stcg(part + i * 32, acc[i]);
    if (g == 0)
#pragma unroll
      for (int h = 0; h < kCols; ++h)
#pragma unroll
        for (int i = 0; i < 2; ++i)
          __stcg(&p.part_ml[mine * kFewRows + 8 * h + 2 * t + i], make_float2(st->m[h][i], st->l[h][i]));
    if (!done) {
      __syncwarp();
      return;
    }
    const int c0 = line.piece_of(first), c1 = line.piece_of(first + c.units - 1);
    __threadfence();
    __syncwarp();
    int last = 0;
    if (lane == 0) last = arrive_last(p, c0, c1);
    if (!__shfl_sync(0xffffffffu, last, 0)) return;
    __threadfence();
    at0 = 2 * c0;
    parts = c1 - c0 + 1;
    skip = place_of(line, c0, first) - at0;
#pragma unroll
    for (int h = 0; h < kCols; ++h)
#pragma unroll
      for (int i = 0; i < 2; ++i) st->m[h][i] = -INFINITY, st->l[h][i] = 0.f;
#pragma unroll
    for (int i = 0; i < kFrag; ++i) acc[i] = 0.f;
  }
#pragma unroll
  for (int h = 0; h < kCols; ++h)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int row = 8 * h + 2 * t + i;
      if (row >= n_rows) continue;
      const int tok = row / p.a.group;
      const int64_t at = (static_cast<int64_t>(sp.row0) + c.tile * p.tokens + tok) * p.a.q_heads + c.head * p.a.group +
                         (row - tok * p.a.group);
      const float l = st->l[h][i], inv = l == 0.f ? 0.f : p.a.c.v_mul / l;
      uint32_t w[kDim / 16];
#pragma unroll
      for (int j = 0; j < kDim / 16; ++j) {
        const __nv_bfloat162 x = __floats2bfloat162_rn(st->o[h][j][i] * inv, st->o[h][j][i + 2] * inv);
        w[j] = inv == 0.f ? 0u : *reinterpret_cast<const uint32_t*>(&x);
      }
      uint4* to = reinterpret_cast<uint4*>(p.a.out + at * kDim + g * (kDim / 8));
#pragma unroll
      for (int j = 0; j < kDim / 64; ++j) to[j] = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
      if (g == 0) write_lse(p, at, st->m[h][i], l, rw.c[h][i]);
    }
  __syncwarp();
}

}  // namespace

template <int kDim, int kCols, int kTeam>
__global__ void __launch_bounds__(few_warps(kCols) * 32, 1) k_attend_few(const __grid_constant__ AttendFewArgs p) {
  using L = Layout<kDim, kCols>;
  constexpr int kWarps = few_warps(kCols), kThreads = kWarps * 32, kUnit = kTeam * kWarpKeys;
  extern __shared__ __align__(128) uint8_t raw[];
  auto* sh = reinterpret_cast<Shared<kDim, kCols, kWarps, kTeam>*>(raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x < kWarps * L::kStages) mbar_init(&sh->full[0][0] + threadIdx.x, 1);
  if (threadIdx.x == 0) {
    sh->poison = 0;
    sh->abort = 0;
  }
  fence_mbar_init();
  pdl_wait();
  pdl_trigger();
  // the line of units: `per` neighbouring sequences to a thread
  const int per = (p.a.s.n + kThreads - 1) / kThreads, i0 = threadIdx.x * per, i1 = min(i0 + per, p.a.s.n);
  int64_t sum = 0;
  for (int i = i0; i < i1; ++i) {
    const int64_t n = units_of_seq<kTeam>(p, i);
    sh->before[i] = n;
    sum += n;
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
  for (int i = i0; i < i1; ++i) {
    const int64_t n = sh->before[i];
    sh->before[i] = at;
    at += n;
  }
  if (threadIdx.x == 0) sh->before[p.a.s.n] = total;
  __syncthreads();
  const int piece = kTeam == 1 ? blockIdx.x * kWarps + warp : blockIdx.x;
  const Line line = {total, min(total, static_cast<int64_t>(gridDim.x) * (kWarps / kTeam))};
  if (piece >= line.pieces) return;  // (all of the team)
  const int64_t u_end = line.first(piece + 1);

  // the ring: f is what is fetched next, c what is worked on
  Cursor f;
  f.u = line.first(piece);
  place<kTeam>(p, sh->before, &f);
  Cursor c = f;
  // lane i looks up the i % 2-th sixteen of the warp's keys, i / 2 units on: 16 units
  // of one tile at a time
  int six = -1;   // its place in the pool, in sixteens
  int ahead = 16;  // units of those that are fetched already
  uint32_t there = 0;  // two bits per stage: sixteens that have a page
  int fs = 0, s = 0;
  uint32_t fph = 0, ph = 0;  // parity of each stage's last fetch; of the stages worked on
  bool dead = false, poison = false;
  State<kDim, kCols> st;
  Rows<kDim, kCols> rows;
  // the tile's first unit here (-1: its rows are not loaded), that of the sums so far, and where those end (0: they have not begun)
  int u0 = -1, v0 = 0, v1 = 0;
  for (int warm = L::kStages;;) {
    if (f.u < u_end && !dead) {
      if (ahead == 16) {
        ahead = 0;
        const int i = (f.unit + (lane >> 1)) * (kUnit / 16) + (kTeam == 1 ? 0 : warp * 2) + (lane & 1);
        six = -1;
        if (i * 16 < f.lim) {
          const int of_page = p.a.c.page_tokens / 16, entry = p.per_magic != 0 ? static_cast<int>(__umulhi(i, p.per_magic)) : i;
          const int page = p.a.s.table[static_cast<int64_t>(f.seq) * p.a.s.max_pages + entry];
          if (page >= 0 && page < p.a.c.n_pages) six = (page * p.a.c.heads + f.head) * of_page + (i - entry * of_page);
        }
      }
      const int from = __shfl_sync(0xffffffffu, six, 2 * ahead + (lane & 1));
      const uint32_t has = __ballot_sync(0xffffffffu, from >= 0) & 3u;
      there = (there & ~(3u << (2 * fs))) | has << (2 * fs);
      fph ^= 1u << fs;
      uint64_t* bar = &sh->full[warp][fs];
      if (lane == 0) mbar_arrive_expect_tx(bar, __popc(has) * L::kSixteen);
      __syncwarp();
      if (lane < 2 && from >= 0)
        bulk_load(smem_u32(sh->ring[warp][fs]) + lane * L::kSixteen, p.a.c.pages + static_cast<int64_t>(from) * L::kSixteen,
                  L::kSixteen, bar);
      fs = fs + 1 == L::kStages ? 0 : fs + 1;
      ++ahead;
      if (++f.u < u_end && ++f.unit == f.units) {
        place<kTeam>(p, sh->before, &f);
        ahead = 16;
      }
    }
    if (warm > 0 && --warm > 0) continue;  // fill the ring first
    if (v1 == 0) {
      if (u0 < 0) {
        u0 = c.unit;
        load_rows<kDim, kCols>(p, c, &rows);
      }
      v0 = c.unit;
      v1 = static_cast<int>(min(static_cast<int64_t>(min(c.units - v0, kFlush)), u_end - c.u)) + v0;
      poison = false;
#pragma unroll
      for (int h = 0; h < kCols; ++h) {
#pragma unroll
        for (int j = 0; j < kDim / 16; ++j)
#pragma unroll
          for (int i = 0; i < 4; ++i) st.o[h][j][i] = 0.f;
        st.m[h][0] = st.m[h][1] = -INFINITY;
        st.l[h][0] = st.l[h][1] = 0.f;
      }
    }
    const int pos = c.unit * kUnit + (kTeam == 1 ? 0 : warp * kWarpKeys);
    const uint32_t has = there >> (2 * s) & 3u;
    if (!dead && !__all_sync(0xffffffffu, mbar_wait(&sh->full[warp][s], ph, &sh->abort))) {
      dead = true;
      if (lane == 0) {
        record_timeout(p.a);
        *reinterpret_cast<volatile uint32_t*>(&sh->abort) = 1u;
      }
    }
    if (pos < c.lim) {
      const uint8_t* stage = sh->ring[warp][s];
      if (has == 3u && pos + kWarpKeys <= rows.all)
        step<kDim, kCols, false>(stage, rows, pos, c.lim, has, &st);
      else
        poison |= step<kDim, kCols, true>(stage, rows, pos, c.lim, has, &st);
    }
    __syncwarp();
    if (++s == L::kStages) {
      s = 0;
      ph ^= 1u;
    }
    if (c.unit + 1 == v1) {
      const bool end = c.u + 1 == u_end, done = end || v1 == c.units;
      if constexpr (kTeam == 1) {
        finish_warp<kDim, kCols>(p, c, line, piece, u0, v0, v1, done, poison, rows, &st);
      } else {
        if (poison) *reinterpret_cast<volatile int*>(&sh->poison) = 1;
        finish_team<kDim, kCols, kWarps>(p, sh, c, line, u0, v0, v1, done, rows, &st);
        if (threadIdx.x == 0) sh->poison = 0;
        __syncthreads();
      }
      if (end) break;
      if (done) u0 = -1;
      v1 = 0;
    }
    ++c.u;
    if (++c.unit == c.units) place<kTeam>(p, sh->before, &c);
  }
  // (the copies in flight must land before the CTA leaves)
  if (dead)
    for (int i = 0; i < L::kStages; ++i) mbar_wait_for(&sh->full[warp][i], (fph >> i & 1u) ^ 1u, 200000000ull);
}

template <int kDim, int kCols, int kTeam>
static cudaError_t launch(const AttendFewArgs& a, int sms, cudaStream_t s) {
  void (*k)(const AttendFewArgs) = k_attend_few<kDim, kCols, kTeam>;
  // (the most a call can ask for, in every call: the attribute is the device's, and other host
  // threads may be between theirs and their launch)
  constexpr size_t kBytes = sizeof(Shared<kDim, kCols, few_warps(kCols), kTeam>), kMost = kBytes + 8 * plan::kMaxSeqs;
  static_assert(kMost <= 227 * 1024, "shared memory of a CTA");
  const size_t smem = kBytes + 8 * static_cast<size_t>(a.a.s.n);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMost));
  if (e != cudaSuccess) return e;
  return launch_kernel(k, dim3(sms), dim3(few_warps(kCols) * 32), smem, s, true, a);
}

template <int kDim>
static cudaError_t launch(const AttendFewArgs& a, int sms, bool alone, cudaStream_t s) {
  if (a.tokens * a.a.group <= 8) return alone ? launch<kDim, 1, 1>(a, sms, s) : launch<kDim, 1, few_warps(1)>(a, sms, s);
  return alone ? launch<kDim, 2, 1>(a, sms, s) : launch<kDim, 2, few_warps(2)>(a, sms, s);
}

cudaError_t launch_attend_few(const AttendFewArgs& args, int sms, bool alone, cudaStream_t s) {
  AttendFewArgs a = args;
  const unsigned per = a.a.c.page_tokens / 16;
  a.per_magic = per == 1 ? 0u : static_cast<unsigned>(((1ull << 32) + per - 1) / per);
  return a.a.c.dim == 64 ? launch<64>(a, sms, alone, s) : launch<128>(a, sms, alone, s);
}

}  // namespace clover
