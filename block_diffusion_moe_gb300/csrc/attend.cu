// Attention on tensor-core tiles (clover_prompt_attention).
//
// One CTA takes two tiles of 128 query rows (the group's heads of consecutive
// tokens of one sequence) over the keys they see, 128 at a time:
//   S = Q K^T          tcgen05.mma, both operands from shared memory
//   P = 2^(c S - m)    one thread per row: m a running maximum, l the sum of P
//   O = O + P V        tcgen05.mma, P (16 bits) from tensor memory
// and in the end O / l. m moves only where the row's maximum has grown by more
// than 2^8 (O and l are scaled then); until then P is at most 2^8, which costs no
// precision: numerators and sums are floating point.
//
// Roles: warps 0-3 and 4-7 the softmax of tile 0 and 1, warp 8 loads (TMA), warp
// 9 issues the MMAs, warp 10 looks after the values no row may see. While one
// tile's softmax runs, the tensor core works for the other.
#include <math.h>

#include "attn_ops.cuh"
#include "launch.cuh"
#include "sm100.cuh"

namespace clover {

namespace {

constexpr int kThreads = 384;
constexpr int kKeys = 128;  // keys per step
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemS = 0, kTmemO = 256;  // of tile t: + 128 t
constexpr float kGrowth = 8.f;

template <int kDim>
struct Layout {
  static constexpr int kTileBytes = 128 * kDim * 2;  // of Q, of K, of V
  static constexpr int kSlab = 128 * 128;            // 64 elements of 128 rows
  static constexpr int kStages = kDim == 128 ? 5 : 10;
};

struct Shared {
  uint64_t q_full[2], full[10], empty[10];
  uint64_t v_ok[10];  // a stage's values have been looked after
  uint64_t s_full[2], p_full[2], o_full[2];
  uint64_t drain;
  uint32_t tmem, abort;
  int poison;
};

// What a CTA works on.
struct Item {
  SeqSpan sp;
  int head;       // key/value head
  int tok0;       // first token of tile 0 in the sequence; tile t: + t * tokens
  int n[2];       // steps of each tile
  int all, any;   // positions below `all` are seen by every row, none from `any` on
};

__device__ __forceinline__ int seen_by(const AttendArgs& p, const SeqSpan& sp, int tok) {
  return seen(sp.len - sp.rows + tok, sp.len, p.a.block);
}

// Called by a whole warp. False: nothing to do.
__device__ __forceinline__ bool item_of(const AttendArgs& p, Item* it) {
  // the last tiles of a sequence see the most: they begin first
  const int idx = gridDim.x - 1 - blockIdx.x;
  const int slot = idx / p.a.c.heads, pair = 2 * p.tokens;
  it->head = idx - slot * p.a.c.heads;
  const int n = p.a.s.n_rows;
  const int s = warp_search(p.a.s.n, slot, [&](int i) { return group_offset(p.a.s.offsets, i, n) / pair + i; });
  it->sp = seq_span(p.a.s, s);
  it->tok0 = (slot - (it->sp.row0 / pair + s)) * pair;
  if (it->tok0 < 0 || it->tok0 >= it->sp.rows) return false;
  it->any = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int last = min(it->tok0 + (t + 1) * p.tokens, it->sp.rows) - 1;
    const int lim = last < it->tok0 + t * p.tokens ? 0 : seen_by(p, it->sp, last);
    it->n[t] = (lim + kKeys - 1) / kKeys;
    it->any = max(it->any, lim);
  }
  it->all = seen_by(p, it->sp, it->tok0);
  return true;
}

__device__ __forceinline__ bool warp_wait(const AttendArgs& p, Shared* sh, uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_wait(bar, parity, &sh->abort))) return true;
  if (elect_one()) {
    atomicOr(p.a.err, kErrMbarTimeout);
    *reinterpret_cast<volatile uint32_t*>(&sh->abort) = 1u;
  }
  __syncwarp();
  return false;
}

// The ring's stages hold K of step 0, V of step 0, K of step 1, ...
template <int kDim>
struct Ring {
  int st = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ void next(int by = 1) {
    st += by;
    if (st >= Layout<kDim>::kStages) {
      st -= Layout<kDim>::kStages;
      ph ^= 1u;
    }
  }
};

template <int kDim>
__device__ void load_role(const AttendArgs& p, Shared* sh, const Item& it, uint32_t q, uint32_t ring) {
  using L = Layout<kDim>;
  const uint64_t keep = l2_policy_evict_last();
  const int steps = max(it.n[0], it.n[1]);
  if (elect_one()) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (it.n[t] == 0) continue;
      mbar_arrive_expect_tx(&sh->q_full[t], kDim / 64 * p.a.group * p.tokens * 128);
#pragma unroll
      for (int d = 0; d < kDim / 64; ++d)
        tma_load_3d(q + t * L::kTileBytes + d * L::kSlab, &p.tm_q, &sh->q_full[t], d * 64, it.head * p.a.group,
                    it.sp.row0 + it.tok0 + t * p.tokens, keep);
    }
  }
  __syncwarp();
  Ring<kDim> r;
  uint32_t issued = 0, parity = 0;
  for (int i = 0; i < 2 * steps; ++i) {
    if (!warp_wait(p, sh, &sh->empty[r.st], r.ph ^ 1u)) break;
    if (elect_one()) {
      mbar_arrive_expect_tx(&sh->full[r.st], L::kTileBytes);
#pragma unroll
      for (int d = 0; d < kDim / 64; ++d)
        tma_load_3d(ring + r.st * L::kTileBytes + d * L::kSlab, i & 1 ? &p.tm_v : &p.tm_k, &sh->full[r.st], d * 64, it.head,
                    it.sp.key0 + (i >> 1) * kKeys, keep);
    }
    __syncwarp();
    issued |= 1u << r.st;
    parity = (parity & ~(1u << r.st)) | (r.ph << r.st);
    r.next();
  }
  // the copies in flight must land before the CTA leaves
  if (*reinterpret_cast<volatile uint32_t*>(&sh->abort)) {
    for (int i = 0; i < L::kStages; ++i)
      if (issued & (1u << i)) mbar_wait_for(&sh->full[i], (parity >> i) & 1u, 200000000ull);
    for (int t = 0; t < 2; ++t)
      if (it.n[t] > 0) mbar_wait_for(&sh->q_full[t], 0, 200000000ull);
  }
}

template <int kDim>
__device__ void mma_role(const AttendArgs& p, Shared* sh, const Item& it, uint32_t q, uint32_t ring) {
  using L = Layout<kDim>;
  constexpr uint32_t kIdS = umma_idesc_bf16(128, kKeys), kIdO = umma_idesc_bf16(128, kDim) | kUmmaBMnMajor;
  const uint32_t tmem = sh->tmem;
  const int steps = max(it.n[0], it.n[1]);
  const int first_masked = it.all / kKeys;  // steps from here on wait for the values to be looked after
  Ring<kDim> rk, rv;
  rv.next();
  uint32_t v_parity = 0;
  // tile t's scores of step j; the ring's rk holds its keys
  auto scores = [&](int t) {
    if (elect_one()) {
      const uint64_t a = umma_desc_sw128(q + t * L::kTileBytes), b = umma_desc_sw128(ring + rk.st * L::kTileBytes);
#pragma unroll
      for (int s = 0; s < kDim / 16; ++s) {
        const uint32_t o = (s / 4) * (L::kSlab >> 4) + (s % 4) * 2;
        umma_bf16(tmem + kTmemS + t * 128, a + o, b + o, kIdS, s > 0);
      }
      umma_commit(&sh->s_full[t]);
    }
    __syncwarp();
  };
  auto sums = [&](int t, int j) {
    if (elect_one()) {
      const uint64_t b = umma_desc_sw128_mn(ring + rv.st * L::kTileBytes, L::kSlab);
#pragma unroll
      for (int s = 0; s < kKeys / 16; ++s)
        umma_bf16_ta(tmem + kTmemO + t * 128, tmem + kTmemS + t * 128 + s * 8, b + s * 128, kIdO, j > 0 || s > 0);
      if (j + 1 == it.n[t]) umma_commit(&sh->o_full[t]);
    }
    __syncwarp();
  };
  auto release = [&](int st) {
    if (elect_one()) umma_commit(&sh->empty[st]);
    __syncwarp();
  };
  bool ok = true;
  for (int t = 0; t < 2 && ok; ++t)
    if (it.n[t] > 0) ok = warp_wait(p, sh, &sh->q_full[t], 0);
  if (ok) ok = warp_wait(p, sh, &sh->full[rk.st], rk.ph);
  if (ok) {
    tc_fence_after();
    for (int t = 0; t < 2; ++t)
      if (it.n[t] > 0) scores(t);
    release(rk.st);
  }
  for (int j = 0; j < steps && ok; ++j) {
    rk.next(2);
    const bool more = j + 1 < steps;
    ok = warp_wait(p, sh, &sh->full[rv.st], rv.ph);
    if (ok && j >= first_masked) {
      ok = warp_wait(p, sh, &sh->v_ok[rv.st], (v_parity >> rv.st) & 1u);
      v_parity ^= 1u << rv.st;
    }
    if (ok && more) ok = warp_wait(p, sh, &sh->full[rk.st], rk.ph);
    for (int t = 0; t < 2 && ok; ++t) {
      if (j >= it.n[t]) continue;
      ok = warp_wait(p, sh, &sh->p_full[t], j & 1);
      if (!ok) break;
      tc_fence_after();
      sums(t, j);
      if (j + 1 < it.n[t]) scores(t);
    }
    if (!ok) break;
    release(rv.st);
    if (more) release(rk.st);
    rv.next(2);
  }
  if (elect_one()) umma_commit(&sh->drain);
  __syncwarp();
  mbar_wait_for(&sh->drain, 0, 200000000ull);
}

// Values that not every row sees: a weight of 0 does not keep an infinity or a
// NaN out of a sum. Rows of V past every row's sight become zeros, and so do
// infinities and NaN among the others, which the end of the softmax role adds
// to the rows that do see them.
template <int kDim>
__device__ void guard_role(const AttendArgs& p, Shared* sh, const Item& it, uint8_t* ring) {
  using L = Layout<kDim>;
  const int lane = threadIdx.x & 31, steps = max(it.n[0], it.n[1]);
  Ring<kDim> r;
  // every stage in turn, keys and whole steps too: who leaves one out can take a
  // later phase of its barrier for the one it waits for
  for (int i = 0; i < 2 * steps; ++i, r.next()) {
    if (!warp_wait(p, sh, &sh->full[r.st], r.ph)) return;
    const int j = i >> 1;
    if (i % 2 == 0 || (j + 1) * kKeys <= it.all) {
      if (lane == 0) mbar_arrive(&sh->empty[r.st]);
      continue;
    }
    uint8_t* v = ring + r.st * L::kTileBytes;
    const int lo = max(it.all - j * kKeys, 0), hi = min(it.any - j * kKeys, kKeys);
    constexpr int kPer = kDim / 8;  // 16-byte pieces of a row
    uint32_t top = 0;
    const int n = (hi - lo) * kPer;
#pragma unroll 4
    for (int k = lane; k < n; k += 32) {
      const int row = lo + k / kPer, c = k % kPer;
      const uint4 x = *reinterpret_cast<const uint4*>(v + (c / 8) * L::kSlab + row * 128 + (c % 8) * 16);
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
    }
    if (__any_sync(0xffffffffu, (top & 0xFFFFu) >= 0x7F80u || (top >> 16) >= 0x7F80u)) {
      for (int k = lane; k < (hi - lo) * kDim; k += 32) {
        const int row = lo + k / kDim, d = k % kDim;
        uint16_t* x = reinterpret_cast<uint16_t*>(v + (d / 64) * L::kSlab + row * 128 + ((d % 64 / 8) ^ (row & 7)) * 16) + d % 8;
        if ((*x & 0x7F80u) == 0x7F80u) *x = 0;
      }
      if (lane == 0) *reinterpret_cast<volatile int*>(&sh->poison) = 1;
    }
    for (int k = lane; k < (kKeys - hi) * kPer; k += 32) {
      const int row = hi + k / kPer, c = k % kPer;
      *reinterpret_cast<uint4*>(v + (c / 8) * L::kSlab + row * 128 + (c % 8) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async_shared();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&sh->v_ok[r.st]);
      mbar_arrive(&sh->empty[r.st]);
    }
  }
}

template <int kDim>
__device__ void softmax_role(const AttendArgs& p, Shared* sh, const Item& it, int t) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x & 127;
  const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
  const uint32_t s_at = sh->tmem + kTmemS + t * 128 + lanes, o_at = sh->tmem + kTmemO + t * 128 + lanes;
  const int tok_in = r / p.a.group, tok = it.tok0 + t * p.tokens + tok_in;
  const bool mine = tok_in < p.tokens && tok < it.sp.rows;
  const int lim = mine ? seen_by(p, it.sp, tok) : 0;
  int whole = mine ? lim : 0x7fffffff;  // every row of the warp sees the positions below
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) whole = min(whole, __shfl_xor_sync(0xffffffffu, whole, o));
  const float c = p.a.scale_log2;
  float m = -INFINITY, l = 0.f;  // m: of c S
  const int n = it.n[t];
  for (int j = 0; j < n; ++j) {
    if (!warp_wait(p, sh, &sh->s_full[t], j & 1)) return;
    tc_fence_after();
    uint32_t s[4][32];
#pragma unroll
    for (int i = 0; i < 4; ++i) tmem_ld32_async(s_at + i * 32, s[i]);
    tmem_wait_ld(s);
    if ((j + 1) * kKeys > whole) {
      const int left = lim - j * kKeys;
#pragma unroll
      for (int i = 0; i < 128; ++i)
        if (i >= left) s[i / 32][i % 32] = 0xFF800000u;
    }
    float top[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top[i] = __uint_as_float(s[i][0]);
#pragma unroll
      for (int k = 1; k < 32; ++k) top[i] = fmaxf(top[i], __uint_as_float(s[i][k]));
    }
    const float m1 = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * c;
    if (__any_sync(0xffffffffu, m1 - m > kGrowth)) {
      const float up = fmaxf(m, m1);
      const float f = m == up ? 1.f : exp2_fast(m - up);
      m = up;
      l *= f;
      if (j > 0) {
#pragma unroll 1
        for (int i = 0; i < kDim / 32; ++i) {
          uint32_t o[1][32];
          tmem_ld32_async(o_at + i * 32, o[0]);
          tmem_wait_ld(o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[0][k] = __float_as_uint(__uint_as_float(o[0][k]) * f);
          tmem_st32(o_at + i * 32, o[0]);
        }
      }
    }
    const float base = m == -INFINITY ? 0.f : m;
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t w[32];
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const int i = 64 * h + 2 * k;
        const float a = exp2_fast(fmaf(__uint_as_float(s[i / 32][i % 32]), c, -base));
        const float b = exp2_fast(fmaf(__uint_as_float(s[(i + 1) / 32][(i + 1) % 32]), c, -base));
        sum[(2 * k) & 3] += a;
        sum[(2 * k + 1) & 3] += b;
        const __nv_bfloat162 x = __floats2bfloat162_rn(a, b);
        w[k] = *reinterpret_cast<const uint32_t*>(&x);
      }
      tmem_st32(s_at + h * 32, w);
    }
    tmem_wait_st();
    l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&sh->p_full[t]);
  }
  if (n > 0 && !warp_wait(p, sh, &sh->o_full[t], 0)) return;
  tc_fence_after();
  const int64_t at = (static_cast<int64_t>(it.sp.row0 + tok) * p.a.q_heads + it.head * p.a.group + (r - tok_in * p.a.group));
  const float inv = l == 0.f ? 0.f : p.a.c.v_mul / l;
  const bool poison = *reinterpret_cast<volatile int*>(&sh->poison) != 0;
#pragma unroll 1
  for (int i = 0; i < kDim / 32; ++i) {
    uint32_t o[1][32];
    __syncwarp();
    if (n > 0) {
      tmem_ld32_async(o_at + i * 32, o[0]);
      tmem_wait_ld(o);
    }
#pragma unroll
    for (int k = 0; k < 32; ++k) o[0][k] = n > 0 ? __float_as_uint(__uint_as_float(o[0][k]) * inv) : 0u;
    if (!mine) continue;
    if (poison) {
      for (int j = it.all; j < lim; ++j) {
        const uint16_t* v = reinterpret_cast<const uint16_t*>(p.a.v.data + (it.sp.key0 + j) * p.a.v.row + it.head * p.a.v.head);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
          const uint32_t x = v[i * 32 + k];
          if ((x & 0x7F80u) == 0x7F80u) o[0][k] = __float_as_uint(__uint_as_float(o[0][k]) + __uint_as_float(x << 16));
        }
      }
    }
    uint32_t w[2][8];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(__uint_as_float(o[0][2 * k]), __uint_as_float(o[0][2 * k + 1]));
      w[k / 8][k % 8] = *reinterpret_cast<const uint32_t*>(&x);
    }
    store32b(p.a.out + at * kDim + i * 32, p.a.wide_out, w[0]);
    store32b(p.a.out + at * kDim + i * 32 + 16, p.a.wide_out, w[1]);
  }
  if (mine && p.a.lse != nullptr) p.a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
}

}  // namespace

template <int kDim>
__global__ void __launch_bounds__(kThreads, 1) k_attend(const __grid_constant__ AttendArgs p) {
  using L = Layout<kDim>;
  extern __shared__ uint8_t raw[];
  uint8_t* q = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  uint8_t* ring = q + 2 * L::kTileBytes;
  Shared* sh = reinterpret_cast<Shared*>(ring + L::kStages * L::kTileBytes);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&sh->q_full[t], 1);
      mbar_init(&sh->s_full[t], 1);
      mbar_init(&sh->p_full[t], 4);
      mbar_init(&sh->o_full[t], 1);
    }
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 2);  // the MMAs that read it, and the guard
      mbar_init(&sh->v_ok[i], 1);
    }
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    sh->poison = 0;
    fence_mbar_init();
  }
  if (warp == 8) {
    if (elect_one()) {
      tma_prefetch_desc(&p.tm_q);
      tma_prefetch_desc(&p.tm_k);
      tma_prefetch_desc(&p.tm_v);
    }
    __syncwarp();
  }
  pdl_wait();
  pdl_trigger();
  Item it;
  if (!item_of(p, &it)) return;  // the whole CTA
  if (warp == 9) {
    tmem_alloc(&sh->tmem, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp < 8) {
    regs_inc<216>();
    softmax_role<kDim>(p, sh, it, warp >> 2);
  } else {
    regs_dec<72>();
    if (warp == 8)
      load_role<kDim>(p, sh, it, smem_u32(q), smem_u32(ring));
    else if (warp == 9 && max(it.n[0], it.n[1]) > 0)
      mma_role<kDim>(p, sh, it, smem_u32(q), smem_u32(ring));
    else if (warp == 10)
      guard_role<kDim>(p, sh, it, ring);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(sh->tmem, kTmemCols);
  }
}

template <int kDim>
static cudaError_t launch(const AttendArgs& a, cudaStream_t s) {
  using L = Layout<kDim>;
  const size_t smem = 1024 + (2 + L::kStages) * static_cast<size_t>(L::kTileBytes) + sizeof(Shared);
  const cudaError_t e = cudaFuncSetAttribute(k_attend<kDim>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_kernel(k_attend<kDim>, dim3(static_cast<unsigned>(a.n_slots) * a.a.c.heads), dim3(kThreads), smem, s, true, a);
}

cudaError_t launch_attend(const AttendArgs& args, cudaStream_t s) {
  AttendArgs a = args;
  a.a.wide_out = reinterpret_cast<uintptr_t>(a.a.out) % 32 == 0;
  return a.a.c.dim == 64 ? launch<64>(a, s) : launch<128>(a, s);
}

}  // namespace clover
