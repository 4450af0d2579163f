// Grouped product of rows and matrices in the microscaled 4-bit formats
// (clover_fp4_product): y = alpha_g A_i . B_g^T, optionally SwiGLU, on the
// block-scaled tensor-core instruction (tcgen05.mma kind::mxf4nvf4).
//
// Persistent, one CTA per SM. A tile is 128 rows of one group x 256 rows of its
// matrix (SwiGLU: 128 gate rows and their 128 up rows, so that one thread
// holds both factors). Roles: warp 0 streams codes (TMA, 128-byte swizzle)
// and scale tiles through a ring of stages of 256 K elements, warp 1 copies each
// stage's scales to tensor memory and issues its four MMAs, warps 4-11 drain the
// accumulator (two per TMEM lane quarter, each every other chunk of 32 columns:
// with one the SwiGLU epilogue of a tile took longer than its MMAs).
//
// Where groups are long, pairs of CTAs take tiles of 256 x 256 (kPair): each
// CTA holds its 128 rows of A and half of B, and the pair's MMA reads both
// halves, so an SM takes in 38 KB per stage instead of 54. The single form's
// rate is that of the SM's L2 port (64 bytes a cycle), not the tensor core's.
//
// What bounds it, measured: few rows per group, HBM (256 rows of 256 experts
// 1,024 x 2,048, SwiGLU: 27.7 us, the 192 MB of the matrices that have rows at
// 7.0 TB/s). 65,536 rows over the same experts: 87 us, 435 MB of DRAM traffic at
// 5.0 TB/s; without its loads 72 us (a tile's MMAs and scale copies take 680
// cycles per stage, and the next tile starts some 700 cycles late, when the
// shared accumulator columns are drained). 8,192^3: 178 us, 6.2 PFLOP/s; without
// the scale copies 168, without the codes' loads 162, without MMAs but one per
// stage and the copies 146: the tensor core spends 492 of 740 cycles per stage in
// MMAs and the 12 scale copies, which it executes in order with them, 190. (The
// "without" figures are of copies of this kernel with that part taken out.)
#include <math.h>

#include "fp4.cuh"
#include "launch.cuh"
#include "moe_ops.cuh"
#include "routing.cuh"
#include "sm100.cuh"

namespace clover {

namespace {

constexpr int kThreads = 384;        // 12 warps
constexpr int kEpilogueWarps = 8;
constexpr int kTileM = 128;          // rows of A per tile
constexpr int kTileN = 256;          // rows of B per tile
constexpr int kStageK = 256;         // K elements per stage: 128 bytes of codes per row
constexpr int kABytes = kTileM * kStageK / 2;
// Scale tiles of a stage: 4 chunks of 64 K elements (NV), 2 of 128 (MX)
constexpr int kMaxChunks = 4;
constexpr int kSfABytes = kMaxChunks * 512;
constexpr int kSfBBytes = 2 * kMaxChunks * 512;
constexpr int kMaxStages = 5;

// A stage of one CTA: A codes, B codes (a pair's CTA: half of them), A's
// scales, all of B's scales.
template <bool kPair>
struct Stage {
  static constexpr int kBBytes = (kPair ? kTileN / 2 : kTileN) * kStageK / 2;
  static constexpr int kSfA = kABytes + kBBytes;
  static constexpr int kSfB = kSfA + kSfABytes;
  static constexpr int kBytes = kSfB + kSfBBytes;
  static constexpr int kCount = kPair ? 5 : 4;
};

// Tensor memory: the accumulators of consecutive tiles are columns 0-255 and
// 192-447: 512 columns do not hold two of 256 and the scales, so they share
// columns 192-255, which the epilogue drains first.
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kAcc1 = 192;
constexpr uint32_t kTmemSfA = 448;
constexpr uint32_t kTmemSfB = kTmemSfA + 4 * kMaxChunks;
static_assert(kTmemSfB + 8 * kMaxChunks <= kTmemCols, "scales must fit behind the accumulators");

struct Shared {
  uint64_t full[kMaxStages], empty[kMaxStages];
  uint64_t acc_full;    // a tile's accumulator is complete
  uint64_t acc_shared;  // the columns it shares with the next one are drained
  uint64_t drain;
  uint32_t tmem;
  uint32_t abort;
  int scan[17];
  int off[kFp4MaxGroups];      // first row of each group
  int cnt[kFp4MaxGroups];      // its rows
  int mt[kFp4MaxGroups + 1];   // row tiles of the groups before it
};

__device__ __forceinline__ void give_up(const Fp4ProductArgs& p, Shared* sh) {
  atomicOr(p.err, kErrMbarTimeout);
  *reinterpret_cast<volatile uint32_t*>(&sh->abort) = 1u;
}

// Tile t, group by group, a group's row tiles in turn, the column tiles of a
// row tile next to one another. A pair's row tile is 256 rows, rank's half of
// it the rows here (none, or fewer than none, where the group ends before).
struct Tile {
  int g;
  int row0, rows;    // first row of A, rows of it that belong to the group
  int64_t sf_tile;   // scale tile of those rows
  int n0;            // first row of the B matrix (SwiGLU: of either half)
  bool only;         // no other row tile reads the matrix
};

// Called by a whole warp.
template <bool kPair>
__device__ __forceinline__ Tile tile_at(const Fp4ProductArgs& p, const Shared& sh, int64_t t, int n_tiles, int step,
                                        int rank) {
  const int m = t <= 0x7fffffff ? static_cast<int>(static_cast<uint32_t>(t) / static_cast<uint32_t>(n_tiles))
                                : static_cast<int>(t / n_tiles);
  const int lo = warp_search(p.n_groups, m, [&](int g) { return sh.mt[g]; });
  Tile r;
  r.g = lo;
  r.only = sh.mt[lo + 1] - sh.mt[lo] == 1;
  const int i = kPair ? 2 * (m - sh.mt[lo]) + rank : m - sh.mt[lo];
  r.row0 = sh.off[lo] + i * kTileM;
  r.rows = min(kTileM, sh.cnt[lo] - i * kTileM);
  r.sf_tile = sh.off[lo] / 128 + static_cast<int64_t>(lo) + i;
  r.n0 = static_cast<int>(t - static_cast<int64_t>(m) * n_tiles) * step;
  return r;
}

// First tile of this CTA (or pair) and the distance to its next one.
template <bool kPair>
__device__ __forceinline__ int64_t first_tile() {
  return kPair ? blockIdx.x / 2 : blockIdx.x;
}
template <bool kPair>
__device__ __forceinline__ int64_t tile_step() {
  return kPair ? gridDim.x / 2 : gridDim.x;
}

// The whole warp waits, so that its control flow stays uniform (the elected
// lane's instructions need the warp converged). False: give up.
__device__ __forceinline__ bool warp_wait(const Fp4ProductArgs& p, Shared* sh, uint64_t* bar, uint32_t parity) {
  if (__all_sync(0xffffffffu, mbar_wait(bar, parity, &sh->abort))) return true;
  if (elect_one()) give_up(p, sh);
  __syncwarp();
  return false;
}

// Run by the whole warp; one elected lane issues. The rate of an SM's copies
// follows their number more than their size, so a stage of a full tile is four:
// A codes, A scales, both halves of B's codes, both halves of B's scales.
template <bool kMx, bool kSwiglu, bool kPair>
__device__ void producer(const Fp4ProductArgs& p, Shared* sh, uint8_t* ring, int64_t n_all, int n_tiles, int rank) {
  using St = Stage<kPair>;
  constexpr int kChunk = kMx ? 128 : 64;       // K elements per scale tile
  constexpr int kChunks = kStageK / kChunk;    // scale tiles of a stage
  // column tiles share A tiles and, where a group has several row tiles, those
  // share B tiles; a matrix that is read once leaves L2 to them (32 tokens x 8:
  // 28.9 -> 27.9 us; evict-first for every B tile costs 8,192 x 8 tokens 87 -> 93)
  const uint64_t pol = l2_policy_evict_last(), pol_once = l2_policy_evict_first();
  const uint32_t ring0 = smem_u32(ring);
  const int nk = (p.K + kStageK - 1) / kStageK;
  int st = 0;
  uint32_t ph = 0, issued = 0, parity_bits = 0;
  bool ok = true;
  for (int64_t t = first_tile<kPair>(); t < n_all && ok; t += tile_step<kPair>()) {
    const Tile tl = tile_at<kPair>(p, *sh, t, n_tiles, kSwiglu ? 128 : 256, rank);
    // a tile with few rows copies only the 32-row boxes that hold some; what
    // the others leave in shared memory reaches only accumulator rows that
    // nobody stores
    const int boxes = kPair || tl.rows > 96 ? 0 : (tl.rows + 31) / 32;
    const uint32_t a_bytes = boxes == 0 ? kABytes : boxes * 4096;
    // SwiGLU: rows n0 .. n0 + 127 of the group's gate and up matrices; else
    // rows n0 .. n0 + 255 of its matrix. Past the matrix: zeros.
    const int mat = kSwiglu ? 2 * tl.g : tl.g;
    const uint64_t pol_b = tl.only ? pol_once : pol;
    for (int k = 0; k < nk; ++k) {
      if (!warp_wait(p, sh, &sh->empty[st], ph ^ 1u)) {
        ok = false;
        break;
      }
      if (elect_one()) {
        uint64_t* bar = &sh->full[st];
        const uint32_t base = ring0 + static_cast<uint32_t>(st) * St::kBytes;
        const uint32_t bytes = a_bytes + St::kBBytes + 3 * kChunks * 512;
        const int sf = k * kChunks * 64, sf_row = static_cast<int>(tl.sf_tile);
        if (kPair) {
          // both CTAs' copies complete on rank 0's barrier, which alone waits
          // for them (the whole boxes: what lies past the group or the tensor
          // does no harm)
          if (rank == 0) mbar_arrive_expect_tx(bar, 2 * bytes);
          const uint32_t bar0 = cluster_map(smem_u32(bar), 0);
          tma_load_2d_pair(base, &p.tm_a, bar0, k * 128, tl.row0, pol);
          tma_load_3d_pair(base + kABytes, &p.tm_b, bar0, k * 128, kSwiglu ? tl.n0 : tl.n0 + rank * 128,
                           kSwiglu ? mat + rank : mat, pol_b);
          tma_load_2d_pair(base + St::kSfA, &p.tm_a_sf, bar0, sf, sf_row, pol);
          tma_load_3d_pair(base + St::kSfB, &p.tm_b_sf, bar0, sf, tl.n0 / 128, mat, pol);
        } else {
          mbar_arrive_expect_tx(bar, bytes);
          if (boxes == 0)
            tma_load_2d(base, &p.tm_a, bar, k * 128, tl.row0, pol);
          else
            for (int b = 0; b < boxes; ++b)
              tma_load_2d(base + b * 4096, &p.tm_a32, bar, k * 128, tl.row0 + b * 32, pol);
          tma_load_3d(base + kABytes, &p.tm_b, bar, k * 128, tl.n0, mat, pol_b);
          tma_load_2d(base + St::kSfA, &p.tm_a_sf, bar, sf, sf_row, pol);
          tma_load_3d(base + St::kSfB, &p.tm_b_sf, bar, sf, tl.n0 / 128, mat, pol);
        }
      }
      __syncwarp();
      issued |= 1u << st;
      parity_bits = (parity_bits & ~(1u << st)) | (ph << st);
      if (++st == St::kCount) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  // the copies in flight must land before the CTA leaves (a pair's rank 1 sees
  // that through the cluster barrier behind rank 0's wait)
  if (*reinterpret_cast<volatile uint32_t*>(&sh->abort) && rank == 0) {
    for (int i = 0; i < St::kCount; ++i)
      if (issued & (1u << i)) mbar_wait_for(&sh->full[i], (parity_bits >> i) & 1u, 200000000ull);
  }
}

// One stage: its scale tiles to tensor memory, then its MMAs (kSteps of 64 K
// elements), issued by the calling thread.
template <bool kMx, bool kPair, int kSteps>
__device__ __forceinline__ void issue_stage(uint32_t base, uint32_t tmem, uint32_t d, uint32_t accumulate) {
  using St = Stage<kPair>;
  constexpr int kPerTile = kMx ? 2 : 1;  // MMAs per scale tile
  const uint32_t sfa = base + St::kSfA, sfb = base + St::kSfB;
#pragma unroll
  for (int c = 0; c < (kSteps + kPerTile - 1) / kPerTile; ++c) {
    tmem_copy_scales<kPair>(tmem + kTmemSfA + c * 4, sfa + c * 512);
    tmem_copy_scales<kPair>(tmem + kTmemSfB + c * 8, sfb + c * 512);
    tmem_copy_scales<kPair>(tmem + kTmemSfB + c * 8 + 4, sfb + (kStageK / (64 * kPerTile) + c) * 512);
  }
  const uint64_t ad = umma_desc_sw128(base), bd = umma_desc_sw128(base + kABytes);
#pragma unroll
  for (int s = 0; s < kSteps; ++s) {
    const int c = s / kPerTile;
    umma_fp4<kMx, kPair>(d, ad + 2 * s, bd + 2 * s,
                         umma_idesc_fp4(kPair ? 2 * kTileM : kTileM, kTileN, kMx, kMx ? (s & 1) * 2 : 0),
                         tmem + kTmemSfA + c * 4, tmem + kTmemSfB + c * 8, s == 0 ? accumulate : 1u);
  }
}

template <bool kPair>
__device__ __forceinline__ void commit(uint64_t* bar) {
  if (kPair)
    umma_commit_pair(bar);
  else
    umma_commit(bar);
}

// Run by the whole warp (of a pair: rank 0's) with uniform control flow; one
// elected lane issues.
template <bool kMx, bool kPair>
__device__ void mma_issuer(const Fp4ProductArgs& p, Shared* sh, uint8_t* ring, int64_t n_all) {
  using St = Stage<kPair>;
  const uint32_t tmem = sh->tmem;
  const uint32_t ring0 = smem_u32(ring);
  const int nk = (p.K + kStageK - 1) / kStageK;
  const int last = (p.K - (nk - 1) * kStageK) / 64;  // MMAs of the last stage, 1 to 4
  int st = 0, it = 0;
  uint32_t ph = 0;
  bool ok = true;
  for (int64_t t = first_tile<kPair>(); t < n_all && ok; t += tile_step<kPair>(), ++it) {
    // the columns shared with the previous tile's accumulator are free once
    // that one's epilogue has drained them, and it drained the tile before
    // that first
    if (it > 0) {
      if (!warp_wait(p, sh, &sh->acc_shared, (it - 1) & 1)) break;
      if (kPair) asm volatile("fence.acq_rel.cluster;" ::: "memory");  // half of the arrivals came from rank 1
    }
    tc_fence_after();
    const uint32_t d = tmem + (it & 1 ? kAcc1 : 0u);
    for (int k = 0; k < nk; ++k) {
      if (!warp_wait(p, sh, &sh->full[st], ph)) {
        ok = false;
        break;
      }
      tc_fence_after();
      const uint32_t base = ring0 + static_cast<uint32_t>(st) * St::kBytes;
      const uint32_t acc = k != 0 ? 1u : 0u;
      if (elect_one()) {
        if (k + 1 < nk || last == 4) {
          issue_stage<kMx, kPair, 4>(base, tmem, d, acc);
        } else if (last == 3) {
          issue_stage<kMx, kPair, 3>(base, tmem, d, acc);
        } else if (last == 2) {
          issue_stage<kMx, kPair, 2>(base, tmem, d, acc);
        } else {
          issue_stage<kMx, kPair, 1>(base, tmem, d, acc);
        }
        commit<kPair>(&sh->empty[st]);
        if (k + 1 == nk) commit<kPair>(&sh->acc_full);
      }
      __syncwarp();
      if (++st == St::kCount) {
        st = 0;
        ph ^= 1u;
      }
    }
  }
  if (elect_one()) {
    if (kPair)
      umma_commit_own_pair(&sh->drain);
    else
      umma_commit(&sh->drain);
  }
  __syncwarp();
  mbar_wait_for(&sh->drain, 0, 200000000ull);
}

// Stores 32 consecutive bf16 of one row, columns c0 .. c0 + 31 of `width`.
__device__ __forceinline__ void store32(__nv_bfloat16* row, int c0, int width, bool vec, const float (&v)[32]) {
  if (vec && c0 + 32 <= width) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 b = __floats2bfloat162_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
        o[i] = *reinterpret_cast<const uint32_t*>(&b);
      }
      *reinterpret_cast<uint4*>(row + c0 + 8 * j) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c0 + j < width) row[c0 + j] = __float2bfloat16_rn(v[j]);
  }
}

// z / (1 + e^-z), below zero as z e^z / (1 + e^z): e^-z would leave fp32's range
// where the result is still an ordinary number.
__device__ __forceinline__ float silu(float z) {
  const float e = __expf(-fabsf(z));
  return __fdividef(z < 0.f ? z * e : z, 1.f + e);
}

template <bool kSwiglu, bool kPair>
__device__ void epilogue(const Fp4ProductArgs& p, Shared* sh, int64_t n_all, int n_tiles, int rank) {
  const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int half = (threadIdx.x >> 7) & 1;  // which of the quarter's two warps
  const bool vec = p.b_rows % 8 == 0;  // rows of y 16-byte aligned
  int it = 0;
  for (int64_t t = first_tile<kPair>(); t < n_all; t += tile_step<kPair>(), ++it) {
    const Tile tl = tile_at<kPair>(p, *sh, t, n_tiles, kSwiglu ? 128 : 256, rank);
    if (!warp_wait(p, sh, &sh->acc_full, it & 1)) return;
    tc_fence_after();
    const bool odd = it & 1;
    const uint32_t acc = sh->tmem + (static_cast<uint32_t>(q * 32) << 16) + (odd ? kAcc1 : 0u);
    const int r = q * 32 + lane;
    const bool on = r < tl.rows;
    const float alpha = p.alpha * (p.group_alpha != nullptr ? p.group_alpha[tl.g] : 1.f);
    __nv_bfloat16* row = p.y + static_cast<int64_t>(tl.row0 + r) * p.b_rows;
    // chunks of 32 columns; the two that hold the shared columns come first
    // (the last two of the even accumulator, the first two of the odd one)
    constexpr int kChunks = kSwiglu ? 4 : 8;
    for (int i = half; i < kChunks; i += 2) {
      const int c = odd ? i : (i + kChunks - 2) % kChunks;
      float v[32], u[kSwiglu ? 32 : 1];
      tmem_ld32(acc + c * 32, v);
      if constexpr (kSwiglu) tmem_ld32(acc + 128 + c * 32, u);
      if (i == half) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          if (kPair)
            mbar_arrive_cluster(cluster_map(smem_u32(&sh->acc_shared), 0));
          else
            mbar_arrive(&sh->acc_shared);
        }
      }
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        v[j] *= alpha;
        if constexpr (kSwiglu) v[j] = silu(v[j]) * (u[j] * alpha);
      }
      if (on) store32(row, tl.n0 + c * 32, p.b_rows, vec, v);
    }
  }
}

}  // namespace

template <bool kMx, bool kSwiglu, bool kPair>
__global__ void __launch_bounds__(kThreads, 1) k_fp4_product(const __grid_constant__ Fp4ProductArgs p) {
  using St = Stage<kPair>;
  extern __shared__ uint8_t raw[];
  uint8_t* ring = raw + ((1024u - (smem_u32(raw) & 1023u)) & 1023u);
  Shared* sh = reinterpret_cast<Shared*>(ring + static_cast<size_t>(St::kCount) * St::kBytes);
  const int warp = threadIdx.x >> 5;
  const int rank = kPair ? static_cast<int>(cluster_rank()) : 0;
  if (threadIdx.x == 0) {
    tma_prefetch_desc(&p.tm_a);
    tma_prefetch_desc(&p.tm_a_sf);
    tma_prefetch_desc(&p.tm_b);
    tma_prefetch_desc(&p.tm_b_sf);
    for (int i = 0; i < St::kCount; ++i) {
      mbar_init(&sh->full[i], 1);
      mbar_init(&sh->empty[i], 1);
    }
    mbar_init(&sh->acc_full, 1);
    mbar_init(&sh->acc_shared, kPair ? 2 * kEpilogueWarps : kEpilogueWarps);
    mbar_init(&sh->drain, 1);
    sh->abort = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    if (kPair) {
      tmem_alloc_pair(&sh->tmem, kTmemCols);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(&sh->tmem, kTmemCols);
      tmem_relinquish();
    }
  }
  pdl_wait();
  pdl_trigger();
  // the groups' rows and row tiles, two groups per thread
  static_assert(2 * kThreads > kFp4MaxGroups, "every group needs a thread");
  int tiles[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int g = 2 * threadIdx.x + j;
    tiles[j] = 0;
    if (g < p.n_groups) {
      const int lo = p.offsets != nullptr ? group_offset(p.offsets, g, p.n_rows) : 0;
      const int hi = p.offsets != nullptr ? group_offset(p.offsets, g + 1, p.n_rows) : p.n_rows;
      sh->off[g] = lo;
      sh->cnt[g] = max(hi - lo, 0);
      constexpr int kRows = kPair ? 2 * kTileM : kTileM;
      tiles[j] = (sh->cnt[g] + kRows - 1) / kRows;
    }
  }
  int m_tiles;
  const int before = block_excl_scan(tiles[0] + tiles[1], sh->scan, &m_tiles);
  if (2 * threadIdx.x <= p.n_groups) sh->mt[2 * threadIdx.x] = before;
  if (2 * threadIdx.x + 1 <= p.n_groups) sh->mt[2 * threadIdx.x + 1] = before + tiles[0];
  // (kThreads covers n_groups itself: the total)
  tc_fence_before();
  if (kPair)
    cluster_sync();  // both CTAs' barriers are set up
  else
    __syncthreads();
  tc_fence_after();
  const int step = kSwiglu ? 128 : 256;
  const int n_tiles = (p.b_rows + step - 1) / step;
  const int64_t n_all = static_cast<int64_t>(m_tiles) * n_tiles;
  if (warp == 0) {
    producer<kMx, kSwiglu, kPair>(p, sh, ring, n_all, n_tiles, rank);
  } else if (warp == 1) {
    if (rank == 0) mma_issuer<kMx, kPair>(p, sh, ring, n_all);
  } else if (warp >= 4) {
    epilogue<kSwiglu, kPair>(p, sh, n_all, n_tiles, rank);
  }
  __syncwarp();
  tc_fence_before();
  if (kPair)
    cluster_sync();  // neither CTA's memory goes away under the other's work
  else
    __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    if (kPair)
      tmem_dealloc_pair(sh->tmem, kTmemCols);
    else
      tmem_dealloc(sh->tmem, kTmemCols);
  }
}

namespace {

template <bool kPair>
cudaError_t launch(const Fp4ProductArgs& a, bool mx, bool swiglu, int grid, cudaStream_t s) {
  void (*k)(const Fp4ProductArgs) =
      mx ? (swiglu ? k_fp4_product<true, true, kPair> : k_fp4_product<true, false, kPair>)
         : (swiglu ? k_fp4_product<false, true, kPair> : k_fp4_product<false, false, kPair>);
  const size_t smem = 1024 + static_cast<size_t>(Stage<kPair>::kCount) * Stage<kPair>::kBytes + sizeof(Shared);
  const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
  if (e != cudaSuccess) return e;
  return launch_kernel(k, dim3(grid), dim3(kThreads), smem, s, true, a, kPair ? 2 : 1);
}

}  // namespace

// Looked up on every call: the address belongs to the current context.
static __device__ __align__(256) uint32_t g_fp4_product_ws[64];

cudaError_t fp4_product_shared(void** p) { return cudaGetSymbolAddress(p, g_fp4_product_ws); }

cudaError_t launch_fp4_product(const Fp4ProductArgs& a, bool mx, bool swiglu, bool pair, int sms, cudaStream_t s) {
  return pair ? launch<true>(a, mx, swiglu, sms / 2 * 2, s) : launch<false>(a, mx, swiglu, sms, s);
}

}  // namespace clover
