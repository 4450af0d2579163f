// Writing rows of keys and values to the paged 4-bit cache and reading them
// back (clover_kv_write, clover_kv_read).
#include "attn_ops.cuh"
#include "launch.cuh"

namespace clover {

namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 4;              // blocks of 16 elements that a thread has in flight
constexpr int kBatch = kThreads * kUnroll;
constexpr int kMaxRows = kBatch / 8;    // rows of a CTA: a row has at least 8 blocks

// Where a row's sixteen of head 0 begins, and the row in it; six < 0: outside the
// cache (no page, or a negative position), -2: of no sequence.
struct RowPlace {
  int64_t six;
  int in;
};

__device__ __forceinline__ RowPlace place_row(const KvCopyArgs& a, int row) {
  RowPlace r = {-2, 0};
  const int q = seq_of_row(a.s, row);
  if (q < 0) return r;
  const SeqSpan sp = seq_span(a.s, q);
  if (row >= sp.row0 + sp.rows) return r;
  r.six = -1;
  const int p = sp.len - sp.rows + (row - sp.row0);
  if (p < 0) return r;
  const int slot = p / a.c.page_tokens, page = a.s.table[static_cast<int64_t>(q) * a.s.max_pages + slot];
  if (page < 0 || page >= a.c.n_pages) return r;
  const int in_page = p - slot * a.c.page_tokens;
  r.six = static_cast<int64_t>(page) * a.c.heads * (a.c.page_tokens / 16) + in_page / 16;
  r.in = in_page % 16;
  return r;
}

// Block i of a CTA's: of which of its rows, keys or values, head, block of the head.
struct Block {
  int row, head, block;
  bool value;
};

template <int kDim>
__device__ __forceinline__ Block block_of(const KvCopyArgs& a, int i) {
  constexpr int kPer = kDim / 16;
  const int per_row = 2 * a.c.heads * kPer;
  Block b;
  b.row = a.row_magic != 0 ? static_cast<int>(__umulhi(i, a.row_magic)) : i / per_row;
  i -= b.row * per_row;
  b.value = i >= per_row / 2;
  i -= b.value ? per_row / 2 : 0;
  b.head = i / kPer;
  b.block = i % kPer;
  return b;
}

template <int kDim>
__device__ __forceinline__ uint8_t* codes_of(const KvCopyArgs& a, const RowPlace& p, const Block& b, uint8_t** scale) {
  uint8_t* six = a.c.pages + (p.six + static_cast<int64_t>(b.head) * (a.c.page_tokens / 16)) * (18 * kDim) + (b.value ? 9 * kDim : 0);
  *scale = six + 8 * kDim + p.in * (kDim / 16) + b.block;
  return six + p.in * (kDim / 2) + b.block * 8;
}

}  // namespace

// x = code * scale * 2^exp in blocks of 16: the scale is the block's largest magnitude
// over 6, rounded to e4m3, the codes x over it, rounded to e2m1. Both kernels move bytes:
// HBM bounds them. A CTA takes as many rows as make about 1,024 blocks of 16 elements;
// their places are looked up once, and each thread has the loads of four blocks in
// flight. (With each thread looking up its block's place, 131,072 rows of 2 heads of
// 128 took 46 us to read, and 29 so: 5.9 TB/s. 6,646 rows of 8 heads, written and
// read back: 19 us, 2.9 TB/s, of which two launches are 5.)
template <int kDim, bool kBf16>
__global__ void __launch_bounds__(kThreads) k_kv_write(const KvCopyArgs a) {
  __shared__ float s_inv[2][128];
  __shared__ RowPlace s_place[kMaxRows];
  if (kBf16) {
    const int i = threadIdx.x;
    s_inv[i >> 7][i & 127] = scale_inverse(i & 127, i < 128 ? a.c.k_mul : a.c.v_mul);
  }
  pdl_wait();
  pdl_trigger();
  const int row0 = blockIdx.x * a.cta_rows, rows = min(a.cta_rows, a.s.n_rows - row0);
  constexpr int kSize = kBf16 ? 2 : 4, kWords = 4 * kSize;
  const int n = rows * 2 * a.c.heads * (kDim / 16);
  for (int base = 0; base < n; base += kBatch) {  // (mostly once)
    const int i0 = base + threadIdx.x;
    uint32_t in[kUnroll][kWords];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= n) continue;
      const Block b = block_of<kDim>(a, i);
      const AttnRows& x = b.value ? a.v : a.k;
      const uint8_t* src = x.data + (row0 + b.row) * x.row + b.head * x.head + b.block * (16 * kSize);
#pragma unroll
      for (int v = 0; v < kSize / 2; ++v) load32b(src + v * 32, a.wide, *reinterpret_cast<uint32_t(*)[8]>(&in[u][8 * v]));
    }
    // (while those are on their way)
    if (base == 0) {
      if (threadIdx.x < rows) s_place[threadIdx.x] = place_row(a, row0 + threadIdx.x);
      __syncthreads();
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= n) continue;
      const Block b = block_of<kDim>(a, i);
      const RowPlace p = s_place[b.row];
      if (p.six < 0) continue;
      uint32_t words[2];
      const uint32_t sb = quantize_block<false, kBf16, false>(in[u], b.value ? a.c.v_mul : a.c.k_mul, s_inv[b.value], words);
      uint8_t* scale;
      *reinterpret_cast<uint2*>(codes_of<kDim>(a, p, b, &scale)) = make_uint2(words[0], words[1]);
      *scale = static_cast<uint8_t>(sb);
    }
  }
}

template <int kDim>
__global__ void __launch_bounds__(kThreads) k_kv_read(const KvCopyArgs a) {
  __shared__ RowPlace s_place[kMaxRows];
  pdl_wait();
  pdl_trigger();
  const int row0 = blockIdx.x * a.cta_rows, rows = min(a.cta_rows, a.s.n_rows - row0);
  if (threadIdx.x < rows) s_place[threadIdx.x] = place_row(a, row0 + threadIdx.x);
  __syncthreads();
  const int n = rows * 2 * a.c.heads * (kDim / 16);
  for (int i0 = threadIdx.x; i0 < n; i0 += kBatch) {
    uint2 codes[kUnroll];
    uint32_t scales[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      codes[u] = make_uint2(0, 0);
      scales[u] = 0;
      if (i >= n) continue;
      const Block b = block_of<kDim>(a, i);
      const RowPlace p = s_place[b.row];
      if (p.six < 0) continue;
      uint8_t* scale;
      codes[u] = *reinterpret_cast<const uint2*>(codes_of<kDim>(a, p, b, &scale));
      scales[u] = *scale;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int i = i0 + u * kThreads;
      if (i >= n) continue;
      const Block b = block_of<kDim>(a, i);
      if (s_place[b.row].six == -2) continue;
      const float s = e4m3_to_float(scales[u]) * (b.value ? a.c.v_mul : a.c.k_mul);  // exact: |exp| <= 64
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float2 v = e2m1_values(((j < 4 ? codes[u].x : codes[u].y) >> (8 * (j & 3))) & 0xFFu);
        const __nv_bfloat162 h = __floats2bfloat162_rn(v.x * s, v.y * s);
        o[j] = *reinterpret_cast<const uint32_t*>(&h);
      }
      __nv_bfloat16* out = b.value ? a.v_out : a.k_out;
      store32b(out + (static_cast<int64_t>(row0 + b.row) * a.c.heads + b.head) * kDim + b.block * 16, a.wide, o);
    }
  }
}

namespace {

// How many rows a CTA takes, and how many CTAs that makes: few rows spread over more
// CTAs, down to one row each.
unsigned set_rows(KvCopyArgs* a) {
  const int per_row = 2 * a->c.heads * (a->c.dim / 16), most = per_row >= kBatch ? 1 : kBatch / per_row;
  const int spread = (a->s.n_rows + 2 * plan::kAttendSms - 1) / (2 * plan::kAttendSms);
  a->cta_rows = spread < most ? spread : most;
  // (blocks of a CTA stay below 2^15, where this quotient is exact for divisors up to 2^16)
  a->row_magic = a->cta_rows > 1 ? static_cast<uint32_t>(((1ull << 32) + per_row - 1) / per_row) : 0;
  return static_cast<unsigned>((a->s.n_rows + a->cta_rows - 1) / a->cta_rows);
}

}  // namespace

cudaError_t launch_kv_write(const KvCopyArgs& args, bool bf16, cudaStream_t s) {
  KvCopyArgs a = args;
  a.wide = true;
  for (const AttnRows* r : {&a.k, &a.v})
    a.wide &= reinterpret_cast<uintptr_t>(r->data) % 32 == 0 && r->row % 32 == 0 && r->head % 32 == 0;
  void (*k)(const KvCopyArgs) = a.c.dim == 64 ? (bf16 ? k_kv_write<64, true> : k_kv_write<64, false>)
                                              : (bf16 ? k_kv_write<128, true> : k_kv_write<128, false>);
  return launch_kernel(k, dim3(set_rows(&a)), dim3(kThreads), 0, s, true, a);
}

cudaError_t launch_kv_read(const KvCopyArgs& args, cudaStream_t s) {
  KvCopyArgs a = args;
  a.wide = reinterpret_cast<uintptr_t>(a.k_out) % 32 == 0 && reinterpret_cast<uintptr_t>(a.v_out) % 32 == 0;
  const unsigned grid = set_rows(&a);
  return launch_kernel(a.c.dim == 64 ? k_kv_read<64> : k_kv_read<128>, dim3(grid), dim3(kThreads), 0, s, true, a);
}

}  // namespace clover
