// Writing rows of keys and values to the paged 4-bit cache and reading them
// back (clover_kv_write, clover_kv_read).
#include "attn_ops.cuh"
#include "launch.cuh"
#include "sm100.cuh"

namespace clover {

namespace {

constexpr int kThreads = 256;

// Block b of the call's blocks of 16 elements, in the order row, key or value,
// head, block of the head.
struct Place {
  int row, head, block;
  bool value;
  uint8_t* codes;  // null: no page
  uint8_t* scale;
  bool in;  // the row belongs to a sequence
};

__device__ __forceinline__ Place place_of(const KvCache& c, const AttnSeqs& s, int64_t b) {
  const int per_head = c.dim / 16, per_row = 2 * c.heads * per_head;
  Place r;
  r.row = static_cast<int>(b / per_row);
  const int i = static_cast<int>(b - static_cast<int64_t>(r.row) * per_row);
  r.value = i >= per_row / 2;
  const int j = r.value ? i - per_row / 2 : i;
  r.head = j / per_head;
  r.block = j - r.head * per_head;
  r.codes = r.scale = nullptr;
  const int q = seq_of_row(s, r.row);
  r.in = false;
  if (q < 0) return r;
  const SeqSpan sp = seq_span(s, q);
  if (r.row >= sp.row0 + sp.rows) return r;
  r.in = true;
  const int p = sp.len - sp.rows + (r.row - sp.row0);
  if (p < 0) return r;
  uint8_t* six = kv_sixteen(c, s, q, r.head, p);
  if (six == nullptr) return r;
  six += r.value ? 9 * c.dim : 0;
  r.codes = six + p % 16 * (c.dim / 2) + r.block * 8;
  r.scale = six + 8 * c.dim + p % 16 * per_head + r.block;
  return r;
}

}  // namespace

// One thread per block of 16 elements.
template <bool kBf16>
__global__ void __launch_bounds__(kThreads) k_kv_write(const KvCopyArgs a) {
  __shared__ float s_inv[2][128];
  if (kBf16) {
    const int i = threadIdx.x;
    s_inv[i >> 7][i & 127] = scale_inverse(i & 127, i < 128 ? a.c.k_mul : a.c.v_mul);
    __syncthreads();
  }
  pdl_wait();
  pdl_trigger();
  const int64_t b = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (b >= static_cast<int64_t>(a.s.n_rows) * (2 * a.c.heads * (a.c.dim / 16))) return;
  const Place p = place_of(a.c, a.s, b);
  if (p.codes == nullptr) return;
  constexpr int kSize = kBf16 ? 2 : 4;
  const AttnRows& x = p.value ? a.v : a.k;
  const uint8_t* src = x.data + p.row * x.row + p.head * x.head + p.block * (16 * kSize);
  uint32_t in[4 * kSize], words[2];
#pragma unroll
  for (int v = 0; v < kSize / 2; ++v) load32b(src + v * 32, a.wide, *reinterpret_cast<uint32_t(*)[8]>(&in[8 * v]));
  const uint32_t sb = quantize_block<false, kBf16, false>(in, p.value ? a.c.v_mul : a.c.k_mul, s_inv[p.value], words);
  *reinterpret_cast<uint2*>(p.codes) = make_uint2(words[0], words[1]);
  *p.scale = static_cast<uint8_t>(sb);
}

__global__ void __launch_bounds__(kThreads) k_kv_read(const KvCopyArgs a) {
  pdl_wait();
  pdl_trigger();
  const int64_t b = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
  if (b >= static_cast<int64_t>(a.s.n_rows) * (2 * a.c.heads * (a.c.dim / 16))) return;
  const Place p = place_of(a.c, a.s, b);
  if (!p.in) return;
  uint32_t o[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (p.codes != nullptr) {
    const float s = e4m3_to_float(*p.scale) * (p.value ? a.c.v_mul : a.c.k_mul);  // exact: |exp| <= 64
    const uint2 u = *reinterpret_cast<const uint2*>(p.codes);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 v = e2m1_values(((j < 4 ? u.x : u.y) >> (8 * (j & 3))) & 0xFFu);
      const __nv_bfloat162 h = __floats2bfloat162_rn(v.x * s, v.y * s);
      o[j] = *reinterpret_cast<const uint32_t*>(&h);
    }
  }
  __nv_bfloat16* out = p.value ? a.v_out : a.k_out;
  store32b(out + (static_cast<int64_t>(p.row) * a.c.heads + p.head) * a.c.dim + p.block * 16, a.wide, o);
}

namespace {
dim3 block_grid(const KvCopyArgs& a) {
  const int64_t n = static_cast<int64_t>(a.s.n_rows) * (2 * a.c.heads * (a.c.dim / 16));
  return dim3(static_cast<unsigned>((n + kThreads - 1) / kThreads));
}
}  // namespace

cudaError_t launch_kv_write(const KvCopyArgs& args, bool bf16, cudaStream_t s) {
  KvCopyArgs a = args;
  a.wide = true;
  for (const AttnRows* r : {&a.k, &a.v})
    a.wide &= reinterpret_cast<uintptr_t>(r->data) % 32 == 0 && r->row % 32 == 0 && r->head % 32 == 0;
  return launch_kernel(bf16 ? k_kv_write<true> : k_kv_write<false>, block_grid(a), dim3(kThreads), 0, s, true, a);
}

cudaError_t launch_kv_read(const KvCopyArgs& args, cudaStream_t s) {
  KvCopyArgs a = args;
  a.wide = reinterpret_cast<uintptr_t>(a.k_out) % 32 == 0 && reinterpret_cast<uintptr_t>(a.v_out) % 32 == 0;
  return launch_kernel(k_kv_read, block_grid(a), dim3(kThreads), 0, s, true, a);
}

}  // namespace clover
