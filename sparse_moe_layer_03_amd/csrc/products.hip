// Products C = A B^T on the matrix cores, dense or grouped by expert over ragged row counts, in bf16 with fp32
// sums or in 8-bit integers with int32 sums and a scale per A row and per B row.
//
// Both types move the same bytes: a lane feeds 16 bytes of a row (8 bf16 or 16 codes) to one 32 x 32 matrix
// instruction, so tiles, staging and addressing below count bytes and only the instruction and the epilogue
// differ.  B (the weights) is the instruction's first operand: a lane then holds, of one output row, four
// consecutive columns per register group.
//
// Grouped: expert e owns positions off[e] .. off[e] + count(e) - 1.  Position p is output row id = rows[p] (or p)
// and reads A row id / a_div; ids outside [0, R) are padding and are skipped.
#include "block_internal.h"

namespace moe {
namespace {

typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4v __attribute__((ext_vector_type(4)));

template <bool I8>
struct Acc {
  typedef f32x16 t32;
};
template <>
struct Acc<true> {
  typedef i32x16 t32;
};

__device__ __forceinline__ f32x16 mma32(const u32x4& b, const u32x4& a, const f32x16& c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, b), __builtin_bit_cast(bf16x8, a), c, 0, 0,
                                                 0);
}
__device__ __forceinline__ i32x16 mma32(const u32x4& b, const u32x4& a, const i32x16& c) {
  return __builtin_amdgcn_mfma_i32_32x32x32_i8(__builtin_bit_cast(i32x4v, b), __builtin_bit_cast(i32x4v, a), c, 0, 0,
                                               0);
}

// Positions of expert e, kept inside [0, P).
__device__ __forceinline__ void expert_range(const ProductArgs& p, int e, int& first, int& count) {
  const int lo = min(max(p.off[e], 0), p.P);
  const int n = p.counts ? p.counts[e] : p.off[e + 1] - lo;
  first = lo;
  count = min(max(n, 0), p.P - lo);
}

// Output row of a position, -1 for padding.
__device__ __forceinline__ int output_row(const ProductArgs& p, int pos) {
  const int id = p.rows ? p.rows[pos] : pos;
  return (unsigned)id < (unsigned)p.R ? id : -1;
}

// Tile `idx` of the list of all experts' BM-row tiles in expert order: (expert, first position, rows), or rows = 0
// past the end.  Thread e < E counts expert e's tiles; `s` is LDS of 260 ints.
template <int BM>
__device__ __forceinline__ void find_tile(const ProductArgs& p, int idx, int* s, int& expert, int& first, int& rows) {
  const int tid = threadIdx.x, lane = tid & 63;
  int lo = 0, n = 0;
  if (tid < p.E) expert_range(p, tid, lo, n);
  const int tiles = (n + BM - 1) / BM;
  int incl = tiles;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(incl, d);
    if (lane >= d) incl += o;
  }
  if (tid < 256 && lane == 63) s[tid >> 6] = incl;
  if (tid == 0) s[6] = 0;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < (tid >> 6) && w < 4; ++w) before += s[w];
  const int excl = before + incl - tiles;
  if (tid < p.E && idx >= excl && idx < excl + tiles) {
    s[4] = tid;
    s[5] = lo + (idx - excl) * BM;
    s[6] = min(BM, n - (idx - excl) * BM);
  }
  __syncthreads();
  expert = s[4];
  first = s[5];
  rows = s[6];
}

__device__ __forceinline__ int swz8(int row, int chunk) { return chunk ^ (((row >> 1) ^ ((row & 1) << 2)) & 7); }

// Four consecutive columns of one output row.
template <bool I8, class A>
__device__ __forceinline__ void store4(const ProductArgs& p, int id, int expert, int n, const A& acc, int q0) {
  float v[4];
  if constexpr (I8) {
    const float sa = p.a_scale[id / p.a_div];
    const float4 sb = *reinterpret_cast<const float4*>(p.b_scale + (size_t)expert * p.N + n);
    const float f[4] = {sb.x, sb.y, sb.z, sb.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = (float)acc[q0 + i] * sa * f[i];
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = acc[q0 + i];
  }
  if (p.bias) {
    const float4 b = *reinterpret_cast<const float4*>(p.bias + n);
    v[0] += b.x, v[1] += b.y, v[2] += b.z, v[3] += b.w;
  }
  const size_t at = (size_t)id * p.N + n;
  if (p.add) {
    const u32x2 w = *reinterpret_cast<const u32x2*>(p.add + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += bf16_to_f32((uint16_t)(w[i >> 1] >> (16 * (i & 1))));
  }
  if (p.c_f32)
    *reinterpret_cast<float4*>(static_cast<float*>(p.c) + at) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.c) + at) = u32x2{cvt_bf16x2(v[0], v[1]), cvt_bf16x2(v[2], v[3])};
}

// 64 x 64 tile per workgroup, four waves of 32 x 32, both operands through one LDS stage of 128-byte rows.
template <bool I8>
__global__ __launch_bounds__(256) void product_kernel(ProductArgs p) {
  __shared__ u32x4 sa[64 * 8], sb[64 * 8];
  __shared__ int s_tile[8], s_row[64];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int expert = 0, first = blockIdx.x * 64, rows = min(64, p.P - first);
  if (p.off) find_tile<64>(p, blockIdx.x, s_tile, expert, first, rows);
  if (rows <= 0) return;
  if (tid < 64) s_row[tid] = tid < rows ? output_row(p, first + tid) : -1;
  __syncthreads();
  const int n0 = blockIdx.y * 64;
  const int wm = wave >> 1, wn = wave & 1;
  typename Acc<I8>::t32 acc = {};
  for (int kb = 0; kb < p.Kb; kb += 128) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 32 + tid / 8, c = tid % 8, k = kb + c * 16;
      const int id = s_row[r];
      u32x4 va = {0u, 0u, 0u, 0u}, vb = {0u, 0u, 0u, 0u};
      if (id >= 0 && k < p.Kb)
        va = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p.a) + (size_t)(id / p.a_div) * p.Kb + k);
      if (n0 + r < p.N && k < p.Kb)
        vb = *reinterpret_cast<const u32x4*>(static_cast<const char*>(p.b) + ((size_t)expert * p.N + n0 + r) * p.Kb + k);
      sa[r * 8 + swz8(r, c)] = va;
      sb[r * 8 + swz8(r, c)] = vb;
    }
    __syncthreads();
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int c = 2 * s + (lane >> 5), ra = wm * 32 + (lane & 31), rb = wn * 32 + (lane & 31);
      acc = mma32(sb[rb * 8 + swz8(rb, c)], sa[ra * 8 + swz8(ra, c)], acc);
    }
    __syncthreads();
  }
  const int id = s_row[wm * 32 + (lane & 31)];
  if (id < 0) return;
#pragma unroll
  for (int g = 0; g < 4; ++g) {
    const int n = n0 + wn * 32 + 8 * g + 4 * (lane >> 5);
    if (n < p.N) store4<I8>(p, id, expert, n, acc, 4 * g);
  }
}

}  // namespace

hipError_t launch_product(const ProductArgs& p, bool i8, hipStream_t st) {
  const int64_t tiles = p.off ? p.P / 64 + (p.E < p.P ? p.E : p.P) : ((int64_t)p.P + 63) / 64;
  const dim3 grid((unsigned)tiles, (unsigned)((p.N + 63) / 64));
  if (i8)
    product_kernel<true><<<grid, 256, 0, st>>>(p);
  else
    product_kernel<false><<<grid, 256, 0, st>>>(p);
  return hipGetLastError();
}

}  // namespace moe
