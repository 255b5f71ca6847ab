// Row operators around the layer: the norms at a block's boundary with gate and residual scale, and rows of
// 8-bit integers with one scale per row.
//
// All three kernels are bound by the bytes of their rows: a row is read once with 16-byte loads, held in registers as
// long as its sums need it, and written once.  A row has as many waves as let a lane hold one 16-byte chunk of it (up
// to 16 waves; rows of up to 512 elements go four to a workgroup): fewer, fuller waves took longer in every norm, the
// weights' loads waiting behind the reductions (one token of 2048 3.8 -> 2.7 us, 8192 tokens 31.1 -> 26.7, 3000 rows of
// 16384 139 -> 83).  Now, with a copy of 1 GiB at 4.8 to 5.3 TB/s: norm behind, gate, add, norm before, 8192 x 2048 25.9
// us (5.2 TB/s); fp32 stream with a gate per token, 1021 x 4096 11.4 (5.1); norm before alone with r', 8192 x 2048, to
// bf16 rows 25.1, to 8-bit rows 24.0, to both 29.5 (these from inputs outside the Infinity Cache); quantise 8192 x 4096
// 20.5 (4.9); SwiGLU rows 65536 x 512 30.8 (5.4).
//
// Sums run over a lane's chunks in order, then over the lanes in a fixed tree and the waves in order, so results do not
// depend on scheduling.
//
// Quantisation of a row: a = max(max |x|, 2^-100), scale = a / 127, code = rint(x (127 / a)), so that
// |x - scale * code| <= scale / 2 up to fp32 rounding and no code leaves [-127, 127].  The floor on a keeps both
// factors normal floats; rows below it become zero codes.  The maximum is taken on the magnitudes' bit patterns
// (ordered as the magnitudes are, Inf and NaN above all finite ones): a row holding one of these gets scale NaN and
// zero codes, and every product with it is NaN.
#include "block_internal.h"

namespace moe {
namespace {

// Threads of a workgroup whose rows have WPR waves each: four rows of one wave, else one row.
template <int WPR>
constexpr int kRowThreads = WPR == 1 ? 256 : 64 * WPR;

// A launch holds fewer than 2^32 threads per grid dimension: workgroups beyond 2^20 go to the second one.
dim3 row_grid(int64_t blocks) {
  return blocks <= (1 << 20) ? dim3((unsigned)blocks) : dim3(1u << 20, (unsigned)((blocks + (1 << 20) - 1) >> 20));
}
__device__ __forceinline__ int64_t block_index() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

// Maximum over the 64 lanes by the same DPP steps as wave_sum (0 is the identity).
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xf, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xa, 0xf, false));
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xc, 0xf, false));
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

// Sum (maximum) over the WPR waves of a row; `part` is a kernel's own LDS array per reduction.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < WPR; ++w) v += part[w];
  }
  return v;
}
template <int WPR>
__device__ __forceinline__ uint32_t row_max(uint32_t v, uint32_t* part) {
  v = wave_max_u32(v);
  if constexpr (WPR > 1) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WPR; ++w) v = max(v, part[w]);
  }
  return v;
}

__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7fffffffu; }

// Scale of a row and the factor its elements are multiplied with; a row with Inf or NaN: NaN and 0.
struct RowScale {
  float scale, inv;
  bool bad;
};
__device__ __forceinline__ RowScale row_scale(uint32_t max_bits) {
  RowScale s;
  s.bad = max_bits >= 0x7f800000u;
  const float a = fmaxf(__uint_as_float(max_bits), kQuantTiny);
  s.scale = s.bad ? __uint_as_float(0x7fc00000u) : a / 127.0f;
  s.inv = s.bad ? 0.0f : 127.0f / a;
  return s;
}

// Eight codes in two words, the first element in the lowest byte.
__device__ __forceinline__ u32x2 codes8(const float* f, const RowScale& s) {
  u32x2 w = {0u, 0u};
  if (s.bad) return w;
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i >> 2] |= ((uint32_t)(__float2int_rn(f[i] * s.inv)) & 0xffu) << (8 * (i & 3));
  return w;
}

__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = cvt_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}

// A row's chunks of 8 elements: chunk c of lane l is WPR * 64 * c + l.
template <int CPL, int WPR, bool F32, bool YIN>
__global__ __launch_bounds__(kRowThreads<WPR>) void block_norm_kernel(NormArgs p) {
  __shared__ float part_y[WPR], part_r[WPR];
  __shared__ uint32_t part_q[WPR];
  constexpr int LANES = 64 * WPR;
  const int lane = threadIdx.x % LANES;
  const int64_t t = block_index() * (kRowThreads<WPR> / LANES) + threadIdx.x / LANES;
  if (t >= p.T) return;
  const int nch = p.H / 8;
  const float n_inv = 1.0f / (float)p.H;
  float v[CPL][8];
  const int64_t row = t * p.H;
  if constexpr (YIN) {
    const uint16_t* y = p.y + row;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int ch = c * LANES + lane;
      u32x4 w = {0u, 0u, 0u, 0u};
      if (ch < nch) w = *reinterpret_cast<const u32x4*>(y + ch * 8);
      chunk_to_f32(w, v[c]);
    }
  }
  u32x4 rw[CPL][F32 ? 2 : 1];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int ch = c * LANES + lane;
#pragma unroll
    for (int h = 0; h < (F32 ? 2 : 1); ++h) {
      rw[c][h] = u32x4{0u, 0u, 0u, 0u};
      if (ch < nch)
        rw[c][h] = F32 ? reinterpret_cast<const u32x4*>(static_cast<const float*>(p.r) + row)[ch * 2 + h]
                       : reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.r) + row)[ch];
    }
  }
  // the weights and the gate are read here too, not behind the reductions they follow
  u32x4 pw[CPL], gw[CPL], nw[CPL];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int ch = min(c * LANES + lane, nch - 1);
    if (YIN && p.w_post) pw[c] = reinterpret_cast<const u32x4*>(p.w_post)[ch];
    if (YIN && p.gate) gw[c] = reinterpret_cast<const u32x4*>(p.gate + t * p.gate_ld)[ch];
    if (p.w_pre) nw[c] = reinterpret_cast<const u32x4*>(p.w_pre)[ch];
  }
  float ys = p.y_scale;
  if (YIN && p.w_post) {
    float s = 0.0f;
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
      for (int i = 0; i < 8; ++i) s += v[c][i] * v[c][i];
    const float rs = rsqrtf(row_sum<WPR>(s, part_y) * n_inv + p.eps);
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int ch = c * LANES + lane;
      if (ch < nch) {
        float w[8];
        chunk_to_f32(pw[c], w);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[c][i] = v[c][i] * rs * (w[i] + p.w_add);
      }
    }
  }
  float s = 0.0f;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int ch = c * LANES + lane;
    float r[8];
    if constexpr (F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) r[i] = __uint_as_float(rw[c][i >> 2][i & 3]);
    } else {
      chunk_to_f32(rw[c][0], r);
    }
    if constexpr (YIN) {
      float g[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = ys;
      if (p.gate && ch < nch) {
        chunk_to_f32(gw[c], g);
#pragma unroll
        for (int i = 0; i < 8; ++i) g[i] *= ys;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = p.r_scale * r[i] + g[i] * v[c][i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[c][i] = p.r_scale * r[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) s += v[c][i] * v[c][i];
    if (p.r_out && ch < nch) {
      if constexpr (F32) {
        u32x4* o = reinterpret_cast<u32x4*>(static_cast<float*>(p.r_out) + row) + ch * 2;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          o[h] = u32x4{__float_as_uint(v[c][4 * h]), __float_as_uint(v[c][4 * h + 1]), __float_as_uint(v[c][4 * h + 2]),
                       __float_as_uint(v[c][4 * h + 3])};
      } else {
        reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.r_out) + row)[ch] = pack8(v[c]);
      }
    }
  }
  if (!p.w_pre) return;
  // the norm reads the fp32 sum, before r_out's rounding: each output is rounded once
  const float rs = rsqrtf(row_sum<WPR>(s, part_r) * n_inv + p.eps);
  uint32_t mx = 0;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int ch = c * LANES + lane;
    if (ch < nch) {
      float w[8];
      chunk_to_f32(nw[c], w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        v[c][i] = v[c][i] * rs * (w[i] + p.w_add);
        mx = max(mx, abs_bits(v[c][i]));
      }
      if (p.x) reinterpret_cast<u32x4*>(p.x + row)[ch] = pack8(v[c]);
    }
  }
  if (!p.q) return;
  const RowScale sc = row_scale(row_max<WPR>(mx, part_q));
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int ch = c * LANES + lane;
    if (ch < nch) reinterpret_cast<u32x2*>(p.q + row)[ch] = codes8(v[c], sc);
  }
  if (lane == 0) p.q_scale[t] = sc.scale;
}

// Rows of bf16 (SWIGLU: silu(gate) * up of rows [gate | up]) to codes and a scale per row.
template <int CPL, int WPR, bool SWIGLU>
__global__ __launch_bounds__(kRowThreads<WPR>) void quantize_kernel(const uint16_t* x, const float* row_gate, int R,
                                                                    int K, int8_t* q, float* scale) {
  __shared__ uint32_t part_q[WPR];
  constexpr int LANES = 64 * WPR;
  const int lane = threadIdx.x % LANES;
  const int64_t t = block_index() * (kRowThreads<WPR> / LANES) + threadIdx.x / LANES;
  if (t >= R) return;
  const int nch = K / 8;
  const uint16_t* src = x + t * K * (SWIGLU ? 2 : 1);
  u32x4 w[CPL][SWIGLU ? 2 : 1];
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int ch = c * LANES + lane;
#pragma unroll
    for (int h = 0; h < (SWIGLU ? 2 : 1); ++h) {
      w[c][h] = u32x4{0u, 0u, 0u, 0u};
      if (ch < nch) w[c][h] = reinterpret_cast<const u32x4*>(src + (size_t)h * K)[ch];
    }
  }
  float f[CPL][8];
  uint32_t mx = 0;
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    chunk_to_f32(w[c][0], f[c]);
    if constexpr (SWIGLU) {
      float u[8];
      chunk_to_f32(w[c][1], u);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[c][i] = silu(f[c][i]) * u[i];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) mx = max(mx, abs_bits(f[c][i]));
  }
  const RowScale sc = row_scale(row_max<WPR>(mx, part_q));
#pragma unroll
  for (int c = 0; c < CPL; ++c) {
    const int ch = c * LANES + lane;
    if (ch < nch) reinterpret_cast<u32x2*>(q + t * K)[ch] = codes8(f[c], sc);
  }
  if (lane == 0) scale[t] = SWIGLU && row_gate ? sc.scale * row_gate[t] : sc.scale;
}

template <int CPL, int WPR, bool F32, bool YIN>
void norm_run(const NormArgs& a, hipStream_t st) {
  block_norm_kernel<CPL, WPR, F32, YIN>
      <<<row_grid(WPR == 1 ? ((int64_t)a.T + 3) / 4 : a.T), kRowThreads<WPR>, 0, st>>>(a);
}
template <bool F32, bool YIN>
void norm_launch(const NormArgs& a, hipStream_t st) {
  const int nch = a.H / 8;
  if (nch <= 64)
    norm_run<1, 1, F32, YIN>(a, st);
  else if (nch <= 128)
    norm_run<1, 2, F32, YIN>(a, st);
  else if (nch <= 256)
    norm_run<1, 4, F32, YIN>(a, st);
  else if (nch <= 512)
    norm_run<1, 8, F32, YIN>(a, st);
  else if (nch <= 1024)
    norm_run<1, 16, F32, YIN>(a, st);
  else
    norm_run<2, 16, F32, YIN>(a, st);
}

template <int CPL, int WPR, bool SWIGLU>
void quantize_run(const uint16_t* x, const float* row_gate, int R, int K, int8_t* q, float* scale, hipStream_t st) {
  quantize_kernel<CPL, WPR, SWIGLU>
      <<<row_grid(WPR == 1 ? ((int64_t)R + 3) / 4 : R), kRowThreads<WPR>, 0, st>>>(x, row_gate, R, K, q, scale);
}
template <bool SWIGLU>
hipError_t quantize_launch(const uint16_t* x, const float* row_gate, int R, int K, int8_t* q, float* scale,
                           hipStream_t st) {
  const int nch = K / 8;
  if (nch <= 64)
    quantize_run<1, 1, SWIGLU>(x, row_gate, R, K, q, scale, st);
  else if (nch <= 128)
    quantize_run<1, 2, SWIGLU>(x, row_gate, R, K, q, scale, st);
  else if (nch <= 256)
    quantize_run<1, 4, SWIGLU>(x, row_gate, R, K, q, scale, st);
  else if (nch <= 512)
    quantize_run<1, 8, SWIGLU>(x, row_gate, R, K, q, scale, st);
  else if (nch <= 1024)
    quantize_run<1, 16, SWIGLU>(x, row_gate, R, K, q, scale, st);
  else if (nch <= 2048)
    quantize_run<2, 16, SWIGLU>(x, row_gate, R, K, q, scale, st);
  else
    quantize_run<4, 16, SWIGLU>(x, row_gate, R, K, q, scale, st);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_block_norm(const NormArgs& a, hipStream_t st) {
  if (a.f32)
    a.y ? norm_launch<true, true>(a, st) : norm_launch<true, false>(a, st);
  else
    a.y ? norm_launch<false, true>(a, st) : norm_launch<false, false>(a, st);
  return hipGetLastError();
}

hipError_t launch_quantize_i8(const uint16_t* x, int R, int K, int8_t* q, float* scale, hipStream_t st) {
  return quantize_launch<false>(x, nullptr, R, K, q, scale, st);
}

hipError_t launch_swiglu_i8(const uint16_t* gu, const float* row_gate, int R, int I, int8_t* q, float* scale,
                            hipStream_t st) {
  return quantize_launch<true>(gu, row_gate, R, I, q, scale, st);
}

}  // namespace moe
