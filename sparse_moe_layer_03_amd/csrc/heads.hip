// Heads of q, k and v rows: norm of each head, rotary positions, and the paged cache's write and read.
//
// A head of D elements is a group of LPH lanes (8, 16 or 32) with a 16-byte chunk each.  All is bound by the rows'
// bytes.  The angle of a pair i at position p is the fraction of p * freq[i] turns: the product is taken in 64 bits
// (in 32 a position of 10^6 would leave the angle of the fastest pair 0.06 rad off), its sine and cosine in 32.  A
// workgroup works them out once per token for all heads, into LDS.
//
// Quantisation of a row as in moe_quantize_i8: a = max(max |x|, 2^-100), scale = a / top, code = x (top / a) rounded to
// nearest, top = 127 or 448; a row that holds Inf or NaN gets scale NaN and codes 0.
#include "attend_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;  // heads whose loads a lane has in flight

// LDS written by some lanes of a wave and read by others of it: in order, and the compiler keeps it so.
__device__ __forceinline__ void wave_fence() { __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront"); }

template <int LPH>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int d = 1; d < LPH; d <<= 1) v += __shfl_xor(v, d);
  return v;
}
template <int LPH>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < LPH; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = cvt_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}

template <int LPH>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadArgs p, int tokens) {
  constexpr int G = kThreads / LPH;  // heads at work at once
  __shared__ float stage[8][kThreads];
  extern __shared__ float2 table[];  // [tokens][8][stride]: cosine and sine of pair i at [i & 7][i >> 3]
  const int tid = threadIdx.x, c = tid % LPH, group = tid / LPH;
  const int units = p.Hq + 2 * p.Hkv;
  const int64_t t0 = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * tokens;
  if (t0 >= p.T) return;
  const int nt = (int)min((int64_t)tokens, p.T - t0), total = nt * units;
  const int half = p.rot / 2, stride = (half + 7) / 8;
  const bool in = c * 8 < p.D;

  struct Unit {
    int tok, head, kind;  // kind 0: q, 1: k, 2: v
    bool live;
  };
  auto unit = [&](int base, int u) {
    const int i = base + u * G + group;
    Unit n;
    n.live = i < total;
    n.tok = n.live ? i / units : 0;
    const int j = n.live ? i - n.tok * units : 0;
    n.kind = j < p.Hq ? 0 : j < p.Hq + p.Hkv ? 1 : 2;
    n.head = n.kind == 0 ? j : n.kind == 1 ? j - p.Hq : j - p.Hq - p.Hkv;
    return n;
  };
  auto load = [&](const Unit& n) {
    u32x4 w = {0u, 0u, 0u, 0u};
    if (n.live && in) {
      const int64_t t = t0 + n.tok;
      const uint16_t* x = n.kind == 0 ? p.q + t * p.q_ld : n.kind == 1 ? p.k + t * p.k_ld : p.v + t * p.v_ld;
      w = *reinterpret_cast<const u32x4*>(x + n.head * p.D + c * 8);
    }
    return w;
  };

  u32x4 raw[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) raw[u] = load(unit(0, u));
  float wq[8], wk[8];
  if (p.w_q && in) chunk_to_f32(*reinterpret_cast<const u32x4*>(p.w_q + c * 8), wq);
  if (p.w_k && in) chunk_to_f32(*reinterpret_cast<const u32x4*>(p.w_k + c * 8), wk);
  for (int i = tid; i < nt * half; i += kThreads) {
    const int tok = i / half, pair = i - tok * half;
    const double turns = (double)p.pos[t0 + tok] * p.freq[pair];
    float s, co;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &co);
    table[(tok * 8 + (pair & 7)) * stride + (pair >> 3)] = make_float2(co * p.mscale, s * p.mscale);
  }
  __syncthreads();

  for (int base = 0; base < total; base += kUnits * G) {
    if (base > 0) {
#pragma unroll
      for (int u = 0; u < kUnits; ++u) raw[u] = load(unit(base, u));
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      if (base + u * G >= total) break;
      const Unit n = unit(base, u);
      float f[8];
      chunk_to_f32(raw[u], f);
      const bool is_k = n.kind == 1;
      if (n.kind == 0 ? p.w_q != nullptr : is_k && p.w_k != nullptr) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += f[e] * f[e];
        const float r = 1.0f / sqrtf(group_sum<LPH>(s) / (float)p.D + p.eps);
        if (in)
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = f[e] * r * ((is_k ? wk[e] : wq[e]) + p.w_add);
      }
      if (p.rot > 0 && n.kind != 2) {
        const float2* tab = table + n.tok * 8 * stride;
        if (p.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const int i = c * 4 + e / 2;
            if (i < half) {
              const float2 a = tab[(i & 7) * stride + (i >> 3)];
              const float x = f[e], y = f[e + 1];
              f[e] = x * a.x - y * a.y;
              f[e + 1] = y * a.x + x * a.y;
            }
          }
        } else {
          wave_fence();
#pragma unroll
          for (int e = 0; e < 8; ++e) stage[e][tid] = f[e];
          wave_fence();
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = c * 8 + e;
            if (i < p.rot) {
              const bool first = i < half;
              const int pair = first ? i : i - half, other = first ? i + half : i - half;
              const float2 a = tab[(pair & 7) * stride + (pair >> 3)];
              const float o = stage[other & 7][tid - c + (other >> 3)];
              f[e] = f[e] * a.x + (first ? -o : o) * a.y;
            }
          }
        }
      }
      const int64_t t = t0 + n.tok;
      if (n.kind == 0) {
        if (n.live && in) *reinterpret_cast<u32x4*>(p.q_out + t * p.out_ld + n.head * p.D + c * 8) = pack8(f);
        continue;
      }
      const int slot = p.slots[t];
      const bool write = n.live && (unsigned)slot < (unsigned)p.n_slots;
      const int64_t row =
          ((int64_t)(slot >> p.page_shift) * p.Hkv + n.head << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
      void* cache = is_k ? p.k_cache : p.v_cache;
      if (p.type == MOE_BF16) {
        if (write && in) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(cache) + row * p.D + c * 8) = pack8(f);
        continue;
      }
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
      m = group_max<LPH>(m);
      const bool bad = m >= 0x7f800000u;
      const float a = fmaxf(__uint_as_float(m), kQuantTiny), top = p.type == MOE_I8 ? 127.0f : 448.0f;
      const float inv = top / a;
      u32x2 w = {0u, 0u};
      if (p.type == MOE_I8) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e >> 2] |= ((uint32_t)__float2int_rn(f[e] * inv) & 0xffu) << (8 * (e & 3));
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          int v = __builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h] * inv, f[4 * h + 1] * inv, 0, false);
          w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[4 * h + 2] * inv, f[4 * h + 3] * inv, v, true);
        }
      }
      if (bad) w = u32x2{0u, 0u};
      if (write && in) *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(cache) + row * p.D + c * 8) = w;
      if (write && c == 0) (is_k ? p.k_scale : p.v_scale)[row] = bad ? __uint_as_float(0x7fc00000u) : a / top;
    }
  }
}

// Rows of the cache by slot, 8 elements a thread.
__global__ __launch_bounds__(kThreads) void cache_read_kernel(CacheReadArgs p) {
  const int cph = p.D / 8, per = 2 * p.Hkv * cph;  // chunks of a head, of a slot's k and v rows
  const int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kThreads + threadIdx.x;
  if (i >= (int64_t)p.n * per) return;
  const int r = (int)(i / per), j = (int)(i - (int64_t)r * per), hh = j / cph, c = j - hh * cph;
  const bool is_v = hh >= p.Hkv;
  const int head = is_v ? hh - p.Hkv : hh;
  const int slot = p.slots[r];
  if ((unsigned)slot >= (unsigned)p.n_slots) return;
  const int64_t row =
      ((int64_t)(slot >> p.page_shift) * p.Hkv + head << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
  const void* cache = is_v ? p.v_cache : p.k_cache;
  const int64_t to = ((int64_t)r * p.Hkv + head) * p.D + c * 8;
  void* out = is_v ? p.v : p.k;
  float f[8];
  if (p.type == MOE_BF16) {
    const u32x4 w = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(cache) + row * p.D + c * 8);
    if (!p.out_f32) {
      *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + to) = w;
      return;
    }
    chunk_to_f32(w, f);
  } else {
    const u32x2 w = *reinterpret_cast<const u32x2*>(static_cast<const uint8_t*>(cache) + row * p.D + c * 8);
    const float s = (is_v ? p.v_scale : p.k_scale)[row];
    if (p.type == MOE_I8) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = (float)((int32_t)(w[e >> 2] << (24 - 8 * (e & 3))) >> 24);
    } else {
      chunk_to_f32(w, f);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) f[e] *= s;
  }
  if (p.out_f32) {
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(out) + to);
    o[0] = make_float4(f[0], f[1], f[2], f[3]);
    o[1] = make_float4(f[4], f[5], f[6], f[7]);
  } else {
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + to) = pack8(f);
  }
}

}  // namespace

// A launch holds fewer than 2^32 threads per grid dimension.
static dim3 grid_of(int64_t blocks) {
  return blocks <= (1 << 20) ? dim3((unsigned)blocks) : dim3(1u << 20, (unsigned)((blocks + (1 << 20) - 1) >> 20));
}

hipError_t launch_heads(const HeadArgs& a, hipStream_t st) {
  const int lph = a.D <= 64 ? 8 : a.D <= 128 ? 16 : 32;
  const int units = a.Hq + 2 * a.Hkv, at_once = kThreads / lph;
  // tokens of a workgroup: enough heads for its lanes, as long as there are workgroups for every CU
  int tokens = 1;
  while (tokens * units < kUnits * at_once && a.T / tokens > 2048 && tokens < 16) tokens *= 2;
  const size_t lds = (size_t)tokens * 8 * ((a.rot / 2 + 7) / 8) * sizeof(float2);
  const dim3 blocks = grid_of((a.T + tokens - 1) / tokens);
  if (lph == 8)
    heads_kernel<8><<<blocks, kThreads, lds, st>>>(a, tokens);
  else if (lph == 16)
    heads_kernel<16><<<blocks, kThreads, lds, st>>>(a, tokens);
  else
    heads_kernel<32><<<blocks, kThreads, lds, st>>>(a, tokens);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheReadArgs& a, hipStream_t st) {
  const int64_t blocks = ((int64_t)a.n * 2 * a.Hkv * (a.D / 8) + kThreads - 1) / kThreads;
  cache_read_kernel<<<grid_of(blocks), kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
