// Heads of q, k and v rows: norm of each head, rotary positions, and the paged cache's write and read.
//
// A head of D elements is a group of LPH lanes (8, 16 or 32) with a 16-byte chunk each.  A group works on heads of one
// token, so that the sines and cosines of its chunk's pairs stay in registers; what lanes exchange (sums, maxima, the
// other half of a rotated pair) goes by lane permutations.  No LDS and no barriers in the usual layouts.  The rows'
// bytes bound it: 8192 tokens of 32 heads of 128 rotated, 134 MB, take 28.1 us (4.8 TB/s, a large copy 5.1).
// Quantised, the vector instructions come on top: 8192 tokens with 16 heads of q and 8 each of k and v of 128, normed,
// rotated and written in 8 bits, 117 MB, take 31.5 us (3.7 TB/s; 54 us with a table of a token's sines in LDS and sums
// by LDS permutes).
//
// The angle of a pair i at position p is the fraction of p * freq[i] turns: the product is taken in 64 bits (in 32 a
// position of 10^6 would leave the angle of the fastest pair 0.06 rad off), its sine and cosine in 32.
//
// Quantisation of a row as in moe_quantize_i8: a = max(max |x|, 2^-100), scale = a / top, code = x / scale rounded to
// nearest, top = 127 or 448, as x times top / a in fp32, rounded once; a row that holds Inf or NaN gets scale NaN and
// codes 0.
#include "attend_internal.h"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 2;  // heads whose loads a lane has in flight

template <int CTRL, int BANKS = 0xf>
__device__ __forceinline__ float dpp(float old, float v) {
  return __int_as_float(
      __builtin_amdgcn_update_dpp(__float_as_int(old), __float_as_int(v), CTRL, 0xf, BANKS, false));
}
// The lanes 16 apart within pairs of rows: (row 0, row 0, row 2, row 2) and (row 1, row 1, row 3, row 3).
__device__ __forceinline__ void rows_apart(float v, float& even, float& odd) {
  const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v), false, false);
  even = __uint_as_float(x[0]), odd = __uint_as_float(x[1]);
}
// All-lane reduction over groups of LPH lanes: neighbours, pairs, quads mirrored, eights mirrored, rows.
template <int LPH, class F>
__device__ __forceinline__ float group_reduce(float v, F f) {
  v = f(v, dpp<0xb1>(v, v));
  v = f(v, dpp<0x4e>(v, v));
  v = f(v, dpp<0x141>(v, v));
  if constexpr (LPH > 8) v = f(v, dpp<0x140>(v, v));
  if constexpr (LPH > 16) {
    float a, b;
    rows_apart(v, a, b);
    v = f(a, b);
  }
  return v;
}
// The value of the lane LPH / 2 away.
template <int LPH>
__device__ __forceinline__ float other_half(float v, int c) {
  if constexpr (LPH == 16) return dpp<0x128>(v, v);
  if constexpr (LPH == 8) return dpp<0x12c, 0x5>(dpp<0x124, 0xa>(v, v), v);
  float a, b;
  rows_apart(v, a, b);
  return c < LPH / 2 ? b : a;
}

__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 v;
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = cvt_bf16x2(f[2 * i], f[2 * i + 1]);
  return v;
}

// How pairs lie: within a chunk, in chunks LPH / 2 lanes apart (the whole head in halves), in chunks some lanes apart,
// anywhere.
enum { kInside, kWhole, kApart, kOdd };

// TYPE: of the cache, -1 for none.  per_token: groups of a token.
template <int LPH, int TYPE, int PAIRS>
__global__ __launch_bounds__(kThreads) void heads_kernel(HeadArgs p, int per_token) {
  constexpr int G = kThreads / LPH;  // groups of a workgroup
  __shared__ float stage[PAIRS == kOdd ? 8 : 1][PAIRS == kOdd ? kThreads : 1];
  const int tid = threadIdx.x, c = tid % LPH;
  const int64_t group = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * G + tid / LPH;
  const int64_t t = group / per_token;
  if (t >= p.T) return;
  const int first = (int)(group - t * per_token);
  const int units = TYPE < 0 ? p.Hq : p.Hq + 2 * p.Hkv;
  const int half = p.rot / 2;
  const bool in = c * 8 < p.D;

  auto load = [&](int j) {
    u32x4 w = {0u, 0u, 0u, 0u};
    if (j < units && in) {
      const uint16_t* x = p.q + t * p.q_ld + j * p.D;
      if (TYPE >= 0 && j >= p.Hq)
        x = j < p.Hq + p.Hkv ? p.k + t * p.k_ld + (j - p.Hq) * p.D : p.v + t * p.v_ld + (j - p.Hq - p.Hkv) * p.D;
      w = *reinterpret_cast<const u32x4*>(x + c * 8);
    }
    return w;
  };
  u32x4 raw[kUnits];
#pragma unroll
  for (int u = 0; u < kUnits; ++u) raw[u] = load(first + u * per_token);

  float wq[8], wk[8];
  if (p.w_q && in) chunk_to_f32(*reinterpret_cast<const u32x4*>(p.w_q + c * 8), wq);
  if (TYPE >= 0 && p.w_k && in) chunk_to_f32(*reinterpret_cast<const u32x4*>(p.w_k + c * 8), wk);
  const int slot = TYPE >= 0 ? p.slots[t] : 0;
  // sines and cosines of the chunk's elements (kInside: of its pairs); 1 and 0 behind the rotated part
  constexpr int NC = PAIRS == kInside ? 4 : 8;
  float co[NC], si[NC];
  const bool lower = c * 8 < half;  // (unless kInside or kOdd) the chunk holds pairs' first elements
  if (p.rot > 0) {
    const double pos = (double)p.pos[t];
    auto angle = [&](int pair, float& cs, float& sn) {
      const double turns = pos * p.freq[pair];
      sincospif(2.0f * (float)(turns - rint(turns)), &sn, &cs);
      cs *= p.mscale, sn *= p.mscale;
    };
    if constexpr (PAIRS == kWhole) {
      // the lanes LPH / 2 apart hold the same pairs: each works out four of the eight
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float cs, sn;
        angle((c & (LPH / 2 - 1)) * 8 + (lower ? e : e + 4), cs, sn);
        const float oc = other_half<LPH>(cs, c), os = other_half<LPH>(sn, c);
        co[e] = lower ? cs : oc, si[e] = lower ? -sn : os;
        co[e + 4] = lower ? oc : cs, si[e + 4] = lower ? -os : sn;
      }
    } else {
#pragma unroll
      for (int e = 0; e < NC; ++e) {
        const int i = PAIRS == kInside ? c * 4 + e : c * 8 + e;
        co[e] = 1.0f, si[e] = 0.0f;
        if (PAIRS == kInside ? i < half : i < p.rot) {
          angle(PAIRS == kInside || i < half ? i : i - half, co[e], si[e]);
          // the second element of a pair takes the first with the other sign
          if (PAIRS != kInside && i < half) si[e] = -si[e];
        }
      }
    }
  }

  const float d_inv = 1.0f / (float)p.D;
  const int64_t page_row = TYPE >= 0 ? ((int64_t)(slot >> p.page_shift) * p.Hkv << p.page_shift) +
                                           (slot & ((1 << p.page_shift) - 1))
                                     : 0;
  const bool keep = TYPE >= 0 && (unsigned)slot < (unsigned)p.n_slots;
  for (int j0 = first; j0 < units; j0 += kUnits * per_token) {
    u32x4 ahead[kUnits];
#pragma unroll
    for (int u = 0; u < kUnits; ++u) ahead[u] = load(j0 + (kUnits + u) * per_token);
#pragma unroll
    for (int u = 0; u < kUnits; ++u) {
      const int j = j0 + u * per_token;
      if (j >= units) break;
      const int kind = TYPE < 0 || j < p.Hq ? 0 : j < p.Hq + p.Hkv ? 1 : 2;  // q, k, v
      float f[8];
      chunk_to_f32(raw[u], f);
      if (kind == 0 ? p.w_q != nullptr : kind == 1 && p.w_k != nullptr) {
        float s = 0.0f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += f[e] * f[e];
        s = group_reduce<LPH>(s, [](float a, float b) { return a + b; });
        const float r = __builtin_amdgcn_rsqf(s * d_inv + p.eps);  // 1 ulp
#pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = f[e] * r * ((kind == 1 ? wk[e] : wq[e]) + p.w_add);
        if (!in)
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = 0.0f;
      }
      if (p.rot > 0 && kind != 2) {
        if constexpr (PAIRS == kInside) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if (c * 4 + e < half) {
              const float x = f[2 * e], y = f[2 * e + 1];
              f[2 * e] = x * co[e] - y * si[e];
              f[2 * e + 1] = y * co[e] + x * si[e];
            }
          }
        } else if constexpr (PAIRS == kWhole) {
#pragma unroll
          for (int e = 0; e < 8; ++e) f[e] = f[e] * co[e] + other_half<LPH>(f[e], c) * si[e];
        } else if constexpr (PAIRS == kApart) {
          const int from = (tid & 63) + (lower ? half / 8 : -(half / 8));
          float o[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = __shfl(f[e], from);
          if (c * 8 < p.rot)
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * co[e] + o[e] * si[e];
        } else {
          // (of one wave: in order)
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int e = 0; e < 8; ++e) stage[e][tid] = f[e];
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int i = c * 8 + e;
            if (i < p.rot) {
              const int other = i < half ? i + half : i - half;
              f[e] = f[e] * co[e] + stage[other & 7][tid - c + (other >> 3)] * si[e];
            }
          }
        }
      }
      if (kind == 0) {
        if (in) *reinterpret_cast<u32x4*>(p.q_out + t * p.out_ld + j * p.D + c * 8) = pack8(f);
        continue;
      }
      if constexpr (TYPE >= 0) {
        const int head = j - p.Hq - (kind == 2 ? p.Hkv : 0);
        const int64_t row = page_row + ((int64_t)head << p.page_shift);
        void* cache = kind == 1 ? p.k_cache : p.v_cache;
        if constexpr (TYPE == MOE_BF16) {
          if (keep && in) *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(cache) + row * p.D + c * 8) = pack8(f);
          continue;
        }
        // the maximum of the magnitudes' bit patterns, ordered as they are, Inf and NaN above all finite ones
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(f[e]) & 0x7fffffffu);
        m = __float_as_uint(group_reduce<LPH>(__uint_as_float(m), [](float a, float b) {
          return __uint_as_float(max(__float_as_uint(a), __float_as_uint(b)));
        }));
        const bool bad = m >= 0x7f800000u;
        constexpr float top = TYPE == MOE_I8 ? 127.0f : 448.0f;
        const float a = fmaxf(__uint_as_float(m), kQuantTiny), scale = a * (1.0f / top);
        // top / a as inv + low, to twice 24 bits: by the scale's reciprocal (a's own is no normal number for the
        // largest) and residuals.  Quotients halfway between two codes, which rows of bf16 values have many of, are
        // then found as such: x * top / a is representable there, and code() rounds once.
        const float near = __builtin_amdgcn_rcpf(scale), back = near * (1.0f / top);
        const float inv = fmaf(fmaf(-near, a, top), back, near), low = fmaf(-inv, a, top) * back;
        auto code = [&](float x) { return fmaf(x, inv, x * low); };
        u32x2 w = {0u, 0u};
        if constexpr (TYPE == MOE_I8) {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e >> 2] |= ((uint32_t)__float2int_rn(code(f[e])) & 0xffu) << (8 * (e & 3));
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int v = __builtin_amdgcn_cvt_pk_fp8_f32(code(f[4 * h]), code(f[4 * h + 1]), 0, false);
            w[h] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(code(f[4 * h + 2]), code(f[4 * h + 3]), v, true);
          }
        }
        if (bad) w = u32x2{0u, 0u};
        if (keep && in) *reinterpret_cast<u32x2*>(static_cast<uint8_t*>(cache) + row * p.D + c * 8) = w;
        if (keep && c == 0) (kind == 1 ? p.k_scale : p.v_scale)[row] = bad ? __uint_as_float(0x7fc00000u) : scale;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnits; ++u) raw[u] = ahead[u];
  }
}

// Rows of the cache by slot, 8 elements a thread: a copy that gathers and widens, bound by its bytes (8192 tokens of
// 8 + 8 heads of 128 from 8 bits to bf16, 50 MB, 12 us).
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
      (((int64_t)(slot >> p.page_shift) * p.Hkv + head) << p.page_shift) + (slot & ((1 << p.page_shift) - 1));
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

template <int LPH, int TYPE>
static void heads_pairs(const HeadArgs& a, int per_token, dim3 grid, hipStream_t st) {
  if (a.interleaved || a.rot == 0)
    heads_kernel<LPH, TYPE, kInside><<<grid, kThreads, 0, st>>>(a, per_token);
  else if (a.rot == 8 * LPH)
    heads_kernel<LPH, TYPE, kWhole><<<grid, kThreads, 0, st>>>(a, per_token);
  else if (a.rot % 16 == 0)
    heads_kernel<LPH, TYPE, kApart><<<grid, kThreads, 0, st>>>(a, per_token);
  else
    heads_kernel<LPH, TYPE, kOdd><<<grid, kThreads, 0, st>>>(a, per_token);
}

template <int LPH>
static void heads_type(const HeadArgs& a, hipStream_t st) {
  constexpr int G = kThreads / LPH;
  // groups of a token: as many as fill the CUs (2^15 groups of 16 lanes), at most one per head
  const int units = a.Hq + 2 * a.Hkv;
  const int64_t want = ((int64_t)(1 << 19) / LPH + a.T - 1) / a.T;
  const int per_token = (int)(want < units ? want : units);
  const dim3 grid = grid_of(((int64_t)a.T * per_token + G - 1) / G);
  if (a.Hkv == 0)
    heads_pairs<LPH, -1>(a, per_token, grid, st);
  else if (a.type == MOE_I8)
    heads_pairs<LPH, MOE_I8>(a, per_token, grid, st);
  else if (a.type == MOE_E4M3)
    heads_pairs<LPH, MOE_E4M3>(a, per_token, grid, st);
  else
    heads_pairs<LPH, MOE_BF16>(a, per_token, grid, st);
}

hipError_t launch_heads(const HeadArgs& a, hipStream_t st) {
  if (a.D <= 64)
    heads_type<8>(a, st);
  else if (a.D <= 128)
    heads_type<16>(a, st);
  else
    heads_type<32>(a, st);
  return hipGetLastError();
}

hipError_t launch_cache_read(const CacheReadArgs& a, hipStream_t st) {
  const int64_t blocks = ((int64_t)a.n * 2 * a.Hkv * (a.D / 8) + kThreads - 1) / kThreads;
  cache_read_kernel<<<grid_of(blocks), kThreads, 0, st>>>(a);
  return hipGetLastError();
}

}  // namespace moe
