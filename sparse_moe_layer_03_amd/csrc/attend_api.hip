// C ABI of the operators around attention: argument checks, all before anything is enqueued.
#include <math.h>

#include "api_checks.h"
#include "attention_kernel.h"

using namespace moe;

namespace {

constexpr int kMaxT = 1 << 24;
constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // tokens a cache or a page table row can name
constexpr int64_t kMaxRows = (int64_t)1 << 30;    // tokens times query heads
constexpr int64_t kMaxPairs = (int64_t)1 << 22;   // sequences times key heads

bool aligned8(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 7u) == 0; }

int check_heads(const char* f, int T, int D, int rot, int pairs, float eps, float mscale) {
  if (T < 0 || T > kMaxT) return fail(MOE_ERR_SHAPE, "%s: T=%d outside [0, 2^24]", f, T);
  if (D < 8 || D > kMaxHeadDim || D % 8 != 0)
    return fail(MOE_ERR_SHAPE, "%s: D=%d must be a multiple of 8 in [8, %d]", f, D, kMaxHeadDim);
  if (rot < 0 || rot > D || rot % 2 != 0)
    return fail(MOE_ERR_SHAPE, "%s: rot=%d must be an even number of the head's %d elements", f, rot, D);
  if (pairs != MOE_ROPE_HALF && pairs != MOE_ROPE_INTERLEAVED)
    return fail(MOE_ERR_SHAPE, "%s: pairs=%d is neither MOE_ROPE_HALF nor MOE_ROPE_INTERLEAVED", f, pairs);
  if (!(eps >= 0.0f)) return fail(MOE_ERR_SHAPE, "%s: eps must not be negative", f);
  if (!isfinite(mscale)) return fail(MOE_ERR_SHAPE, "%s: mscale must be finite", f);
  return MOE_OK;
}

int check_ld(const char* f, const char* name, int64_t ld, int64_t row) {
  if (ld < row || ld % 8 != 0 || ld > ((int64_t)1 << 32))
    return fail(MOE_ERR_SHAPE, "%s: %s=%lld must be a multiple of 8, at least %lld and at most 2^32", f, name,
                (long long)ld, (long long)row);
  return MOE_OK;
}

int check_count(const char* f, const char* name, int n) {
  if (n < 1 || n > kMaxHeads) return fail(MOE_ERR_SHAPE, "%s: %s=%d outside [1, %d]", f, name, n, kMaxHeads);
  return MOE_OK;
}

int check_angles(const char* f, int rot, const int32_t* pos, const double* freq) {
  if (rot > 0 && (!pos || !freq)) return fail(MOE_ERR_NULL, "%s: pos and freq are required with rot > 0", f);
  if (!aligned4(pos)) return fail(MOE_ERR_ALIGN, "%s: pos must be 4-byte aligned", f);
  if (!aligned8(freq)) return fail(MOE_ERR_ALIGN, "%s: freq must be 8-byte aligned", f);
  return MOE_OK;
}

// page_shift: the page size's logarithm.
int check_cache(const char* f, int type, int n_pages, int P, int Hkv, int& page_shift) {
  if (type != MOE_BF16 && type != MOE_I8 && type != MOE_E4M3)
    return fail(MOE_ERR_SHAPE, "%s: type=%d is none of MOE_BF16, MOE_I8 and MOE_E4M3", f, type);
  int rc = check_count(f, "Hkv", Hkv);
  if (rc) return rc;
  if (P < 16 || P > 1024 || (P & (P - 1)) != 0)
    return fail(MOE_ERR_SHAPE, "%s: P=%d must be a power of two in [16, 1024]", f, P);
  if (n_pages < 1 || (int64_t)n_pages * P > kMaxTokens)
    return fail(MOE_ERR_SHAPE, "%s: n_pages=%d must be at least 1 and hold at most 2^30 tokens", f, n_pages);
  for (page_shift = 4; (1 << page_shift) < P;) ++page_shift;
  return MOE_OK;
}

int check_scales(const char* f, int type, const float* k_scale, const float* v_scale) {
  if (type != MOE_BF16 && (!k_scale || !v_scale))
    return fail(MOE_ERR_NULL, "%s: an 8-bit cache needs k_scale and v_scale", f);
  if (type == MOE_BF16 && (k_scale || v_scale))
    return fail(MOE_ERR_SHAPE, "%s: a bf16 cache has no scales", f);
  return MOE_OK;
}

template <class... P>
int check_aligned(const char* f, P... ptrs) {
  for (const void* p : {(const void*)ptrs...})
    if (!aligned16(p)) return fail(MOE_ERR_ALIGN, "%s: tensors must be 16-byte aligned", f);
  return MOE_OK;
}

}  // namespace

extern "C" {

int moe_rope_frequencies(int rot, double base, int scaling, double factor, double original, double* freq,
                         float* mscale) {
  const char* f = "moe_rope_frequencies";
  if (rot < 2 || rot > kMaxHeadDim || rot % 2 != 0)
    return fail(MOE_ERR_SHAPE, "%s: rot=%d must be an even number in [2, %d]", f, rot, kMaxHeadDim);
  if (!(base > 1.0) || !isfinite(base)) return fail(MOE_ERR_SHAPE, "%s: base must be above 1", f);
  if (scaling < MOE_ROPE_PLAIN || scaling > MOE_ROPE_YARN)
    return fail(MOE_ERR_SHAPE, "%s: scaling=%d is no scaling", f, scaling);
  if (scaling != MOE_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor)))
    return fail(MOE_ERR_SHAPE, "%s: factor must be at least 1", f);
  if (scaling == MOE_ROPE_YARN && (!(original >= 1.0) || !isfinite(original)))
    return fail(MOE_ERR_SHAPE, "%s: original must be at least 1", f);
  if (scaling == MOE_ROPE_NTK && rot == 2) return fail(MOE_ERR_SHAPE, "%s: MOE_ROPE_NTK needs rot of 4 or more", f);
  if (!freq || !mscale) return fail(MOE_ERR_NULL, "%s: freq and mscale are required", f);
  const double two_pi = 6.283185307179586;
  const double b = scaling == MOE_ROPE_NTK ? base * pow(factor, rot / (rot - 2.0)) : base;
  // pairs that turn 32 times and once within the original context
  const double at32 = rot * log(original / (32.0 * two_pi)) / (2.0 * log(b));
  const double at1 = rot * log(original / two_pi) / (2.0 * log(b));
  const double lo = fmax(floor(at32), 0.0), hi = fmin(ceil(at1), rot - 1.0);
  for (int i = 0; i < rot / 2; ++i) {
    double v = pow(b, -2.0 * i / rot) / two_pi;
    if (scaling == MOE_ROPE_LINEAR) v /= factor;
    if (scaling == MOE_ROPE_YARN) {
      // (at1 < 0: not even pair 0 turns once)
      const double ramp = at1 < 0.0 ? 1.0 : fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
      v = v * (1.0 - ramp) + v / factor * ramp;
    }
    freq[i] = v;
  }
  *mscale = scaling == MOE_ROPE_YARN ? (float)(0.1 * log(factor) + 1.0) : 1.0f;
  return ok();
}

int moe_rope(const uint16_t* x, int64_t x_ld, const uint16_t* w_norm, float w_add, float eps, const int32_t* pos,
             const double* freq, float mscale, int T, int heads, int D, int rot, int pairs, uint16_t* out,
             int64_t out_ld, void* stream) {
  const char* f = "moe_rope";
  int rc = check_heads(f, T, D, rot, pairs, eps, mscale);
  if (rc || (rc = check_count(f, "heads", heads)) || (rc = check_ld(f, "x_ld", x_ld, (int64_t)heads * D)) ||
      (rc = check_ld(f, "out_ld", out_ld, (int64_t)heads * D)))
    return rc;
  if (T == 0) return ok();
  if (!x || !out) return fail(MOE_ERR_NULL, "%s: x and out are required", f);
  if (x == out && x_ld != out_ld) return fail(MOE_ERR_SHAPE, "%s: in place x_ld and out_ld must be equal", f);
  if ((rc = check_angles(f, rot, pos, freq)) || (rc = check_aligned(f, x, w_norm, out)) || (rc = check_arch()))
    return rc;
  HeadArgs a = {};
  a.q = x, a.q_ld = x_ld, a.w_q = w_norm, a.q_out = out, a.out_ld = out_ld;
  a.w_add = w_add, a.eps = eps, a.mscale = mscale, a.pos = pos, a.freq = freq;
  a.T = T, a.Hq = heads, a.D = D, a.rot = rot, a.interleaved = pairs == MOE_ROPE_INTERLEAVED;
  return hip_status(launch_heads(a, (hipStream_t)stream), f);
}

int moe_cache_write(const uint16_t* q, int64_t q_ld, const uint16_t* w_q, uint16_t* q_out, int64_t q_out_ld,
                    const uint16_t* k, int64_t k_ld, const uint16_t* w_k, const uint16_t* v, int64_t v_ld, float w_add,
                    float eps, const int32_t* pos, const double* freq, float mscale, const int32_t* slots, int T,
                    int Hq, int Hkv, int D, int rot, int pairs, int type, int n_pages, int P, void* k_cache,
                    void* v_cache, float* k_scale, float* v_scale, void* stream) {
  const char* f = "moe_cache_write";
  int shift = 0, rc = check_heads(f, T, D, rot, pairs, eps, mscale);
  if (rc || (rc = check_cache(f, type, n_pages, P, Hkv, shift))) return rc;
  if (Hq < 0 || Hq > kMaxHeads) return fail(MOE_ERR_SHAPE, "%s: Hq=%d outside [0, %d]", f, Hq, kMaxHeads);
  if ((rc = check_ld(f, "k_ld", k_ld, (int64_t)Hkv * D)) || (rc = check_ld(f, "v_ld", v_ld, (int64_t)Hkv * D)))
    return rc;
  if (Hq > 0 && ((rc = check_ld(f, "q_ld", q_ld, (int64_t)Hq * D)) ||
                 (rc = check_ld(f, "q_out_ld", q_out_ld, (int64_t)Hq * D))))
    return rc;
  if (T == 0) return ok();
  if (Hq > 0 && (!q || !q_out)) return fail(MOE_ERR_NULL, "%s: q and q_out are required with Hq > 0", f);
  if (Hq == 0 && (q || q_out || w_q)) return fail(MOE_ERR_SHAPE, "%s: q, q_out or w_q given with Hq = 0", f);
  if (Hq > 0 && q == q_out && q_ld != q_out_ld)
    return fail(MOE_ERR_SHAPE, "%s: in place q_ld and q_out_ld must be equal", f);
  if (!k || !v || !slots || !k_cache || !v_cache)
    return fail(MOE_ERR_NULL, "%s: k, v, slots and the caches are required", f);
  if ((rc = check_scales(f, type, k_scale, v_scale)) || (rc = check_angles(f, rot, pos, freq)) ||
      (rc = check_aligned(f, q, w_q, q_out, k, w_k, v, k_cache, v_cache)))
    return rc;
  for (const void* s : {(const void*)slots, (const void*)k_scale, (const void*)v_scale})
    if (!aligned4(s)) return fail(MOE_ERR_ALIGN, "%s: slots and scales must be 4-byte aligned", f);
  if ((rc = check_arch())) return rc;
  HeadArgs a = {};
  a.q = q, a.q_ld = q_ld, a.w_q = w_q, a.q_out = q_out, a.out_ld = q_out_ld;
  a.k = k, a.k_ld = k_ld, a.w_k = w_k, a.v = v, a.v_ld = v_ld;
  a.w_add = w_add, a.eps = eps, a.mscale = mscale, a.pos = pos, a.freq = freq, a.slots = slots;
  a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.D = D, a.rot = rot, a.interleaved = pairs == MOE_ROPE_INTERLEAVED;
  a.type = type, a.n_slots = n_pages * P, a.page_shift = shift;
  a.k_cache = k_cache, a.v_cache = v_cache, a.k_scale = k_scale, a.v_scale = v_scale;
  return hip_status(launch_heads(a, (hipStream_t)stream), f);
}

int moe_cache_read(const void* k_cache, const void* v_cache, const float* k_scale, const float* v_scale, int type,
                   int n_pages, int P, const int32_t* slots, int n, int Hkv, int D, void* k, void* v, int out_type,
                   void* stream) {
  const char* f = "moe_cache_read";
  int shift = 0, rc = check_heads(f, 0, D, 0, MOE_ROPE_HALF, 0.0f, 1.0f);
  if (rc || (rc = check_cache(f, type, n_pages, P, Hkv, shift))) return rc;
  if (n < 0 || n > kMaxT) return fail(MOE_ERR_SHAPE, "%s: n=%d outside [0, 2^24]", f, n);
  if (out_type != MOE_BF16 && out_type != MOE_F32)
    return fail(MOE_ERR_SHAPE, "%s: out_type=%d is neither MOE_BF16 nor MOE_F32", f, out_type);
  if (n == 0) return ok();
  if (!k_cache || !v_cache || !slots || !k || !v)
    return fail(MOE_ERR_NULL, "%s: the caches, slots, k and v are required", f);
  if ((rc = check_scales(f, type, k_scale, v_scale)) || (rc = check_aligned(f, k_cache, v_cache, k, v))) return rc;
  for (const void* s : {(const void*)slots, (const void*)k_scale, (const void*)v_scale})
    if (!aligned4(s)) return fail(MOE_ERR_ALIGN, "%s: slots and scales must be 4-byte aligned", f);
  if ((rc = check_arch())) return rc;
  CacheReadArgs a = {};
  a.k_cache = k_cache, a.v_cache = v_cache, a.k_scale = k_scale, a.v_scale = v_scale;
  a.type = type, a.n_slots = n_pages * P, a.page_shift = shift, a.n = n, a.Hkv = Hkv, a.D = D, a.slots = slots;
  a.k = k, a.v = v, a.out_f32 = out_type == MOE_F32;
  return hip_status(launch_cache_read(a, (hipStream_t)stream), f);
}

static int check_attention(const char* f, int T, int S, int Hq, int Hkv, int D) {
  int rc;
  if (T < 0 || T > kMaxT) return fail(MOE_ERR_SHAPE, "%s: T=%d outside [0, 2^24]", f, T);
  if ((rc = check_count(f, "Hq", Hq)) || (rc = check_count(f, "Hkv", Hkv))) return rc;
  if (Hq % Hkv != 0) return fail(MOE_ERR_SHAPE, "%s: Hq=%d must be a multiple of Hkv=%d", f, Hq, Hkv);
  if (D != 64 && D != 128 && D != 256) return fail(MOE_ERR_SHAPE, "%s: D=%d is none of 64, 128 and 256", f, D);
  if ((int64_t)T * Hq > kMaxRows) return fail(MOE_ERR_SHAPE, "%s: T * Hq exceeds 2^30", f);
  if (S < 0 || (int64_t)S * Hkv > kMaxPairs)
    return fail(MOE_ERR_SHAPE, "%s: S=%d must not be negative nor S * Hkv exceed 2^22", f, S);
  return MOE_OK;
}

size_t moe_attention_workspace_size(int T, int S, int Hq, int Hkv, int D, int64_t max_keys) {
  const char* f = "moe_attention_workspace_size";
  if (check_attention(f, T, S, Hq, Hkv, D)) return 0;
  if (max_keys < 0 || max_keys > kMaxTokens) {
    fail(MOE_ERR_SHAPE, "%s: max_keys=%lld outside [0, 2^30]", f, (long long)max_keys);
    return 0;
  }
  ok();
  return T == 0 || S == 0 ? 0 : attention_workspace(T, S, Hq, Hkv, D, max_keys);
}

int moe_attention(const uint16_t* q, int64_t q_ld, const void* k_cache, const void* v_cache, const float* k_scale,
                  const float* v_scale, int type, const int32_t* pages, const int32_t* q_start, const int32_t* kv_len,
                  int T, int S, int Hq, int Hkv, int D, int n_pages, int P, int max_pages, float scale, int window,
                  uint16_t* out, int64_t out_ld, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const char* f = "moe_attention";
  int shift = 0, rc = check_attention(f, T, S, Hq, Hkv, D);
  if (rc || (rc = check_cache(f, type, n_pages, P, Hkv, shift))) return rc;
  if (max_pages < 1 || (int64_t)max_pages * P > kMaxTokens)
    return fail(MOE_ERR_SHAPE, "%s: max_pages=%d must be at least 1 and hold at most 2^30 tokens", f, max_pages);
  if (!(scale > 0.0f) || !isfinite(scale)) return fail(MOE_ERR_SHAPE, "%s: scale must be positive and finite", f);
  if (window < 0) return fail(MOE_ERR_SHAPE, "%s: window must not be negative", f);
  if ((rc = check_ld(f, "q_ld", q_ld, (int64_t)Hq * D)) || (rc = check_ld(f, "out_ld", out_ld, (int64_t)Hq * D)))
    return rc;
  if (T == 0 || S == 0) return ok();
  if (!q || !k_cache || !v_cache || !pages || !q_start || !kv_len || !out)
    return fail(MOE_ERR_NULL, "%s: q, the caches, pages, q_start, kv_len and out are required", f);
  if (q == out && q_ld != out_ld) return fail(MOE_ERR_SHAPE, "%s: in place q_ld and out_ld must be equal", f);
  if ((rc = check_scales(f, type, k_scale, v_scale)) || (rc = check_aligned(f, q, k_cache, v_cache, out))) return rc;
  for (const void* s : {(const void*)pages, (const void*)q_start, (const void*)kv_len, (const void*)lse,
                        (const void*)k_scale, (const void*)v_scale})
    if (!aligned4(s))
      return fail(MOE_ERR_ALIGN, "%s: pages, q_start, kv_len, lse and scales must be 4-byte aligned", f);
  const size_t need = attention_workspace(T, S, Hq, Hkv, D, (int64_t)max_pages * P);
  if (need > 0) {
    if (!workspace) return fail(MOE_ERR_NULL, "%s: these sizes need a workspace of %zu bytes", f, need);
    if (!aligned16(workspace)) return fail(MOE_ERR_ALIGN, "%s: workspace must be 16-byte aligned", f);
    if (workspace_bytes < need)
      return fail(MOE_ERR_WORKSPACE, "%s: workspace of %zu bytes; %zu needed", f, workspace_bytes, need);
  }
  if ((rc = check_arch())) return rc;
  AttentionArgs a = {};
  a.q = q, a.q_ld = q_ld, a.out = out, a.out_ld = out_ld, a.lse = lse;
  a.k_cache = k_cache, a.v_cache = v_cache, a.k_scale = k_scale, a.v_scale = v_scale, a.type = type;
  a.pages = pages, a.q_start = q_start, a.kv_len = kv_len;
  a.T = T, a.S = S, a.Hq = Hq, a.Hkv = Hkv, a.D = D, a.G = Hq / Hkv;
  a.n_pages = n_pages, a.page_shift = shift, a.max_pages = max_pages;
  a.scale = (float)(scale * 1.4426950408889634);
  // no sequence is longer than 2^30
  a.window = window > (1 << 30) ? 0 : window;
  a.partial = static_cast<float*>(workspace);
  return hip_status(launch_attention(a, (hipStream_t)stream), f);
}

}  // extern "C"

namespace moe {

size_t attention_workspace(int T, int S, int Hq, int Hkv, int D, int64_t max_keys) {
  // the type only widens row tiles that are not shared out, and with a window there are no more shares than without
  const attn::Plan p = attn::plan_of(MOE_BF16, T, S, Hq, Hkv, D, max_keys, 0);
  return p.stream && p.grid > 1 ? p.grid * (sizeof(attn::Part) + (size_t)2 * p.rows * (D + 2) * sizeof(float)) : 0;
}

hipError_t launch_attention(const AttentionArgs& a, hipStream_t st) {
  const int64_t max_keys = (int64_t)a.max_pages << a.page_shift;
  const attn::Plan p = attn::plan_of(a.type, a.T, a.S, a.Hq, a.Hkv, a.D, max_keys, a.window);
  if (a.type == MOE_I8) return attn::run_i8(a, p, st);
  if (a.type == MOE_E4M3) return attn::run_e4m3(a, p, st);
  return attn::run_bf16(a, p, st);
}

}  // namespace moe
