// C ABI of the operators around the layer: argument checks, all before anything is enqueued.
#include "api_checks.h"
#include "block_internal.h"

using namespace moe;

namespace {

int check_rows(const char* f, int R) {
  if (R < 0 || R > kMaxProductRows) return fail(MOE_ERR_SHAPE, "%s: %d rows outside [0, 2^28]", f, R);
  return MOE_OK;
}

int check_product(const char* f, int N, int K, int kmul, int c_type) {
  if (N < 8 || N > kMaxProductN || N % 8 != 0)
    return fail(MOE_ERR_SHAPE, "%s: N=%d must be a multiple of 8 in [8, 2^20]", f, N);
  if (K < kmul || K > kMaxProductK || K % kmul != 0)
    return fail(MOE_ERR_SHAPE, "%s: K=%d must be a multiple of %d in [%d, 65536]", f, K, kmul, kmul);
  if (c_type != MOE_BF16 && c_type != MOE_F32)
    return fail(MOE_ERR_SHAPE, "%s: c_type=%d is neither MOE_BF16 nor MOE_F32", f, c_type);
  return MOE_OK;
}

int check_out(const char* f, int P, int N) {
  if ((int64_t)P * N > kMaxProductOut) return fail(MOE_ERR_SHAPE, "%s: %d rows of %d columns exceed 2^37", f, P, N);
  return MOE_OK;
}

int quantize_args(const char* f, const uint16_t* x, int R, int K, int8_t* q, float* scale) {
  int rc = check_rows(f, R);
  if (rc) return rc;
  if (K < 16 || K > kMaxQuantK || K % 16 != 0)
    return fail(MOE_ERR_SHAPE, "%s: row length %d must be a multiple of 16 in [16, 32768]", f, K);
  if (R == 0) return MOE_OK;
  if (!x || !q || !scale) return fail(MOE_ERR_NULL, "%s: the input, q and scale are required", f);
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale))
    return fail(MOE_ERR_ALIGN, "%s: tensors must be 16-byte aligned", f);
  return MOE_OK;
}

int grouped(const char* f, const void* a, const float* a_scale, const void* b, const float* b_scale,
            const int32_t* off, const int32_t* counts, const int32_t* rows, int a_div, int P, int R, int E, int N,
            int K, void* c, int c_type, bool i8, void* stream) {
  int rc = check_product(f, N, K, i8 ? 16 : 8, c_type);
  if (rc || (rc = check_rows(f, P)) || (rc = check_rows(f, R)) || (rc = check_out(f, P, N))) return rc;
  if (E < 1 || E > kMaxE) return fail(MOE_ERR_SHAPE, "%s: E=%d outside [1, %d]", f, E, kMaxE);
  if (a_div < 1) return fail(MOE_ERR_SHAPE, "%s: a_div=%d must be at least 1", f, a_div);
  if (P == 0 || R == 0) return ok();
  if (!a || !b || !off || !c || (i8 && (!a_scale || !b_scale)))
    return fail(MOE_ERR_NULL, "%s: a, b, off, c%s are required", f, i8 ? ", a_scale and b_scale" : "");
  for (const void* q : {a, b, (const void*)a_scale, (const void*)b_scale, (const void*)c})
    if (!aligned16(q)) return fail(MOE_ERR_ALIGN, "%s: tensors must be 16-byte aligned", f);
  if (!aligned4(off) || !aligned4(counts) || !aligned4(rows))
    return fail(MOE_ERR_ALIGN, "%s: off, counts and rows must be 4-byte aligned", f);
  if ((rc = check_arch())) return rc;
  ProductArgs p = {};
  p.a = a, p.b = b, p.a_scale = a_scale, p.b_scale = b_scale;
  p.off = off, p.counts = counts, p.rows = rows, p.a_div = a_div;
  p.P = P, p.R = R, p.E = E, p.N = N, p.Kb = i8 ? K : 2 * K, p.c = c, p.c_f32 = c_type == MOE_F32;
  return hip_status(launch_product(p, i8, (hipStream_t)stream), f);
}

}  // namespace

extern "C" {

int moe_block_norm(const void* r, int r_type, const uint16_t* y, const uint16_t* w_post, const uint16_t* gate,
                   int gate_rows, float r_scale, float y_scale, const uint16_t* w_pre, float w_add, float eps, int T,
                   int H, void* r_out, uint16_t* x, int8_t* q, float* q_scale, void* stream) {
  const char* f = "moe_block_norm";
  if (T < 0 || T > (1 << 24)) return fail(MOE_ERR_SHAPE, "%s: T=%d outside [0, 2^24]", f, T);
  if (H < 16 || H > kMaxNormH || H % 16 != 0)
    return fail(MOE_ERR_SHAPE, "%s: H=%d must be a multiple of 16 in [16, %d]", f, H, kMaxNormH);
  if (r_type != MOE_BF16 && r_type != MOE_F32)
    return fail(MOE_ERR_SHAPE, "%s: r_type=%d is neither MOE_BF16 nor MOE_F32", f, r_type);
  if (!(eps >= 0.0f)) return fail(MOE_ERR_SHAPE, "%s: eps must not be negative", f);
  if (T == 0) return ok();  // tensors without elements have no address
  if (!y && (w_post || gate)) return fail(MOE_ERR_SHAPE, "%s: w_post or gate given without y", f);
  if (gate && gate_rows != 1 && gate_rows != T)
    return fail(MOE_ERR_SHAPE, "%s: gate_rows=%d must be 1 or T=%d", f, gate_rows, T);
  if ((q == nullptr) != (q_scale == nullptr)) return fail(MOE_ERR_NULL, "%s: q and q_scale go together", f);
  if ((w_pre != nullptr) != (x || q)) return fail(MOE_ERR_NULL, "%s: w_pre goes together with x or q", f);
  if (!r_out && !w_pre) return fail(MOE_ERR_NULL, "%s: no output", f);
  if (!r) return fail(MOE_ERR_NULL, "%s: r is required", f);
  for (const void* p : {r, (const void*)y, (const void*)w_post, (const void*)gate, (const void*)w_pre,
                        (const void*)r_out, (const void*)x, (const void*)q, (const void*)q_scale})
    if (!aligned16(p)) return fail(MOE_ERR_ALIGN, "%s: tensors must be 16-byte aligned", f);
  int rc = check_arch();
  if (rc) return rc;
  NormArgs a = {};
  a.r = r, a.y = y, a.w_post = w_post, a.gate = gate, a.gate_ld = gate && gate_rows != 1 ? H : 0, a.w_pre = w_pre;
  a.r_scale = r_scale, a.y_scale = y_scale, a.w_add = w_add, a.eps = eps, a.T = T, a.H = H;
  a.r_out = r_out, a.x = x, a.q = q, a.q_scale = q_scale, a.f32 = r_type == MOE_F32;
  return hip_status(launch_block_norm(a, (hipStream_t)stream), f);
}

int moe_quantize_i8(const uint16_t* x, int R, int K, int8_t* q, float* scale, void* stream) {
  int rc = quantize_args("moe_quantize_i8", x, R, K, q, scale);
  if (rc) return rc;
  if (R == 0) return ok();
  if ((rc = check_arch())) return rc;
  return hip_status(launch_quantize_i8(x, R, K, q, scale, (hipStream_t)stream), "moe_quantize_i8");
}

int moe_swiglu_i8(const uint16_t* gu, const float* row_gate, int R, int I, int8_t* q, float* scale, void* stream) {
  int rc = quantize_args("moe_swiglu_i8", gu, R, I, q, scale);
  if (rc) return rc;
  if (R == 0) return ok();
  if (!aligned4(row_gate)) return fail(MOE_ERR_ALIGN, "moe_swiglu_i8: row_gate must be 4-byte aligned");
  if ((rc = check_arch())) return rc;
  return hip_status(launch_swiglu_i8(gu, row_gate, R, I, q, scale, (hipStream_t)stream), "moe_swiglu_i8");
}

int moe_gemm_i8(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale, const float* bias,
                const uint16_t* add, int M, int N, int K, void* c, int c_type, void* stream) {
  const char* f = "moe_gemm_i8";
  int rc = check_product(f, N, K, 16, c_type);
  if (rc || (rc = check_rows(f, M)) || (rc = check_out(f, M, N))) return rc;
  if (M == 0) return ok();
  if (!a || !a_scale || !b || !b_scale || !c)
    return fail(MOE_ERR_NULL, "%s: a, a_scale, b, b_scale and c are required", f);
  for (const void* q : {(const void*)a, (const void*)a_scale, (const void*)b, (const void*)b_scale, (const void*)bias,
                        (const void*)add, (const void*)c})
    if (!aligned16(q)) return fail(MOE_ERR_ALIGN, "%s: tensors must be 16-byte aligned", f);
  if ((rc = check_arch())) return rc;
  ProductArgs p = {};
  p.a = a, p.b = b, p.a_scale = a_scale, p.b_scale = b_scale, p.bias = bias, p.add = add, p.a_div = 1;
  p.P = M, p.R = M, p.E = 1, p.N = N, p.Kb = K, p.c = c, p.c_f32 = c_type == MOE_F32;
  return hip_status(launch_product(p, true, (hipStream_t)stream), f);
}

int moe_gemm(const uint16_t* a, const uint16_t* b, const float* bias, int act, const uint16_t* add, int M, int N, int K,
             void* c, int c_type, void* stream) {
  const char* f = "moe_gemm";
  int rc = check_product(f, N, K, 8, c_type);
  if (rc || (rc = check_rows(f, M)) || (rc = check_out(f, M, N))) return rc;
  if (act != MOE_ACT_NONE && act != MOE_ACT_SILU && act != MOE_ACT_GELU)
    return fail(MOE_ERR_SHAPE, "%s: act=%d is no MOE_ACT_ value", f, act);
  if (M == 0) return ok();
  if (!a || !b || !c) return fail(MOE_ERR_NULL, "%s: a, b and c are required", f);
  for (const void* q : {(const void*)a, (const void*)b, (const void*)bias, (const void*)add, (const void*)c})
    if (!aligned16(q)) return fail(MOE_ERR_ALIGN, "%s: tensors must be 16-byte aligned", f);
  if ((rc = check_arch())) return rc;
  ProductArgs p = {};
  p.a = a, p.b = b, p.bias = bias, p.act = act, p.add = add, p.a_div = 1;
  p.P = M, p.R = M, p.E = 1, p.N = N, p.Kb = 2 * K, p.c = c, p.c_f32 = c_type == MOE_F32;
  return hip_status(launch_product(p, false, (hipStream_t)stream), f);
}

int moe_grouped_gemm(const uint16_t* a, const uint16_t* b, const int32_t* off, const int32_t* counts,
                     const int32_t* rows, int a_div, int P, int R, int E, int N, int K, void* c, int c_type,
                     void* stream) {
  return grouped("moe_grouped_gemm", a, nullptr, b, nullptr, off, counts, rows, a_div, P, R, E, N, K, c, c_type, false,
                 stream);
}

int moe_grouped_gemm_i8(const int8_t* a, const float* a_scale, const int8_t* b, const float* b_scale,
                        const int32_t* off, const int32_t* counts, const int32_t* rows, int a_div, int P, int R, int E,
                        int N, int K, void* c, int c_type, void* stream) {
  return grouped("moe_grouped_gemm_i8", a, a_scale, b, b_scale, off, counts, rows, a_div, P, R, E, N, K, c, c_type,
                 true, stream);
}

}  // extern "C"
