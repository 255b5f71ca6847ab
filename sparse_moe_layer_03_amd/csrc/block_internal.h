// Internal declarations of the operators around the layer: norms with gate and residual scale, 8-bit
// integer rows, and dense and expert-grouped products (see include/moe.h).
#pragma once

#include "moe_internal.h"

namespace moe {

constexpr int kMaxNormH = 16384;   // a norm's row is held in one workgroup's registers
constexpr int kMaxQuantK = 32768;  // likewise a quantised row
constexpr int kMaxProductK = 65536;  // 2^14 * K stays below 2^31: the int32 sums of 8-bit products cannot overflow
constexpr int kMaxProductN = 1 << 20;
constexpr int kMaxProductRows = 1 << 28;
constexpr int64_t kMaxProductOut = (int64_t)1 << 37;  // positions times columns: output elements of 256 GB in bf16

// Rows are quantised against at least this magnitude, so that the scale and its inverse stay normal floats.
constexpr float kQuantTiny = 0x1p-100f;

// Two floats to bf16, round to nearest even, NaN kept (one gfx950 instruction).
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t cvt_bf16x2(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, (bf16x2{(__bf16)lo, (__bf16)hi}));
}

struct NormArgs {
  const void* r;  // residual rows, bf16 or fp32
  const uint16_t* y;
  const uint16_t* w_post;
  const uint16_t* gate;
  int64_t gate_ld;  // 0: one gate row for all tokens
  const uint16_t* w_pre;
  float r_scale, y_scale, w_add, eps;
  int T, H;
  void* r_out;
  uint16_t* x;
  int8_t* q;
  float* q_scale;
  int f32;  // r and r_out are fp32
};
hipError_t launch_block_norm(const NormArgs& a, hipStream_t st);

hipError_t launch_quantize_i8(const uint16_t* x, int R, int K, int8_t* q, float* scale, hipStream_t st);
hipError_t launch_swiglu_i8(const uint16_t* gu, const float* row_gate, int R, int I, int8_t* q, float* scale,
                            hipStream_t st);

// A product C = A B^T, dense (off == NULL: P rows, one matrix B) or grouped by expert.
struct ProductArgs {
  const void* a;
  const void* b;          // [E, N, K], dense: [N, K]
  const float* a_scale;   // per A row (8-bit products)
  const float* b_scale;   // per B row [E, N]
  const float* bias;      // dense: [N] or NULL
  const uint16_t* add;    // dense: [P, N] bf16 or NULL
  int act;                // dense bf16: MOE_ACT_*
  const int32_t* off;     // [E + 1] first position of each expert; NULL: dense
  const int32_t* counts;  // [E] positions of each expert, NULL: off[e + 1] - off[e]
  const int32_t* rows;    // [P] output row of each position, NULL: the position itself
  int a_div;              // A row = output row / a_div
  unsigned div_mul;       // the same division as a multiplication (set by launch_product)
  int div_shift;
  int P;                  // positions
  int R;                  // output rows; others are skipped
  int E, N;
  int Kb;                 // bytes of an A or B row, a multiple of 16
  void* c;
  int c_f32;
};
hipError_t launch_product(const ProductArgs& p, bool i8, hipStream_t st);

}  // namespace moe
