// Internal declarations of the operators around attention: rotary positions, the paged cache, attention over it (see
// include/moe.h).
#pragma once

#include "block_internal.h"
#include "moe.h"

namespace moe {

constexpr int kMaxHeadDim = 256;

// Heads of q, k and v rows on their way: rotated to q_out, or into the cache.
struct HeadArgs {
  const uint16_t* q;  // [T, Hq * D], rows q_ld apart
  const uint16_t* k;  // [T, Hkv * D], rows k_ld apart; Hkv 0: no cache
  const uint16_t* v;
  int64_t q_ld, k_ld, v_ld, out_ld;
  const uint16_t* w_q;  // norm weights [D] or NULL
  const uint16_t* w_k;
  uint16_t* q_out;
  float w_add, eps, mscale;
  const int32_t* pos;
  const double* freq;
  const int32_t* slots;
  int T, Hq, Hkv, D, rot, interleaved;
  int type;     // of the cache
  int n_slots;  // pages times tokens of a page
  int page_shift;
  void* k_cache;
  void* v_cache;
  float* k_scale;
  float* v_scale;
};
hipError_t launch_heads(const HeadArgs& a, hipStream_t st);

struct CacheReadArgs {
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  int type, n_slots, page_shift, n, Hkv, D;
  const int32_t* slots;
  void* k;
  void* v;
  int out_f32;
};
hipError_t launch_cache_read(const CacheReadArgs& a, hipStream_t st);

struct AttentionArgs {
  const uint16_t* q;
  int64_t q_ld, out_ld;
  const void* k_cache;
  const void* v_cache;
  const float* k_scale;
  const float* v_scale;
  const int32_t* pages;    // [S, max_pages]
  const int32_t* q_start;  // [S + 1]
  const int32_t* kv_len;   // [S]
  int T, S, Hq, Hkv, D, G;  // G = Hq / Hkv
  int type, n_pages, page_shift, max_pages;
  float scale;  // of the scores, times log2 e
  int window;   // 0: none
  uint16_t* out;
  float* lse;
  float* partial;  // workspace of split sequences
};
size_t attention_workspace(int T, int S, int Hq, int Hkv, int D, int64_t max_keys);
hipError_t launch_attention(const AttentionArgs& a, hipStream_t st);

}  // namespace moe
