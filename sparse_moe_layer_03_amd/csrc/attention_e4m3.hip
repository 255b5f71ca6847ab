// Attention over a paged cache of type MOE_E4M3.
#include "attention_kernel.h"

namespace moe {
namespace attn {

hipError_t run_e4m3(const AttentionArgs& a, const Plan& plan, hipStream_t st) { return run_all<MOE_E4M3>(a, plan, st); }

}  // namespace attn
}  // namespace moe
