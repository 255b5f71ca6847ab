// Attention over a paged cache of type MOE_BF16.
#include "attention_kernel.h"

namespace moe {
namespace attn {

hipError_t run_bf16(const AttentionArgs& a, const Plan& plan, hipStream_t st) { return run_all<MOE_BF16>(a, plan, st); }

}  // namespace attn
}  // namespace moe
