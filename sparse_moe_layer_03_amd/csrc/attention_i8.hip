// Attention over a paged cache of type MOE_I8.
#include "attention_kernel.h"

namespace moe {
namespace attn {

hipError_t run_i8(const AttentionArgs& a, const Plan& plan, hipStream_t st) { return run_all<MOE_I8>(a, plan, st); }

}  // namespace attn
}  // namespace moe
