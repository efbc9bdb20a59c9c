// moe_fwd_gate_up_generic.hip -- the MoE forward's gate/up kernel for H not a multiple of 128.
#include "moe_fwd_gate_up.hpp"

namespace mx {

template hipError_t fwd_gate_up_launch<128, 128, true>(MoeFwdArgs, hipStream_t);

}  // namespace mx
