// moe_fwd_gate_up_256.hip -- the MoE forward's gate/up kernel at 256 x 256 tiles.
#include "moe_fwd_gate_up.hpp"

namespace mx {

template hipError_t fwd_gate_up_launch<256, 256, v3::kFp8>(MoeFwdArgs, hipStream_t);

}  // namespace mx
