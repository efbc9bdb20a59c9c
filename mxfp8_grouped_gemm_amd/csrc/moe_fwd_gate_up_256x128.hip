// moe_fwd_gate_up_256x128.hip -- the MoE forward's gate/up kernel at 256 x 128 tiles.
#include "moe_fwd_gate_up.hpp"

namespace mx {

template hipError_t fwd_gate_up_launch<256, 128>(MoeFwdArgs, hipStream_t);

}  // namespace mx
