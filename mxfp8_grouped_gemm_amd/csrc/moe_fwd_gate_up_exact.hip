// moe_fwd_gate_up_exact.hip -- the gate/up kernel at 128 x 128 tiles with exact products.
#include "moe_fwd_gate_up.hpp"

namespace mx {
template hipError_t fwd_gate_up_launch<128, 128, v3::kFp8Bf16>(MoeFwdArgs, hipStream_t);
}
