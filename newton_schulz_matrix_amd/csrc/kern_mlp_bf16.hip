// kern_mlp_bf16.hip - kernel builds of the gated feed-forward block's products
// on bf16 operands (see mlp.hpp).
#include "mlp.hpp"

namespace nsr {

NS_MLP_LAUNCHERS(__bf16)

}  // namespace nsr
