// kern_mlp_f16.hip - kernel builds of the gated feed-forward block's products
// on f16 operands (see mlp.hpp).
#include "mlp.hpp"

namespace nsr {

NS_MLP_LAUNCHERS(_Float16)

}  // namespace nsr
