// kern_mlp_f32.hip - kernel builds of the gated feed-forward block's products
// on f32 operands (see mlp.hpp).
#include "mlp.hpp"

namespace nsr {

NS_MLP_LAUNCHERS(float)

}  // namespace nsr
