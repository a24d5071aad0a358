// kern_xent_f32.hip - kernel builds of the cross entropy's products on fp32
// operands (see xent.hpp).
#include "xent.hpp"

namespace nsr {

NS_XENT_LAUNCHERS(float)

}  // namespace nsr
