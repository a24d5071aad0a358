// kern_xent_f16.hip - kernel builds of the cross entropy's products on fp16
// operands (see xent.hpp).
#include "xent.hpp"

namespace nsr {

NS_XENT_LAUNCHERS(_Float16)

}  // namespace nsr
