// kern_xent_bf16.hip - kernel builds of the cross entropy's products on bf16
// operands (see xent.hpp).
#include "xent.hpp"

namespace nsr {

NS_XENT_LAUNCHERS(__bf16)

}  // namespace nsr
