// Dense 4-bit product: the kernels of one weight format.
#define MOE_LINEAR_INST
#include "moe_linear_launch.h"

namespace moeq4 {
template int linear_launch<kLinAffine32>(bool, const LinearArgs&, unsigned char*, hipStream_t);
}
