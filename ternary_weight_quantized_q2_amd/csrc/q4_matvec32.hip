// q4_matvec32.hip - 4-bit products with groups of 32 inputs.
#include "q4_matvec.h"

namespace q2dev {
template hipError_t launch_matvec<GROUP_32>(const MatvecArgs&, hipStream_t);
}
