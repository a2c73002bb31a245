// q4_matvec64.hip - 4-bit products with groups of 64 inputs.
#include "q4_matvec.h"

namespace q2dev {
template hipError_t launch_matvec<GROUP_64>(const MatvecArgs&, hipStream_t);
}
