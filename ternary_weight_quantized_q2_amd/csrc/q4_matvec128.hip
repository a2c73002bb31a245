// q4_matvec128.hip - 4-bit products with groups of 128 inputs and their multiples.
#include "q4_matvec.h"

namespace q2dev {
template hipError_t launch_matvec<GROUP_128>(const MatvecArgs&, hipStream_t);
}
