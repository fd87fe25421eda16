// Attention kernels for keys of 3 bits.
#include "kv_attend_wide.hpp"

namespace tq {

template hipError_t at_launch_k<3>(const AttendParams& p, int vbits, int D, int rows, hipStream_t s);

}  // namespace tq
