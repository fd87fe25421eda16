// Attention kernels for keys of 8 bits.
#include "kv_attend_wide.hpp"

namespace tq {

template hipError_t at_launch_k<8>(const AttendParams& p, int vbits, int D, int rows, hipStream_t s);

}  // namespace tq
