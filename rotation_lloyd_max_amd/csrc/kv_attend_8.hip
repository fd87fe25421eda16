// Attention kernels for keys of 8 bits.
#include "kv_attend.hpp"

namespace tq {

template hipError_t at_launch_k<8>(const AttendParams& p, int vbits, int D, int R, hipStream_t s);

}  // namespace tq
