// qmm_attn_f16_f16.hip -- the attention kernels of one pair of key and value
// kinds (each pair compiles on its own, in parallel).
#include "qmm_attn.h"

namespace qmm {
namespace attn {
hipError_t launch_f16_f16(Args &a, int NB, int f16, hipStream_t s) { return run_kinds<C_F16, C_F16>(a, NB, f16, s); }
}  // namespace attn
}  // namespace qmm
