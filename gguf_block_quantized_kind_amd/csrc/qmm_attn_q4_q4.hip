// qmm_attn_q4_q4.hip -- the attention kernels of one pair of key and value
// kinds (each pair compiles on its own, in parallel).
#include "qmm_attn.h"

namespace qmm {
namespace attn {
hipError_t launch_q4_q4(Args &a, int NB, int f16, hipStream_t s) { return run_kinds<C_Q4_0, C_Q4_0>(a, NB, f16, s); }
}  // namespace attn
}  // namespace qmm
