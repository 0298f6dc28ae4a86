// linear_attn_f32.hip -- the chunked linear-attention kernels for fp32 io.
#include "linear_attn_kernel.h"

namespace linattn {

hipError_t launch_f32(const Args& a, int64_t blocks, bool state_only, hipStream_t st) {
  return launch<float>(a, blocks, state_only, st);
}

}  // namespace linattn
