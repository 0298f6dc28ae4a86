// linear_attn_bf16.hip -- the chunked linear-attention kernels for bf16 io.
#include "linear_attn_kernel.h"

namespace linattn {

hipError_t launch_bf16(const Args& a, int64_t blocks, bool state_only, hipStream_t st) {
  return launch<bf16_t>(a, blocks, state_only, st);
}

}  // namespace linattn
