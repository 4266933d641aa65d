// Attention over the 4-bit key/value cache: the bfloat16 kernels.
#include "attention_kernels.h"

namespace i8mp {

hipError_t launch_kv_attention_bf16(const KvAttnArgs& a, hipStream_t stream) {
    return a.c.blocks == 1 ? launch<true, 1>(a, stream) : a.c.blocks == 2 ? launch<true, 2>(a, stream) : launch<true, 4>(a, stream);
}

}  // namespace i8mp
