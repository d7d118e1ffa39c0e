// The block boundary in fp16 (zero_join_forward.cuh), a source of its own so that the types compile
// side by side.
#include "zero_join_forward.cuh"

namespace zk {

cudaError_t join_f16(const JoinArgs& a, cudaStream_t stream) { return run_join<__half>(a, stream); }

cudaError_t launch_join(const JoinArgs& a, int dtype, cudaStream_t stream) {
    return dtype == ZERO_F16    ? join_f16(a, stream)
           : dtype == ZERO_BF16 ? join_bf16(a, stream)
                                : join_f32(a, stream);
}

}  // namespace zk
