// The block boundary's gradient in fp32 (zero_join_back.cuh), a source of its own so that the types
// compile side by side.
#include "zero_join_back.cuh"

namespace zk {

cudaError_t join_back_f32(const JoinArgs& a, float* ws, cudaStream_t stream) {
    return run_join_back<float>(a, ws, stream);
}

}  // namespace zk
