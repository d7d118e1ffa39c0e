// The block boundary in fp32 (zero_join_forward.cuh), a source of its own so that the types compile
// side by side.
#include "zero_join_forward.cuh"

namespace zk {

cudaError_t join_f32(const JoinArgs& a, cudaStream_t stream) { return run_join<float>(a, stream); }

}  // namespace zk
