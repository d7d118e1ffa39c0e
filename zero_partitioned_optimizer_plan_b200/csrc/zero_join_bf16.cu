// The block boundary in bfloat16 (zero_join_forward.cuh), a source of its own so that the types compile
// side by side.
#include "zero_join_forward.cuh"

namespace zk {

cudaError_t join_bf16(const JoinArgs& a, cudaStream_t stream) { return run_join<bf16>(a, stream); }

}  // namespace zk
