// The block boundary's gradient in fp16 (zero_join_back.cuh), a source of its own so that the types
// compile side by side.
#include "zero_join_back.cuh"

namespace zk {

cudaError_t join_back_f16(const JoinArgs& a, float* ws, cudaStream_t stream) {
    return run_join_back<__half>(a, ws, stream);
}

// Enough for every type and set of outputs: the vectors' partial sums, and a partial gate row
// per team (at least as many as units) where a gate row's rows may be dealt to several.
uint64_t join_workspace(uint64_t rows, uint64_t cols, uint64_t gate_rows) {
    if (cols == 0) return 0;
    uint64_t floats = vector_partials((uint32_t)cols);
    if (gate_rows && rows) {
        uint64_t most = 0;
        for (const uint32_t warps : {8u, 12u, 16u})
            for (const uint32_t chunks : {1u, 2u}) {
                const BackGeom g = back_geom((uint32_t)rows, cols,
                                             (uint32_t)(gate_rows < rows ? gate_rows : rows),
                                             chunks, warps, kMaxParts);
                if (g.parts > 1 && g.clusters * g.teams > most) most = g.clusters * g.teams;
            }
        floats += most * cols;
    }
    return (floats * 4 + 15) / 16 * 16;
}

cudaError_t launch_join_backward(const JoinArgs& a, int dtype, void* ws, cudaStream_t stream) {
    return dtype == ZERO_F16    ? join_back_f16(a, (float*)ws, stream)
           : dtype == ZERO_BF16 ? join_back_bf16(a, (float*)ws, stream)
                                : join_back_f32(a, (float*)ws, stream);
}

}  // namespace zk
