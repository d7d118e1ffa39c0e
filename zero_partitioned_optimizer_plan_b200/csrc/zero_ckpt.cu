// 8-bit activation checkpoints for sm_100a: a matrix of activations to records of one byte per
// value and one fp32 scale per 128 columns, and back ("ZeRO" ZeRO-R: what partitioning the model
// states leaves is the activation checkpoints; the pages give no format, this is the library's).
//
// Per block of 128 columns of a row: scale = amax/127, q = round_half_even(x/scale), stored as
// q + 128; an inf or NaN poisons the block (scale NaN, q 0). The read is T(q*scale).
//
// One warp per block and row: lane l holds columns 4l..4l+3 of the block.
#include "zero_act.cuh"

namespace zk {
namespace {

template <typename T>
__global__ void __launch_bounds__(256) ckpt_save_kernel(uint64_t rows, CkptShape s, const T* x,
                                                        uint64_t ldx, uint8_t* ckpt) {
    grid_wait();
    const int lane = threadIdx.x & 31;
    const uint64_t units = rows * s.blocks;
    for (uint64_t w = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < units;
         w += (uint64_t)gridDim.x * 8) {
        const uint64_t r = w / s.blocks;
        const uint32_t b = (uint32_t)(w - r * s.blocks);
        const uint32_t c0 = b * 128u + lane * 4u;
        float v[4];
        uint32_t amax = 0;
        for (int j = 0; j < 4; ++j) {
            v[j] = c0 + j < s.cols ? to_f(x[r * ldx + c0 + j]) : 0.0f;
            amax = max(amax, abs_bits(v[j]));
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
        const float scale = q8_scale(amax);
        uint8_t* row = ckpt + r * s.row_bytes;
        if (c0 < s.code_bytes) {
            uint32_t word = 0;
            for (int j = 0; j < 4; ++j) word |= q8_code(v[j], scale) << (8 * j);
            *reinterpret_cast<uint32_t*>(row + c0) = word;
        }
        if (lane == 0) *reinterpret_cast<float*>(row + s.code_bytes + 4u * b) = scale;
        if (b + 1 == s.blocks) {   // zeros behind the scales
            const uint64_t at = s.code_bytes + 4ull * s.blocks + 4ull * lane;
            if (at < s.row_bytes) *reinterpret_cast<uint32_t*>(row + at) = 0u;
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(256) ckpt_load_kernel(uint64_t rows, CkptShape s,
                                                        const uint8_t* ckpt, T* out,
                                                        uint64_t ldo) {
    grid_wait();
    const int lane = threadIdx.x & 31;
    const uint64_t units = rows * s.blocks;
    for (uint64_t w = (uint64_t)blockIdx.x * 8 + (threadIdx.x >> 5); w < units;
         w += (uint64_t)gridDim.x * 8) {
        const uint64_t r = w / s.blocks;
        const uint32_t b = (uint32_t)(w - r * s.blocks);
        const uint32_t c0 = b * 128u + lane * 4u;
        const uint8_t* row = ckpt + r * s.row_bytes;
        if (c0 >= s.cols) continue;
        const float scale = ckpt_scales(row, s)[b];
        const uint32_t word = *reinterpret_cast<const uint32_t*>(row + c0);
        for (int j = 0; j < 4; ++j)
            if (c0 + j < s.cols)
                out[r * ldo + c0 + j] = from_f<T>(q8_value(word >> (8 * j) & 255u, scale));
    }
}

cudaError_t unit_grid(uint64_t units, unsigned* grid) {
    DevInfo di;
    const cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    const uint64_t blocks = (units + 7) / 8, cap = (uint64_t)di.sms * 8;
    *grid = (unsigned)(blocks < cap ? blocks : cap);
    return cudaSuccess;
}

}  // namespace

cudaError_t launch_ckpt_save(uint64_t rows, const CkptShape& s, int dtype, const Mat& x,
                             uint8_t* ckpt, cudaStream_t stream) {
    unsigned grid = 1;
    const cudaError_t e = unit_grid(rows * s.blocks, &grid);
    if (e != cudaSuccess) return e;
    if (dtype == ZERO_F16)
        return launch_act(ckpt_save_kernel<__half>, dim3(grid), 256, 0, stream, rows, s,
                          (const __half*)x.p, x.ld, ckpt);
    if (dtype == ZERO_BF16)
        return launch_act(ckpt_save_kernel<bf16>, dim3(grid), 256, 0, stream, rows, s,
                          (const bf16*)x.p, x.ld, ckpt);
    return launch_act(ckpt_save_kernel<float>, dim3(grid), 256, 0, stream, rows, s,
                      (const float*)x.p, x.ld, ckpt);
}

cudaError_t launch_ckpt_load(uint64_t rows, const CkptShape& s, int dtype, const uint8_t* ckpt,
                             const Mat& out, cudaStream_t stream) {
    unsigned grid = 1;
    const cudaError_t e = unit_grid(rows * s.blocks, &grid);
    if (e != cudaSuccess) return e;
    if (dtype == ZERO_F16)
        return launch_act(ckpt_load_kernel<__half>, dim3(grid), 256, 0, stream, rows, s, ckpt,
                          (__half*)out.p, out.ld);
    if (dtype == ZERO_BF16)
        return launch_act(ckpt_load_kernel<bf16>, dim3(grid), 256, 0, stream, rows, s, ckpt,
                          (bf16*)out.p, out.ld);
    return launch_act(ckpt_load_kernel<float>, dim3(grid), 256, 0, stream, rows, s, ckpt,
                      (float*)out.p, out.ld);
}

}  // namespace zk
