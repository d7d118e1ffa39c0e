// Activation-side calls: geometry of the 8-bit checkpoint and the launchers' arguments, shared
// by the argument checks (zero_act_api.cpp) and the kernels (zero_ckpt.cu, zero_join_*.cu,
// zero_join_back_*.cu, zero_wgrad.cu). Internal.
#pragma once

#include <cstdint>

#include <cuda_runtime.h>

#include "zero_internal.h"

namespace zk {

// A row-major matrix: element (r, c) at p + r*ld + c.
struct Mat {
    void* p;
    uint64_t ld;
};

// The 8-bit checkpoint of a matrix of `cols` columns (see ZERO_CKPT_ROW_BYTES).
struct CkptShape {
    uint32_t cols;
    uint32_t code_bytes;   // cols rounded up to 16
    uint32_t blocks;       // ceil(cols/128)
    uint64_t row_bytes;
};

inline CkptShape ckpt_shape(uint64_t cols) {
    CkptShape s;
    s.cols = (uint32_t)cols;
    s.code_bytes = (uint32_t)ZERO_CKPT_CODE_BYTES(cols);
    s.blocks = (uint32_t)((cols + 127) / 128);
    s.row_bytes = ZERO_CKPT_ROW_BYTES(cols);
    return s;
}

// Rows `pitch` bytes apart: a matrix, or a checkpoint's records. The boundary's calls keep row
// numbers and pitches below 2^31, so that an address is one multiply-add.
struct Rows {
    void* p;
    uint32_t pitch;
};

// A boundary's operands (null where absent).
struct JoinArgs {
    uint32_t rows, cols;
    int post, pre;                 // zero_norm
    float post_eps, pre_eps, rs, bs;
    uint32_t gate_rows;
    Rows gate, x, h;
    bool x_codes, h_codes;         // x, h are checkpoints
    const void *post_w, *post_b, *pre_w, *pre_b;
    // forward
    Rows y, u, save_y, save_h;
    // backward (x holds the saved y there)
    Rows dy, du, dx, dh, dgate;
    void *dpost_w, *dpost_b, *dpre_w, *dpre_b;
    int has_branch, accumulate;
    CkptShape ck;
};

uint64_t join_workspace(uint64_t rows, uint64_t cols, uint64_t gate_rows);
uint64_t wgrad_workspace(uint64_t t, uint64_t o, uint64_t i);

cudaError_t launch_ckpt_save(uint64_t rows, const CkptShape& s, int dtype, const Mat& x,
                             uint8_t* ckpt, cudaStream_t stream);
cudaError_t launch_ckpt_load(uint64_t rows, const CkptShape& s, int dtype, const uint8_t* ckpt,
                             const Mat& out, cudaStream_t stream);
cudaError_t launch_join(const JoinArgs& a, int dtype, cudaStream_t stream);
cudaError_t launch_join_backward(const JoinArgs& a, int dtype, void* ws, cudaStream_t stream);
// One source per type (zero_join_*.cu).
cudaError_t join_f16(const JoinArgs& a, cudaStream_t stream);
cudaError_t join_bf16(const JoinArgs& a, cudaStream_t stream);
cudaError_t join_f32(const JoinArgs& a, cudaStream_t stream);
cudaError_t join_back_f16(const JoinArgs& a, float* ws, cudaStream_t stream);
cudaError_t join_back_bf16(const JoinArgs& a, float* ws, cudaStream_t stream);
cudaError_t join_back_f32(const JoinArgs& a, float* ws, cudaStream_t stream);

struct WgradArgs {
    uint64_t tokens;
    uint32_t outf, inf;
    Mat dy, dw;
    const uint8_t* ckpt;
    CkptShape ck;
    int accumulate;
    uint32_t* status;
};
cudaError_t launch_wgrad(const WgradArgs& a, int dtype, void* ws, cudaStream_t stream);

}  // namespace zk
