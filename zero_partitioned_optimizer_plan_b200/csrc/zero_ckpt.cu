// 8-bit activation checkpoints for sm_100a: a matrix of activations to records of one byte per
// value and one fp32 scale per 128 columns, and back ("ZeRO" ZeRO-R: what partitioning the model
// states leaves is the activation checkpoints; the pages give no format, this is the library's).
//
// Per block of 128 columns of a row: scale = amax/127, q = round_half_even(x/scale), stored as
// q + 128; an inf or NaN poisons the block (scale NaN, q 0). The read is T(q*scale).
//
// Bound by HBM: each direction moves the values once and about half as many bytes of records
// (fp16). A warp takes kN * 256 neighbouring columns of a row at a time and loads them all
// before it works on the first: one address and one step per piece, and the two divisions that
// the scales need once per piece (pieces of one chunk each, stepped separately, issued twice the
// instructions, and the kernel was bound by them).
#include "zero_act.cuh"

namespace zk {
namespace {

constexpr int kThreads = 128;

// The pieces of a matrix, row by row, and the step to the same warp's next piece.
struct Pieces {
    uint64_t rows;
    uint32_t per_row;
    uint32_t step_rows, step_pieces;   // warps of the grid = step_rows * per_row + step_pieces
};

struct Piece {
    uint64_t row;
    uint32_t at;
    __device__ __forceinline__ void next(const Pieces& p) {
        row += p.step_rows;
        at += p.step_pieces;
        if (at >= p.per_row) {
            at -= p.per_row;
            ++row;
        }
    }
};

__device__ __forceinline__ Piece first_piece(const Pieces& p) {
    const uint64_t w = (uint64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    Piece a;
    a.row = w / p.per_row;
    a.at = (uint32_t)(w - a.row * p.per_row);
    return a;
}

template <typename T, int kA, int kN>
__global__ void __launch_bounds__(kThreads, kA != kNarrow && sizeof(T) == 2 ? 7 : 6)
    ckpt_save_kernel(Pieces p, CkptShape s, Mat x, uint8_t* ckpt) {
    grid_wait();
    const uint32_t lane = threadIdx.x & 31;
    for (Piece i = first_piece(p); i.row < p.rows; i.next(p)) {
        const T* src = (const T*)x.p + i.row * x.ld;
        uint8_t* row = ckpt + i.row * s.row_bytes;
        Raw<T> raw[kN];
#pragma unroll
        for (int k = 0; k < kN; ++k)
            raw[k] = load_raw<T, kA>(src, Cols<kA>(i.at * kN + k, lane, s.cols));
        save_chunks<T, kA, kN>(row, s, i.at * kN, 1, lane, raw);
        if (i.at == 0) save_pad(row, s, lane);
    }
}

template <typename T, int kA, int kN>
__global__ void __launch_bounds__(kThreads) ckpt_load_kernel(Pieces p, CkptShape s,
                                                             const uint8_t* ckpt, Mat y) {
    grid_wait();
    const uint32_t lane = threadIdx.x & 31;
    for (Piece i = first_piece(p); i.row < p.rows; i.next(p)) {
        const uint8_t* row = ckpt + i.row * s.row_bytes;
        T* dst = (T*)y.p + i.row * y.ld;
        Raw<T> raw[kN];
#pragma unroll
        for (int k = 0; k < kN; ++k)
            raw[k] = load_codes<T, kA>(row, s, Cols<kA>(i.at * kN + k, lane, s.cols));
#pragma unroll
        for (int k = 0; k < kN; ++k) {
            F8 v;
            widen_codes<T>(raw[k], v);
            store_raw<T, kA>(dst, Cols<kA>(i.at * kN + k, lane, s.cols), narrow<T>(v));
        }
    }
}

// As many warps as pieces, at most kWaves CTAs per SM.
constexpr int kWaves = 32;

// Chunks per piece: four, unless a row is shorter or would leave most of a piece unused.
int chunks_per_piece(uint32_t cols) {
    const uint32_t chunks = (cols + kWarpCols - 1) / kWarpCols;
    return chunks >= 3 ? 4 : (int)chunks;
}

cudaError_t split(uint64_t rows, const CkptShape& s, int n, Pieces* p, unsigned* grid) {
    DevInfo di;
    const cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    p->rows = rows;
    p->per_row = (s.cols + n * kWarpCols - 1) / (n * kWarpCols);
    const uint64_t warps = kThreads / 32;
    const uint64_t blocks = (rows * p->per_row + warps - 1) / warps;
    const uint64_t cap = (uint64_t)di.sms * kWaves;
    *grid = (unsigned)(blocks < cap ? blocks : cap);
    const uint64_t step = *grid * warps;
    p->step_rows = (uint32_t)(step / p->per_row);
    p->step_pieces = (uint32_t)(step % p->per_row);
    return cudaSuccess;
}

template <typename T, int kN>
cudaError_t run(bool save, uint64_t rows, const CkptShape& s, const Mat& m, uint8_t* ckpt,
                cudaStream_t stream) {
    Pieces p;
    unsigned grid = 1;
    const cudaError_t e = split(rows, s, kN, &p, &grid);
    if (e != cudaSuccess) return e;
    const Access ac = access_of<T>(m.p, m.ld, s.cols);
    if (save)
        return launch_act(ac == kWide   ? ckpt_save_kernel<T, kWide, kN>
                          : ac == kTail ? ckpt_save_kernel<T, kTail, kN>
                                        : ckpt_save_kernel<T, kNarrow, kN>,
                          dim3(grid), kThreads, 0, stream, p, s, m, ckpt);
    return launch_act(ac == kWide   ? ckpt_load_kernel<T, kWide, kN>
                      : ac == kTail ? ckpt_load_kernel<T, kTail, kN>
                                    : ckpt_load_kernel<T, kNarrow, kN>,
                      dim3(grid), kThreads, 0, stream, p, s, (const uint8_t*)ckpt, m);
}

template <typename T>
cudaError_t run_t(bool save, uint64_t rows, const CkptShape& s, const Mat& m, uint8_t* ckpt,
                  cudaStream_t stream) {
    switch (chunks_per_piece(s.cols)) {
        case 1: return run<T, 1>(save, rows, s, m, ckpt, stream);
        case 2: return run<T, 2>(save, rows, s, m, ckpt, stream);
        default: return run<T, 4>(save, rows, s, m, ckpt, stream);
    }
}

cudaError_t run_any(bool save, uint64_t rows, const CkptShape& s, int dtype, const Mat& m,
                    uint8_t* ckpt, cudaStream_t stream) {
    return dtype == ZERO_F16    ? run_t<__half>(save, rows, s, m, ckpt, stream)
           : dtype == ZERO_BF16 ? run_t<bf16>(save, rows, s, m, ckpt, stream)
                                : run_t<float>(save, rows, s, m, ckpt, stream);
}

}  // namespace

cudaError_t launch_ckpt_save(uint64_t rows, const CkptShape& s, int dtype, const Mat& x,
                             uint8_t* ckpt, cudaStream_t stream) {
    return run_any(true, rows, s, dtype, x, ckpt, stream);
}

cudaError_t launch_ckpt_load(uint64_t rows, const CkptShape& s, int dtype, const uint8_t* ckpt,
                             const Mat& out, cudaStream_t stream) {
    return run_any(false, rows, s, dtype, out, const_cast<uint8_t*>(ckpt), stream);
}

}  // namespace zk
