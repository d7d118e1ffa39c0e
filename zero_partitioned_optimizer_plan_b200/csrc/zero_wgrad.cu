// Weight gradient of a linear layer from the 8-bit checkpoint of its input, for sm_100a:
//   dw[o][i] = sum over t of dy[t][o] * a[t][i],   a = the checkpoint's values in dy's type.
//
// 64 x 64 outputs per CTA, 16 x 16 threads of 4 x 4 outputs, 16 tokens at a time in shared
// memory, binary32 sums.
#include "zero_act.cuh"

namespace zk {

uint64_t wgrad_workspace(uint64_t, uint64_t, uint64_t) { return 0; }

namespace {

template <typename T>
__global__ void __launch_bounds__(256) wgrad_kernel(WgradArgs p) {
    __shared__ float sa[16][64], sb[16][64];
    grid_wait();
    const uint32_t o0 = blockIdx.y * 64u, i0 = blockIdx.x * 64u;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    float acc[4][4] = {};
    const T* dy = (const T*)p.dy.p;
    for (uint64_t t0 = 0; t0 < p.tokens; t0 += 16) {
        for (int e = threadIdx.x; e < 16 * 64; e += 256) {
            const uint64_t t = t0 + e / 64;
            const uint32_t o = o0 + e % 64, i = i0 + e % 64;
            sa[e / 64][e % 64] = t < p.tokens && o < p.outf ? to_f(dy[t * p.dy.ld + o]) : 0.0f;
            float v = 0.0f;
            if (t < p.tokens && i < p.inf) {
                const uint8_t* row = p.ckpt + t * p.ck.row_bytes;
                v = round_to<T>(q8_value(row[i], ckpt_scales(row, p.ck)[i / 128]));
            }
            sb[e / 64][e % 64] = v;
        }
        __syncthreads();
        for (int k = 0; k < 16; ++k)
            for (int a = 0; a < 4; ++a)
                for (int b = 0; b < 4; ++b)
                    acc[a][b] = __fmaf_rn(sa[k][ty * 4 + a], sb[k][tx * 4 + b], acc[a][b]);
        __syncthreads();
    }
    T* dw = (T*)p.dw.p;
    for (int a = 0; a < 4; ++a)
        for (int b = 0; b < 4; ++b) {
            const uint32_t o = o0 + ty * 4 + a, i = i0 + tx * 4 + b;
            if (o < p.outf && i < p.inf) {
                T* d = dw + o * p.dw.ld + i;
                *d = from_f<T>(p.accumulate ? __fadd_rn(to_f(*d), acc[a][b]) : acc[a][b]);
            }
        }
}

}  // namespace

cudaError_t launch_wgrad(const WgradArgs& a, int dtype, void*, cudaStream_t stream) {
    const dim3 grid((a.inf + 63) / 64, (a.outf + 63) / 64);
    return dtype == ZERO_F16 ? launch_act(wgrad_kernel<__half>, grid, 256, 0, stream, a)
                             : launch_act(wgrad_kernel<bf16>, grid, 256, 0, stream, a);
}

}  // namespace zk
