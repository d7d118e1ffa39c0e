// The block boundary for sm_100a: y = rs*x + bs*gate*post(h), u = pre(y), and its gradient.
//
// One CTA per row; the row is read again in each pass (statistics of h, of y, the outputs), from
// the L1 cache. The vector gradients are summed by a second kernel, one CTA per 32 columns, from
// row statistics that the first one leaves in the workspace.
#include "zero_act.cuh"

namespace zk {

constexpr int kRowStats = 6;   // mean, 1/deviation of h; of y; the two means of pre's gradient

uint64_t join_workspace(uint64_t rows, uint64_t cols, uint64_t) {
    return cols ? (rows * kRowStats * 4 + 15) / 16 * 16 : 0;
}

namespace {

constexpr int kThreads = 256;

template <typename T>
__device__ __forceinline__ float read_at(const Mat& m, const uint8_t* ck, const CkptShape& s,
                                         uint64_t r, uint32_t c) {
    if (ck) {
        const uint8_t* row = ck + r * s.row_bytes;
        return q8_value(row[c], ckpt_scales(row, s)[c / 128]);
    }
    return to_f(((const T*)m.p)[r * m.ld + c]);
}

template <typename T>
__device__ __forceinline__ float vec_at(const void* v, uint32_t c, float none) {
    return v ? to_f(((const T*)v)[c]) : none;
}

// Sum over the CTA, the same value in every thread, in a fixed order.
__device__ __forceinline__ float cta_sum(float v) {
    __shared__ float part[kThreads / 32];
    for (int d = 16; d > 0; d >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xffffffffu, v, d));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
    __syncthreads();
    float s = 0.0f;
    for (int i = 0; i < kThreads / 32; ++i) s = __fadd_rn(s, part[i]);
    return s;
}

// Mean and 1/deviation of a row given by f(c).
template <typename F>
__device__ __forceinline__ void row_stats(int kind, uint32_t cols, float eps, F f, float* mean,
                                          float* rstd) {
    *mean = 0.0f;
    *rstd = 1.0f;
    if (kind == ZERO_NORM_NONE) return;
    if (kind == ZERO_NORM_LAYER) {
        float s = 0.0f;
        for (uint32_t c = threadIdx.x; c < cols; c += kThreads) s = __fadd_rn(s, f(c));
        *mean = __fdiv_rn(cta_sum(s), (float)cols);
    }
    float q = 0.0f;
    for (uint32_t c = threadIdx.x; c < cols; c += kThreads) {
        const float d = __fsub_rn(f(c), *mean);
        q = __fmaf_rn(d, d, q);
    }
    *rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fadd_rn(__fdiv_rn(cta_sum(q), (float)cols), eps)));
}

template <typename T>
__device__ void save_row(uint8_t* ck, const CkptShape& s, uint64_t r, const T* v) {
    const int lane = threadIdx.x & 31;
    uint8_t* row = ck + r * s.row_bytes;
    for (uint32_t b = threadIdx.x >> 5; b < s.blocks; b += kThreads / 32) {
        float f[4];
        uint32_t amax = 0;
        const uint32_t c0 = b * 128u + lane * 4u;
        for (int j = 0; j < 4; ++j) {
            f[j] = c0 + j < s.cols ? to_f(v[c0 + j]) : 0.0f;
            amax = max(amax, abs_bits(f[j]));
        }
        amax = __reduce_max_sync(0xffffffffu, amax);
        const float scale = q8_scale(amax);
        if (c0 < s.code_bytes) {
            uint32_t word = 0;
            for (int j = 0; j < 4; ++j) word |= q8_code(f[j], scale) << (8 * j);
            *reinterpret_cast<uint32_t*>(row + c0) = word;
        }
        if (lane == 0) *reinterpret_cast<float*>(row + s.code_bytes + 4u * b) = scale;
    }
    const uint64_t at = s.code_bytes + 4ull * s.blocks + 4ull * threadIdx.x;
    if (at < s.row_bytes) *reinterpret_cast<uint32_t*>(row + at) = 0u;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) join_kernel(JoinArgs p) {
    extern __shared__ uint8_t smem[];
    T* ys = reinterpret_cast<T*>(smem);   // y as stored, for its checkpoint
    grid_wait();
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        auto h = [&](uint32_t c) { return read_at<T>(p.h, p.h_ckpt, p.ck, r, c); };
        float hm, hr, ym, yr;
        if (p.has_branch) row_stats(p.post, p.cols, p.post_eps, h, &hm, &hr);
        auto y = [&](uint32_t c) {
            float v = __fmul_rn(p.rs, read_at<T>(p.x, p.x_ckpt, p.ck, r, c));
            if (p.has_branch) {
                float z = h(c);
                if (p.post != ZERO_NORM_NONE)
                    z = __fmaf_rn(__fmul_rn(__fsub_rn(z, hm), hr), vec_at<T>(p.post_w, c, 1.0f),
                                  vec_at<T>(p.post_b, c, 0.0f));
                if (p.gate_rows)
                    z = __fmul_rn(z, to_f(((const T*)p.gate.p)[(r / p.gate_rows) * p.gate.ld + c]));
                v = __fmaf_rn(p.bs, z, v);
            }
            return v;
        };
        row_stats(p.u.p ? p.pre : ZERO_NORM_NONE, p.cols, p.pre_eps, y, &ym, &yr);
        __syncthreads();
        for (uint32_t c = threadIdx.x; c < p.cols; c += kThreads) {
            const float v = y(c);
            if (p.u.p)
                ((T*)p.u.p)[r * p.u.ld + c] =
                    from_f<T>(__fmaf_rn(__fmul_rn(__fsub_rn(v, ym), yr),
                                        vec_at<T>(p.pre_w, c, 1.0f), vec_at<T>(p.pre_b, c, 0.0f)));
            if (p.save_y) ys[c] = from_f<T>(v);
            if (p.y.p) ((T*)p.y.p)[r * p.y.ld + c] = from_f<T>(v);
        }
        if (p.save_h) save_row<T>(p.save_h, p.ck, r, (const T*)p.h.p + r * p.h.ld);
        if (p.save_y) {
            __syncthreads();
            save_row<T>(p.save_y, p.ck, r, ys);
            __syncthreads();
        }
    }
}

// The values of a boundary's gradient at one element, from its row's statistics.
struct Grad {
    float yh, hh, hn, gate, gy, t, gt, du;
};

template <typename T>
__device__ __forceinline__ Grad grad_at(const JoinArgs& p, uint64_t r, uint32_t c, float hm,
                                        float hr, float ym, float yr, float m1, float m2) {
    Grad g = {};
    if (p.du.p) {
        g.du = to_f(((const T*)p.du.p)[r * p.du.ld + c]);
        g.yh = __fmul_rn(__fsub_rn(read_at<T>(p.x, p.x_ckpt, p.ck, r, c), ym), yr);
        const float gu = __fmul_rn(g.du, vec_at<T>(p.pre_w, c, 1.0f));
        g.gy = __fmul_rn(yr, __fsub_rn(__fsub_rn(gu, m1), __fmul_rn(g.yh, m2)));
    }
    if (p.dy.p) g.gy = __fadd_rn(g.gy, to_f(((const T*)p.dy.p)[r * p.dy.ld + c]));
    if (p.has_branch) {
        g.gate = p.gate_rows ? to_f(((const T*)p.gate.p)[(r / p.gate_rows) * p.gate.ld + c]) : 1.0f;
        g.t = __fmul_rn(__fmul_rn(p.bs, g.gate), g.gy);
        g.gt = g.t;
        if (p.h.p || p.h_ckpt) {
            g.hn = read_at<T>(p.h, p.h_ckpt, p.ck, r, c);
            if (p.post != ZERO_NORM_NONE) {
                const float w = vec_at<T>(p.post_w, c, 1.0f);
                g.hh = __fmul_rn(__fsub_rn(g.hn, hm), hr);
                g.hn = __fmaf_rn(g.hh, w, vec_at<T>(p.post_b, c, 0.0f));
                g.gt = __fmul_rn(g.t, w);
            }
        }
    }
    return g;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) join_back_kernel(JoinArgs p, float* stats) {
    grid_wait();
    for (uint64_t r = blockIdx.x; r < p.rows; r += gridDim.x) {
        float hm = 0, hr = 1, ym = 0, yr = 1, m1 = 0, m2 = 0, n1 = 0, n2 = 0;
        if (p.du.p) {
            auto y = [&](uint32_t c) { return read_at<T>(p.x, p.x_ckpt, p.ck, r, c); };
            row_stats(p.pre, p.cols, p.pre_eps, y, &ym, &yr);
            float s1 = 0, s2 = 0;
            for (uint32_t c = threadIdx.x; c < p.cols; c += kThreads) {
                const float gu = __fmul_rn(to_f(((const T*)p.du.p)[r * p.du.ld + c]),
                                           vec_at<T>(p.pre_w, c, 1.0f));
                s1 = __fadd_rn(s1, gu);
                s2 = __fmaf_rn(gu, __fmul_rn(__fsub_rn(y(c), ym), yr), s2);
            }
            m2 = __fdiv_rn(cta_sum(s2), (float)p.cols);
            if (p.pre == ZERO_NORM_LAYER) m1 = __fdiv_rn(cta_sum(s1), (float)p.cols);
        }
        if (p.has_branch && p.post != ZERO_NORM_NONE) {
            auto h = [&](uint32_t c) { return read_at<T>(p.h, p.h_ckpt, p.ck, r, c); };
            row_stats(p.post, p.cols, p.post_eps, h, &hm, &hr);
            float s1 = 0, s2 = 0;
            for (uint32_t c = threadIdx.x; c < p.cols; c += kThreads) {
                const Grad g = grad_at<T>(p, r, c, hm, hr, ym, yr, m1, m2);
                s1 = __fadd_rn(s1, g.gt);
                s2 = __fmaf_rn(g.gt, g.hh, s2);
            }
            n2 = __fdiv_rn(cta_sum(s2), (float)p.cols);
            if (p.post == ZERO_NORM_LAYER) n1 = __fdiv_rn(cta_sum(s1), (float)p.cols);
        }
        if (stats && threadIdx.x == 0) {
            float* s = stats + r * kRowStats;
            s[0] = hm; s[1] = hr; s[2] = ym; s[3] = yr; s[4] = m1; s[5] = m2;
        }
        if (!p.dx.p && !p.dh.p) continue;
        for (uint32_t c = threadIdx.x; c < p.cols; c += kThreads) {
            const Grad g = grad_at<T>(p, r, c, hm, hr, ym, yr, m1, m2);
            // dx may stand in dy's place: with vector gradients it is written by the second kernel
            if (p.dx.p && (!stats || p.dx.p != p.dy.p))
                ((T*)p.dx.p)[r * p.dx.ld + c] = from_f<T>(__fmul_rn(p.rs, g.gy));
            if (p.dh.p)
                ((T*)p.dh.p)[r * p.dh.ld + c] = from_f<T>(
                    p.post == ZERO_NORM_NONE
                        ? g.t
                        : __fmul_rn(hr, __fsub_rn(__fsub_rn(g.gt, n1), __fmul_rn(g.hh, n2))));
        }
    }
}

template <typename T>
__device__ __forceinline__ void put_sum(void* p, uint64_t at, float s, bool add) {
    if (!p) return;
    T* d = (T*)p + at;
    *d = from_f<T>(add ? __fadd_rn(to_f(*d), s) : s);
}

// 32 columns, 8 rows at a time; the 8 partial sums are added in order.
template <typename T>
__global__ void __launch_bounds__(kThreads) join_vectors_kernel(JoinArgs p, const float* stats) {
    __shared__ float part[5][8][32];
    grid_wait();
    const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
    const uint32_t c = blockIdx.x * 32u + cx;
    float s[5] = {};
    auto flush = [&](int k, void* out, uint64_t at, bool add) {
        part[k][ry][cx] = s[k];
        __syncthreads();
        if (ry == 0 && c < p.cols) {
            float v = 0.0f;
            for (int i = 0; i < 8; ++i) v = __fadd_rn(v, part[k][i][cx]);
            put_sum<T>(out, at, v, add);
        }
        __syncthreads();
        s[k] = 0.0f;
    };
    const uint64_t span = p.dgate.p ? p.gate_rows : p.rows;
    for (uint64_t g0 = 0; g0 < p.rows; g0 += span) {
        const uint64_t g1 = span < p.rows - g0 ? g0 + span : p.rows;
        for (uint64_t r = g0 + ry; r < g1 && c < p.cols; r += 8) {
            const float* st = stats + r * kRowStats;
            const Grad g = grad_at<T>(p, r, c, st[0], st[1], st[2], st[3], st[4], st[5]);
            s[0] = __fmaf_rn(__fmul_rn(p.bs, g.gy), g.hn, s[0]);
            s[1] = __fmaf_rn(g.t, g.hh, s[1]);
            s[2] = __fadd_rn(s[2], g.t);
            s[3] = __fmaf_rn(g.du, g.yh, s[3]);
            s[4] = __fadd_rn(s[4], g.du);
            if (p.dx.p && p.dx.p == p.dy.p)
                ((T*)p.dx.p)[r * p.dx.ld + c] = from_f<T>(__fmul_rn(p.rs, g.gy));
        }
        if (p.dgate.p) flush(0, p.dgate.p, g0 / span * p.dgate.ld + c, p.accumulate & ZERO_ACC_GATE);
    }
    const bool add = p.accumulate & ZERO_ACC_PARAMS;
    flush(1, p.dpost_w, c, add);
    flush(2, p.dpost_b, c, add);
    flush(3, p.dpre_w, c, add);
    flush(4, p.dpre_b, c, add);
}

template <typename T>
cudaError_t run_join(const JoinArgs& a, cudaStream_t stream) {
    const unsigned grid = (unsigned)(a.rows < (1u << 20) ? a.rows : (1u << 20));
    return launch_act(join_kernel<T>, dim3(grid), kThreads, a.save_y ? a.cols * sizeof(T) : 0,
                      stream, a);
}

template <typename T>
cudaError_t run_join_back(const JoinArgs& a, void* ws, cudaStream_t stream) {
    const bool vec = a.dgate.p || a.dpost_w || a.dpost_b || a.dpre_w || a.dpre_b;
    if (a.rows) {
        const unsigned grid = (unsigned)(a.rows < (1u << 20) ? a.rows : (1u << 20));
        const cudaError_t e = launch_act(join_back_kernel<T>, dim3(grid), kThreads, 0, stream, a,
                                         vec ? (float*)ws : (float*)nullptr);
        if (e != cudaSuccess) return e;
    }
    if (!vec) return cudaSuccess;
    return launch_act(join_vectors_kernel<T>, dim3((a.cols + 31) / 32), kThreads, 0, stream, a,
                      (const float*)ws);
}

}  // namespace

cudaError_t launch_join(const JoinArgs& a, int dtype, cudaStream_t stream) {
    if (dtype == ZERO_F32 && a.save_y) {
        const cudaError_t e = cudaFuncSetAttribute(
            join_kernel<float>, cudaFuncAttributeMaxDynamicSharedMemorySize,
            ZERO_JOIN_MAX_COLS * (int)sizeof(float));
        if (e != cudaSuccess) return e;
    }
    return dtype == ZERO_F16    ? run_join<__half>(a, stream)
           : dtype == ZERO_BF16 ? run_join<bf16>(a, stream)
                                : run_join<float>(a, stream);
}

cudaError_t launch_join_backward(const JoinArgs& a, int dtype, void* ws, cudaStream_t stream) {
    return dtype == ZERO_F16    ? run_join_back<__half>(a, ws, stream)
           : dtype == ZERO_BF16 ? run_join_back<bf16>(a, ws, stream)
                                : run_join_back<float>(a, ws, stream);
}

}  // namespace zk
