// Device helpers of the activation-side kernels: element types, the 8-bit block rule, and the
// launch with programmatic stream serialization. Internal; everything in an anonymous namespace.
//
// Order on the stream. Every kernel here waits for the kernel before it to complete before its
// first access to memory (griddepcontrol.wait), and none lets the next kernel on the stream
// start early, except a call's own second kernel: so a call is ordered like an ordinary launch,
// also between the calls of a zero_overlap_begin/end region. (There the kernel before it may be one
// that ran alongside others; such a kernel completes only after all of them.)
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

#include "zero_act.h"
#include "zero_device.cuh"

namespace zk {
namespace {

using bf16 = __nv_bfloat16;

__device__ __forceinline__ float to_f(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f(bf16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f(float x) { return x; }

template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ __half from_f<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ bf16 from_f<bf16>(float x) { return __float2bfloat16_rn(x); }
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }

// v as it reads back from memory in type T.
template <typename T>
__device__ __forceinline__ float round_to(float v) { return to_f(from_f<T>(v)); }

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

// The scale of a block from the largest |x| as binary32 bits (they order like the values; an inf
// or NaN is at or above 0x7f800000 and makes the scale NaN).
__device__ __forceinline__ float q8_scale(uint32_t amax) {
    return amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u)
                               : __fdiv_rn(__uint_as_float(amax), 127.0f);
}

// The code bytes of the values x[0..7], as two words, from inv = fl(1/scale). For a scale of at
// least 2^-100 the quotients stay below 127.5, and 1/scale lies strictly between inv*(1 - 2^-21)
// and inv*(1 + 2^-21), wide enough that fl(x/scale) lies between the two products too: where
// both products round to the same integer, fl(x/scale) rounds to it. (Rounding: the fused
// multiply-add into 1.5 * 2^23 + 128 leaves the integer + 128 in the low byte.) The others,
// and smaller, zero or NaN scales, take q8_codes_near.
constexpr float kQ8Bias = 12583040.0f;

// Eight integers + 128, as they lie in the low bytes of kQ8Bias + integer, packed.
__device__ __forceinline__ uint2 q8_bytes(const float (&c)[8]) {
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const uint32_t p = __byte_perm(__float_as_uint(c[4 * k]), __float_as_uint(c[4 * k + 1]), 0x0040u);
        const uint32_t q = __byte_perm(__float_as_uint(c[4 * k + 2]), __float_as_uint(c[4 * k + 3]), 0x0040u);
        w[k] = __byte_perm(p, q, 0x5410u);
    }
    return make_uint2(w[0], w[1]);
}

// The first four values have scale s0, the others s1 (one and the same, or two). Returns false
// if some value needs q8_codes_near.
__device__ __forceinline__ bool q8_codes(const float (&x)[8], float s0, float s1, float inv0,
                                         float inv1, uint2& out) {
    float c[8];
    uint32_t differ = 0;
    const uint64_t bias = f2_pack(kQ8Bias, kQ8Bias);
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        const float inv = j < 4 ? inv0 : inv1;
        const float lo = __fmul_rn(inv, 1.0f - 0x1p-21f), hi = __fmul_rn(inv, 1.0f + 0x1p-21f);
        const uint64_t v = f2_pack(x[j], x[j + 1]), l2 = f2_pack(lo, lo), h2 = f2_pack(hi, hi);
        float a, b;
        f2_unpack(f2_fma(v, l2, bias), a, b);
        f2_unpack(f2_fma(v, h2, bias), c[j], c[j + 1]);
        differ |= __float_as_uint(a) ^ __float_as_uint(c[j]);
        differ |= __float_as_uint(b) ^ __float_as_uint(c[j + 1]);
    }
    out = q8_bytes(c);
    return differ == 0 && s0 >= 0x1p-100f && s1 >= 0x1p-100f;
}

// The integer nearest fl(x/scale), ties to even, as kQ8Bias + integer, where x/scale lies close
// to m, halfway between the integers that the two products a and b rounded to. e = x - m*scale
// is exact (18 bits), and fl(x/scale) is above, at or below m as e is above, within or below
// half a unit in the last place of m times the scale. (At m = 1/2 the places below are narrower,
// but there both answers round to 0.) No division: 16-bit values meet ties often, x = amax/2
// among them.
__device__ __forceinline__ float q8_near(float x, float scale, float a, float b) {
    const float k0 = fminf(a, b), k1 = fmaxf(a, b);
    const float m = __fadd_rn(__fsub_rn(k0, kQ8Bias), 0.5f);
    const float e = __fmaf_rn(-m, scale, x);
    const float half = __fmul_rn(__uint_as_float(__float_as_uint(m) & 0x7f800000u),
                                 __fmul_rn(scale, 0x1p-24f));
    const float even = (__float_as_uint(k0) & 1u) ? k1 : k0;
    return a == b ? a : e > half ? k1 : e < -half ? k0 : even;
}

// The codes where q8_codes returned false. A small scale is first multiplied by 2^80, and the
// values with it (exact, and the quotients stay); it may have been rounded by up to half of
// itself, so the codes are clamped. A scale of 0 or NaN gives q = 0.
__device__ __forceinline__ uint2 q8_codes_near(const float (&x)[8], float s0, float s1, float inv0,
                                               float inv1) {
    const float s[2] = {s0, s1};
    const float inv[2] = {inv0, inv1};
    float c[8];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const bool normal = s[h] >= 0x1p-100f, any = s[h] > 0.0f;
        const float up = normal ? 1.0f : any ? 0x1p80f : 0.0f;
        const float scale = normal ? s[h] : any ? __fmul_rn(s[h], 0x1p80f) : 1.0f;
        const float r = normal ? inv[h] : __fdiv_rn(1.0f, scale);
        const float lo = __fmul_rn(r, 1.0f - 0x1p-21f), hi = __fmul_rn(r, 1.0f + 0x1p-21f);
#pragma unroll
        for (int j = 4 * h; j < 4 * h + 4; ++j) {
            const float v = any ? __fmul_rn(x[j], up) : 0.0f;
            c[j] = q8_near(v, scale, __fmaf_rn(v, lo, kQ8Bias), __fmaf_rn(v, hi, kQ8Bias));
            c[j] = fminf(fmaxf(c[j], kQ8Bias - 127.0f), kQ8Bias + 127.0f);
        }
    }
    return q8_bytes(c);
}

__device__ __forceinline__ float q8_value(uint32_t byte, float scale) {
    return __fmul_rn((float)((int)byte - 128), scale);
}

__device__ __forceinline__ const float* ckpt_scales(const uint8_t* row, const CkptShape& s) {
    return reinterpret_cast<const float*>(row + s.code_bytes);
}

// ---------------------------------------------------------------------------------------------
// Eight columns per lane. A warp covers 256 columns (two blocks of codes) of a row. With 16-byte
// aligned rows a lane's columns are neighbours and move as 16-byte accesses (kWide: a row ends on
// a lane's last column; kTail: it may end inside a lane's columns). Otherwise (kNarrow) lane l
// takes the pairs of columns 2l + 64p, p = 0 .. 3, so that a warp's 4-byte accesses are neighbours;
// 16-bit rows that start inside a 4-byte word are read and written by the words they overlap, the
// halves exchanged between the lanes.
// ---------------------------------------------------------------------------------------------
constexpr uint32_t kWarpCols = 256;

enum Access { kNarrow = 0, kTail = 1, kWide = 2 };

template <int kA>
struct Cols {
    uint32_t c0, cols;
    uint32_t mask;   // bit j: column j exists
    __device__ __forceinline__ Cols() : c0(0), cols(0), mask(0) {}
    __device__ __forceinline__ Cols(uint32_t chunk, uint32_t lane, uint32_t n) : cols(n), mask(0) {
        c0 = chunk * kWarpCols + (kA == kNarrow ? 2u : 8u) * lane;
        const uint32_t left = n > c0 ? n - c0 : 0u;
        if (kA == kNarrow) {
#pragma unroll
            for (int j = 0; j < 8; ++j) mask |= (left > at(j) - c0 ? 1u : 0u) << j;
        } else {
            mask = left >= 8u ? 0xffu : (1u << left) - 1u;
        }
    }
    __device__ __forceinline__ uint32_t at(int j) const {
        return c0 + (kA == kNarrow ? 64 * (j >> 1) + (j & 1) : j);
    }
    __device__ __forceinline__ bool any() const { return mask != 0; }
    // every column of the lane exists (kWide: or none does)
    __device__ __forceinline__ bool whole() const { return kA == kWide ? any() : mask == 0xffu; }
};

// Eight values as they lie in memory: T, or codes (two words) and the scales of the lane's first
// and second four columns.
template <typename T>
struct Raw {
    uint32_t w[2 * sizeof(T)];
};

template <typename T, int kA>
__device__ __forceinline__ Raw<T> load_raw(const T* row, const Cols<kA>& c) {
    Raw<T> r;
#pragma unroll
    for (int k = 0; k < 2 * (int)sizeof(T); ++k) r.w[k] = 0;
    if (kA != kNarrow && c.whole()) {
        const uint4* p = reinterpret_cast<const uint4*>(row + c.c0);
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k) {
            const uint4 q = p[k];
            r.w[4 * k] = q.x;
            r.w[4 * k + 1] = q.y;
            r.w[4 * k + 2] = q.z;
            r.w[4 * k + 3] = q.w;
        }
        return r;
    }
    if (kA == kWide || !c.any()) return r;
    if constexpr (kA == kNarrow && sizeof(T) == 2) {
        if ((reinterpret_cast<uintptr_t>(row) & 3u) == 0) {
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint16_t* q = reinterpret_cast<const uint16_t*>(row) + c.at(2 * p);
                if (c.mask >> (2 * p + 1) & 1u)
                    r.w[p] = *reinterpret_cast<const uint32_t*>(q);
                else if (c.mask >> (2 * p) & 1u)
                    r.w[p] = *q;
            }
            return r;
        }
    }
    // every load is issued (a missing column reads the lane's first one), then sorted out: the
    // loads do not wait for one another
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t i = c.mask >> j & 1u ? c.at(j) : c.c0;
        if constexpr (sizeof(T) == 4)
            v[j] = reinterpret_cast<const uint32_t*>(row)[i];
        else
            v[j] = reinterpret_cast<const uint16_t*>(row)[i];
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const uint32_t x = c.mask >> j & 1u ? v[j] : 0u;
        if constexpr (sizeof(T) == 4)
            r.w[j] = x;
        else
            r.w[j / 2] |= x << 16 * (j & 1);
    }
    return r;
}

template <typename T, int kA>
__device__ __forceinline__ Raw<T> load_codes(const uint8_t* row, const CkptShape& s,
                                             const Cols<kA>& c) {
    Raw<T> r;
    r.w[0] = r.w[1] = 0x80808080u;
    r.w[2] = r.w[3] = 0u;
    if (!c.any()) return r;
    const float* sc = ckpt_scales(row, s);
    if constexpr (kA != kNarrow) {
        const uint2 q = *reinterpret_cast<const uint2*>(row + c.c0);
        r.w[0] = q.x;
        r.w[1] = q.y;
        r.w[2] = r.w[3] = __float_as_uint(sc[c.c0 >> 7]);
    } else {
        // (the second of a pair may be a byte of the padding: q = 0)
        uint32_t v[4];
#pragma unroll
        for (int p = 0; p < 4; ++p)
            v[p] = c.mask >> (2 * p) & 1u
                       ? *reinterpret_cast<const uint16_t*>(row + c.at(2 * p))
                       : 0x8080u;
        r.w[0] = v[0] | v[1] << 16;
        r.w[1] = v[2] | v[3] << 16;
        r.w[2] = __float_as_uint(sc[c.c0 >> 7]);
        r.w[3] = __float_as_uint(sc[(c.c0 >> 7) + (c.mask >> 4 & 1u)]);
    }
    return r;
}

// Pairs of binary32 values (columns 2k and 2k + 1).
using F8 = uint64_t[4];

template <typename T>
__device__ __forceinline__ void widen(const Raw<T>& r, F8& v) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        if constexpr (sizeof(T) == 4) {
            v[k] = f2_pack(__uint_as_float(r.w[2 * k]), __uint_as_float(r.w[2 * k + 1]));
        } else if constexpr (std::is_same<T, bf16>::value) {
            v[k] = f2_pack(__uint_as_float(r.w[k] << 16), __uint_as_float(r.w[k] & 0xffff0000u));
        } else {
            const float2 f = h2x2_to_f2(r.w[k]);
            v[k] = f2_pack(f.x, f.y);
        }
    }
}

// q*scale of the codes: the byte in the mantissa of 2^23, the bias 2^23 + 128 off, both exact.
template <typename T>
__device__ __forceinline__ void widen_codes(const Raw<T>& r, F8& v) {
    const uint64_t bias = f2_pack(8388736.0f, 8388736.0f);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const uint32_t w = r.w[k / 2], j = 2 * (k & 1);
        const float s = __uint_as_float(r.w[2 + k / 2]);
        const uint64_t q = f2_pack(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540u + j)),
                                   __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7541u + j)));
        v[k] = f2_mul(f2_sub(q, bias), f2_pack(s, s));
    }
}

// Row r of a matrix whose rows lie `pitch` bytes apart (both below 2^32: one multiply-add).
template <typename T>
__device__ __forceinline__ T* row_of(const Rows& m, uint32_t r) {
    return reinterpret_cast<T*>(reinterpret_cast<char*>(m.p) + (uint64_t)r * m.pitch);
}

// The values of a row of a matrix or of a checkpoint.
template <typename T, int kA>
__device__ __forceinline__ Raw<T> load_row(const Rows& m, bool codes, const CkptShape& s,
                                           uint32_t r, const Cols<kA>& c) {
    if (codes) return load_codes<T, kA>(row_of<uint8_t>(m, r), s, c);
    return load_raw<T, kA>(row_of<T>(m, r), c);
}

template <typename T>
__device__ __forceinline__ void widen_row(const Raw<T>& raw, bool codes, F8& v) {
    if (codes)
        widen_codes<T>(raw, v);
    else
        widen<T>(raw, v);
}

// A vector of cols values, or `none` everywhere.
template <typename T, int kA>
__device__ __forceinline__ void load_vec(const void* p, float none, const Cols<kA>& c, F8& v) {
    if (p) {
        widen<T>(load_raw<T, kA>((const T*)p, c), v);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) v[k] = f2_pack(none, none);
    }
}

// Zero the columns that do not exist.
template <int kA>
__device__ __forceinline__ void clear_missing(const Cols<kA>& c, F8& v) {
    if (c.whole()) return;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a, b;
        f2_unpack(v[k], a, b);
        v[k] = f2_pack(c.mask >> (2 * k) & 1u ? a : 0.0f, c.mask >> (2 * k + 1) & 1u ? b : 0.0f);
    }
}

__device__ __forceinline__ float sum8(const F8& v) {
    float a, b;
    f2_unpack(f2_add(f2_add(v[0], v[1]), f2_add(v[2], v[3])), a, b);
    return __fadd_rn(a, b);
}

__device__ __forceinline__ float dot8(const F8& x, const F8& y) {
    uint64_t s = f2_mul(x[0], y[0]);
#pragma unroll
    for (int k = 1; k < 4; ++k) s = f2_fma(x[k], y[k], s);
    float a, b;
    f2_unpack(s, a, b);
    return __fadd_rn(a, b);
}

template <typename T>
__device__ __forceinline__ Raw<T> narrow(const F8& v) {
    Raw<T> r;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        float a, b;
        f2_unpack(v[k], a, b);
        if constexpr (sizeof(T) == 4) {
            r.w[2 * k] = __float_as_uint(a);
            r.w[2 * k + 1] = __float_as_uint(b);
        } else if constexpr (std::is_same<T, bf16>::value) {
            asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r.w[k]) : "f"(b), "f"(a));
        } else {
            asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r.w[k]) : "f"(b), "f"(a));
        }
    }
    return r;
}

// A lane's four pairs of 16-bit values to a row; every lane of the warp calls it. In a row that
// starts inside a 4-byte word a pair (c, c + 1) straddles two of them: the lane stores the word
// of c - 1 (from the lane before, or its own pair before across the wrap) and c, and single
// values only at the two ends of the warp's columns and of the row.
__device__ __forceinline__ void store_pairs(uint16_t* row, const Cols<kNarrow>& c,
                                            const uint32_t (&w)[4]) {
    if ((reinterpret_cast<uintptr_t>(row) & 3u) == 0) {
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            uint16_t* q = row + c.at(2 * p);
            if (c.mask >> (2 * p + 1) & 1u)
                *reinterpret_cast<uint32_t*>(q) = w[p];
            else if (c.mask >> (2 * p) & 1u)
                *q = (uint16_t)w[p];
        }
        return;
    }
    const uint32_t lane = threadIdx.x & 31u;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
        const uint32_t give = lane == 31u ? (p > 0 ? w[p > 0 ? p - 1 : 0] : 0u) : w[p];
        const uint32_t before = __shfl_sync(0xffffffffu, give, (lane + 31u) & 31u);
        const uint32_t col = c.at(2 * p);
        const bool own = c.mask >> (2 * p) & 1u;
        if (p == 0 && lane == 0) {
            if (own) row[col] = (uint16_t)w[p];
        } else if (own) {
            *reinterpret_cast<uint32_t*>(row + col - 1) = before >> 16 | w[p] << 16;
        } else if (col == c.cols) {
            row[col - 1] = (uint16_t)(before >> 16);
        }
        if (p == 3 && lane == 31u && (c.mask >> 7 & 1u)) row[col + 1] = (uint16_t)(w[p] >> 16);
    }
}

template <typename T, int kA>
__device__ __forceinline__ void store_raw(T* row, const Cols<kA>& c, const Raw<T>& r) {
    if (kA != kNarrow && c.whole()) {
        uint4* p = reinterpret_cast<uint4*>(row + c.c0);
#pragma unroll
        for (int k = 0; k < (int)sizeof(T) / 2; ++k)
            p[k] = make_uint4(r.w[4 * k], r.w[4 * k + 1], r.w[4 * k + 2], r.w[4 * k + 3]);
        return;
    }
    if (kA == kWide) return;
    if constexpr (kA == kNarrow && sizeof(T) == 2) {
        store_pairs(reinterpret_cast<uint16_t*>(row), c, r.w);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (!(c.mask >> j & 1u)) continue;
            if constexpr (sizeof(T) == 4)
                reinterpret_cast<uint32_t*>(row)[c.at(j)] = r.w[j];
            else
                reinterpret_cast<uint16_t*>(row)[c.at(j)] = (uint16_t)(r.w[j / 2] >> 16 * (j & 1));
        }
    }
}

// Larger magnitude of each half (a NaN stays one); the sign bits of the result mean nothing.
template <typename T>
__device__ __forceinline__ uint32_t amax2(uint32_t a, uint32_t b) {
    uint32_t r;
    if constexpr (std::is_same<T, bf16>::value)
        asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else
        asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Bits of T of the largest magnitude in a word of two (they order like the values).
__device__ __forceinline__ uint32_t amax1(uint32_t h) {
    return max(h & 0x7fffu, h >> 16 & 0x7fffu);
}

// Largest magnitude of the lane's first and second four columns, or (neighbours) of all in m[0].
template <typename T, int kA>
__device__ __forceinline__ void lane_amax(const Raw<T>& r, uint32_t (&m)[2]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
            m[k] = max(max(r.w[4 * k] & 0x7fffffffu, r.w[4 * k + 1] & 0x7fffffffu),
                       max(r.w[4 * k + 2] & 0x7fffffffu, r.w[4 * k + 3] & 0x7fffffffu));
        if (kA != kNarrow) m[0] = max(m[0], m[1]);
    } else {
        const uint32_t a = amax2<T>(r.w[0], r.w[1]), b = amax2<T>(r.w[2], r.w[3]);
        if constexpr (kA != kNarrow) {
            m[0] = amax1(amax2<T>(a, b));
        } else {
            m[0] = amax1(a);
            m[1] = amax1(b);
        }
    }
}

// The bits of the binary32 value of a magnitude that lane_amax gave.
template <typename T>
__device__ __forceinline__ uint32_t amax_bits(uint32_t m) {
    if constexpr (sizeof(T) == 4) return m;
    if constexpr (std::is_same<T, bf16>::value) return m << 16;
    return __float_as_uint(h2f((uint16_t)m));
}

// The largest magnitude of each of the warp's two blocks, the same in every lane.
template <typename T, int kA>
__device__ __forceinline__ void block_amax(const Raw<T>& r, uint32_t lane, uint32_t (&a)[2]) {
    uint32_t m[2];
    lane_amax<T, kA>(r, m);
    if constexpr (kA != kNarrow) {   // 16 lanes per block
        m[1] = lane < 16u ? 0u : m[0];
        m[0] = lane < 16u ? m[0] : 0u;
    }
    a[0] = __reduce_max_sync(0xffffffffu, m[0]);
    a[1] = __reduce_max_sync(0xffffffffu, m[1]);
}

// The code words of N chunks of a warp; every value first takes the short way, so that
// the chunks' instructions interleave and one branch covers them all. scale, inv: of the lane's
// block (neighbours), or of the blocks of its first and second four columns.
template <typename T, int kA, int N>
__device__ __forceinline__ void make_codes(const Raw<T> (&raw)[N], const float (&scale)[N][2],
                                           const float (&inv)[N][2], uint2 (&w)[N]) {
    bool fine[N];
    bool all = true;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        float x[8];
        F8 v;
        widen<T>(raw[k], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) f2_unpack(v[j], x[2 * j], x[2 * j + 1]);
        fine[k] = q8_codes(x, scale[k][0], scale[k][kA == kNarrow], inv[k][0], inv[k][kA == kNarrow], w[k]);
        all = all && fine[k];
    }
    if (all) return;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        if (fine[k]) continue;
        float x[8];
        F8 v;
        widen<T>(raw[k], v);
#pragma unroll
        for (int j = 0; j < 4; ++j) f2_unpack(v[j], x[2 * j], x[2 * j + 1]);
        w[k] = q8_codes_near(x, scale[k][0], scale[k][kA == kNarrow], inv[k][0], inv[k][kA == kNarrow]);
    }
}

// Write a chunk's codes and scales into a checkpoint row.
template <int kA>
__device__ __forceinline__ void store_codes(uint8_t* row, const CkptShape& s, const Cols<kA>& c,
                                            uint32_t lane, uint2 w, const float (&scale)[2]) {
    const uint32_t block = c.c0 >> 7;
    if constexpr (kA != kNarrow) {
        if (c.c0 < s.code_bytes) *reinterpret_cast<uint2*>(row + c.c0) = w;
        if ((lane & 15u) == 0 && block < s.blocks)
            *reinterpret_cast<float*>(row + s.code_bytes + 4u * block) = scale[0];
    } else {
#pragma unroll
        for (int p = 0; p < 4; ++p)
            if (c.at(2 * p) < s.code_bytes)
                *reinterpret_cast<uint16_t*>(row + c.at(2 * p)) =
                    (uint16_t)((p < 2 ? w.x : w.y) >> 16 * (p & 1));
#pragma unroll
        for (int k = 0; k < 2; ++k)
            if (lane == 0 && block + k < s.blocks)
                *reinterpret_cast<float*>(row + s.code_bytes + 4u * (block + k)) = scale[k];
    }
}

// Codes and scales of N chunks of a row, the chunks of `at` .. (missing columns hold zeros);
// every lane of the warp calls it. Lane 2k + b divides for block b of chunk k: two divisions for
// all the scales and their reciprocals.
template <typename T, int kA, int N>
__device__ __forceinline__ void save_chunks(uint8_t* row, const CkptShape& s, uint32_t at,
                                            uint32_t stride, uint32_t lane,
                                            const Raw<T> (&raw)[N]) {
    uint32_t mine = 0;
#pragma unroll
    for (int k = 0; k < N; ++k) {
        uint32_t a[2];
        block_amax<T, kA>(raw[k], lane, a);
        if (lane == 2 * k) mine = a[0];
        if (lane == 2 * k + 1) mine = a[1];
    }
    const float own = q8_scale(amax_bits<T>(mine)), own_inv = __fdiv_rn(1.0f, own);
    float scale[N][2], inv[N][2];
#pragma unroll
    for (int k = 0; k < N; ++k) {
        const int from = 2 * k + (kA != kNarrow ? lane >> 4 : 0);
        scale[k][0] = __shfl_sync(0xffffffffu, own, from);
        inv[k][0] = __shfl_sync(0xffffffffu, own_inv, from);
        if (kA == kNarrow) {
            scale[k][1] = __shfl_sync(0xffffffffu, own, from + 1);
            inv[k][1] = __shfl_sync(0xffffffffu, own_inv, from + 1);
        }
    }
    uint2 w[N];
    make_codes<T, kA, N>(raw, scale, inv, w);
#pragma unroll
    for (int k = 0; k < N; ++k)
        store_codes<kA>(row, s, Cols<kA>(at + k * stride, lane, s.cols), lane, w[k], scale[k]);
}

// Zeros behind a row's scales (at most seven words).
__device__ __forceinline__ void save_pad(uint8_t* row, const CkptShape& s, uint32_t lane) {
    const uint64_t at = s.code_bytes + 4ull * s.blocks + 4ull * lane;
    if (at < s.row_bytes) *reinterpret_cast<uint32_t*>(row + at) = 0u;
}

__device__ __forceinline__ void grid_wait() {
    asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void grid_launch_next() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// How the rows of a matrix of `cols` columns can be moved.
template <typename T>
Access access_of(const void* p, uint64_t ld, uint32_t cols) {
    if (!aligned16(p) || ld % (16 / sizeof(T)) != 0) return kNarrow;
    return cols % 8 == 0 ? kWide : kTail;
}

template <typename K, typename... A>
cudaError_t launch_act(K kernel, dim3 grid, unsigned threads, size_t smem, cudaStream_t stream,
                       A... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    count_launch();
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

}  // namespace
}  // namespace zk
