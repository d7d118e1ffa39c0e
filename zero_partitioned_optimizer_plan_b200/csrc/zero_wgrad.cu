// Weight gradient of a linear layer from the 8-bit checkpoint of its input, for sm_100a:
//   dw[o][i] = sum over t of dy[t][o] * a[t][i],   a = q*scale of the checkpoint.
//
// a is rounded to dy's type for the product (the tensor cores take both operands in one 16-bit
// type, and a scale per token and block cannot be taken out of the sum over the tokens). That adds
// an error of 1.65e-4 of dw's size in fp16 (1.4e-3 in bf16) to the 2.1e-4 (1.6e-3) of rounding dw:
// together 2.65e-4 (2.1e-3) against the exact sum, measured at 16384 x 8192 x 2048 and
// 5003 x 1537 x 1100 and the same in exact arithmetic with a rounded. The checkpoint's own half
// step, amax/254 per value, is far above it, and the values are those that zero_ckpt_load_q8 gives
// a recomputation of the layer. Keeping the rest of a needs a second product (a as the sum of two
// 16-bit values): twice the tensor cores' time, which bounds the long sums.
//
// A matrix product whose summation runs over the tokens, so both operands lie in memory with the
// summation index as the slow one ("MN-major" tiles). Bound by the tensor cores for long sums.
//
// A pair of CTAs (two SMs, tcgen05 cta_group::2) computes 256 x 256 or 512 x 256 outputs (kM = 1, 2
// halves of 256 out-features), 64 tokens per stage:
//   A  dy^T, 128 features per CTA and half, by TMA with the 128-byte swizzle (zeros outside the
//      matrix); a dy with an out-feature count that is no multiple of 8 is first copied to aligned
//      rows in the workspace (its rows' starts differ in alignment; loading it in place by the warps
//      that make B took 117 us where the copy and the product take a third); one whose count is, but
//      whose base or stride is not 16-byte aligned, is loaded in place, so that the workspace goes by
//      the sizes alone and no usual call pays for a copy it does not need (16384 x 2304 x 768 with
//      rows one value apart: one call 384 us, aligned 87).
//   B  a, 128 features (one block of codes) per CTA. TMA brings the codes and their scales, eight
//      warps form T(q*scale) as zero_ckpt_load_q8 does and store the tile swizzled. (Codes loaded
//      by those warps into registers, stages ahead, were 4 times slower: the fence between their
//      stores and the tensor cores also waits for every load in flight.)
//   D  binary32 in tensor memory, written out by eight warps. kM = 1: 128 x 256 per CTA, two of
//      them, one written out while the next tile is computed. kM = 2: 256 x 256 per CTA fill it;
//      both halves use each converted tile of B, and the next tile waits for the write-out.
// A cta_group::2 tile reads each half of B once for both SMs; the same tile of one CTA alone
// (128 x 256) would need 3/2 of the shared-memory reads and twice the byte conversions.
//
// Few output tiles and many tokens: the sum is split over pairs of CTAs into binary32 partial
// tiles in the workspace, added in a fixed order by a second kernel.
#include <cuda.h>

#include "zero_act.cuh"

namespace zk {

namespace {

constexpr uint32_t kTileI = 256;                 // in-features per pair of CTAs
constexpr uint32_t kTileK = 64;                  // tokens per stage
constexpr uint32_t kHalf = 128;                  // features per CTA of either operand
constexpr uint32_t kOpBytes = kHalf * kTileK * 2;        // one operand's stage in one CTA
constexpr uint32_t kCodeBytes = kHalf * kTileK;      // a stage's codes in one CTA
constexpr uint32_t kGroupBytes = kTileK * 128;   // 64 features (128 bytes) x 64 tokens
constexpr int kEpiWarps = 8, kConvWarps = 8;
constexpr int kTmaWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kConvWarp0 = 11;
constexpr int kWgradThreads = 32 * (kConvWarp0 + kConvWarps);
constexpr uint32_t kHeadBytes = 2048;            // barriers, tensor-memory address, scales

// A pair's tile has kM * 256 out-features: kM = 1 keeps two accumulators in tensor memory (one
// is written out while the next tile is computed), kM = 2 fills it with one and shares each
// converted B tile between two products.
template <int kM>
struct Shape {
    static constexpr uint32_t kTileO = 256 * kM;
    static constexpr int kStages = kM == 2 ? 4 : 5;
    static constexpr int kAccs = kM == 2 ? 1 : 2;
    static constexpr uint32_t kBAt = kM * kOpBytes, kRawAt = kBAt + kOpBytes;
    static constexpr uint32_t kStageBytes = kRawAt + kCodeBytes;
    static constexpr size_t kSmem = kHeadBytes + (size_t)kStages * kStageBytes + 1024;
    static_assert(kStageBytes % 1024 == 0, "swizzle atoms");
    static_assert(kSmem <= 227 * 1024, "shared memory of one CTA");
};

constexpr int kMaxLoads = 5;
struct Head {
    uint64_t raw[kMaxLoads];     // each CTA: its codes and scales of a stage are there
    uint64_t full[kMaxLoads];    // in the pair's first CTA: both CTAs' A and B of a stage are there
    uint64_t empty[kMaxLoads];   // both: the products that read a stage are done
    uint64_t acc_full[2];        // both: an accumulator is complete
    uint64_t acc_empty[2];       // first CTA: both CTAs have read an accumulator
    uint32_t tmem;
    float scale[kMaxLoads][kTileK];   // of this CTA's 128 features, per token
};
static_assert(sizeof(Head) <= kHeadBytes, "head");

struct WgradPlan {
    uint32_t m;                  // 256 * m out-features per tile
    uint32_t tiles_o, tiles_i;   // output tiles
    uint32_t kblocks;            // stages of the whole sum
    uint32_t splits;             // parts of the sum
    uint32_t split_blocks;       // stages per part
    uint64_t units;              // tiles * splits
};

constexpr uint32_t kPairs = 74;   // pairs of CTAs that run at once

// Tile height and parts of the sum: the smallest modelled time over both heights and every split
// that leaves the pairs at most two rounds. Measured on B200 (us): a stage 0.47 at 256 x 256 and
// 0.62 at 512 x 256 (the taller tile is faster per output when it is filled); the start of a
// tile's pipeline and its write-out 2.5 and 4; adding the parts, 3 for the second kernel and
// 0.06 per 256 x 256 partial tile for its write and read.
WgradPlan wgrad_plan(uint64_t t, uint64_t o, uint64_t i) {
    WgradPlan best = {};
    best.tiles_i = (uint32_t)((i + kTileI - 1) / kTileI);
    best.kblocks = (uint32_t)((t + kTileK - 1) / kTileK);
    float least = 0.0f;
    for (uint32_t m = 1; m <= 2; ++m) {
        const uint64_t tiles_o = (o + 256 * m - 1) / (256 * m), tiles = tiles_o * best.tiles_i;
        for (uint64_t s = 1; s == 1 || (s <= best.kblocks && tiles * s <= 2 * kPairs); ++s) {
            const uint64_t blocks = (best.kblocks + s - 1) / s;
            const uint64_t parts = blocks ? (best.kblocks + blocks - 1) / blocks : 1;
            const uint64_t units = tiles * parts, rounds = (units + kPairs - 1) / kPairs;
            const float cost = (float)rounds * ((float)blocks * (m == 2 ? 0.62f : 0.47f) +
                                                (m == 2 ? 4.0f : 2.5f)) +
                               (parts > 1 ? 3.0f + 0.06f * (float)(units * m) : 0.0f);
            if (best.m && cost >= least) continue;
            least = cost;
            best.m = m;
            best.tiles_o = (uint32_t)tiles_o;
            best.split_blocks = (uint32_t)blocks;
            best.splits = (uint32_t)parts;
            best.units = units;
        }
    }
    return best;
}

}  // namespace

// Partial tiles, then the aligned copy of dy.
static uint64_t partial_bytes(const WgradPlan& p) {
    return p.splits > 1 ? (uint64_t)p.tiles_o * p.tiles_i * p.splits * 256 * p.m * kTileI * 4 : 0;
}

uint64_t wgrad_workspace(uint64_t t, uint64_t o, uint64_t i) {
    return partial_bytes(wgrad_plan(t, o, i)) + (o % 8 ? t * ((o + 7) / 8 * 8) * 2 : 0);
}

namespace {

// ---------------------------------------------------------------------------------------------
// tcgen05, TMA and cluster primitives (PTX)
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile(
        "barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
            : "memory");
}

// Address of the same shared-memory location in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_to(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

// Arrive on a barrier of the pair. What the arrival publishes was written before a proxy fence
// (operand tiles, which only the tensor cores read) or waited for (tensor memory reads), so the
// arrival itself needs no fence of cluster scope: that one waits for the copies in flight too,
// and made the kernel 2.5 times slower.
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr) : "memory");
}

// mbar_wait in line.
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity) {
    uint64_t t0 = 0;
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 63u) == 0) {
            const uint64_t t = globaltimer_ns();
            if (t0 == 0) t0 = t;
            if (t - t0 > kWaitLimitNs) return false;
        }
    }
}

__device__ __forceinline__ void prefetch_map(const CUtensorMap* map) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}

// 2-D tile global -> this CTA's shared memory; the bytes count on a barrier of the pair.
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, int x, int y,
                                         uint32_t cluster_bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(cluster_bar)
        : "memory");
}

// The same, counted on this CTA's own barrier.
__device__ __forceinline__ void tma_own(uint32_t dst, const CUtensorMap* map, int x, int y,
                                        uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(smem_addr(bar))
        : "memory");
}

// Shared-memory descriptor of an MN-major tile with the 128-byte swizzle: 8 tokens of a group
// of 64 features are 1024 bytes; the next 8 tokens follow (stride 1024), the next 64 features
// are kGroupBytes away.
__device__ __forceinline__ uint64_t tile_desc(uint32_t addr) {
    constexpr uint64_t fixed = (uint64_t)(kGroupBytes >> 4) << 16 |   // next 64 features
                               (uint64_t)(1024 >> 4) << 32 |          // next 8 tokens
                               1ull << 46 |                           // descriptor version
                               2ull << 61;                            // 128-byte swizzle
    return fixed | (uint64_t)(addr >> 4);
}

// Instruction descriptor: binary32 accumulator, both operands T and MN-major, 256 x 256.
template <typename T>
__device__ __forceinline__ constexpr uint32_t mma_desc() {
    constexpr uint32_t fmt = std::is_same<T, bf16>::value ? 1u : 0u;
    return 1u << 4 | fmt << 7 | fmt << 10 | 1u << 15 | 1u << 16 | (kTileI >> 3) << 17 |
           (256u >> 4) << 24;
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                         bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)add)
        : "memory");
}

// Arrive on both CTAs' copy of `bar` when the products issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64"
        " [%0], %1;" ::"r"(smem_addr(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 32 columns of this warp's 32 lanes of tensor memory.
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&v)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, "
        "%19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
          "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
          "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
          "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
          "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
        : "r"(addr)
        : "memory");
}

// ---------------------------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------------------------
struct WgradCall {
    WgradArgs a;
    WgradPlan plan;
    float* partial;      // splits > 1: [unit][256 * m][256] binary32
    int vec;             // widest store into dw its base and stride allow, in bytes
};

struct WgradMaps {
    CUtensorMap dy, codes;
};

struct Unit {
    uint32_t o0, i0, kb0, kb1;
};

// Unit n: the parts of one tile are neighbours; tiles run in bands of 8 along the in-features,
// so that the pairs running at once share the rows of dy and codes they read (through L2).
__device__ __forceinline__ Unit unit_at(const WgradPlan& p, uint64_t n) {
    const uint32_t part = (uint32_t)(n % p.splits);
    const uint32_t tile = (uint32_t)(n / p.splits);
    const uint32_t band = tile / (8 * p.tiles_o);
    const uint32_t in_band = tile - band * 8 * p.tiles_o;
    const uint32_t width = min(8u, p.tiles_i - band * 8);
    Unit u;
    u.o0 = in_band / width * 256u * p.m;
    u.i0 = (band * 8 + in_band % width) * kTileI;
    u.kb0 = part * p.split_blocks;
    u.kb1 = min(u.kb0 + p.split_blocks, p.kblocks);
    return u;
}

template <typename T>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if constexpr (std::is_same<T, bf16>::value)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Four codes to four T: the byte is placed in the mantissa of 2^23 (exact), the bias 2^23 + 128
// taken off (exact), then the product with the scale, rounded as a binary32 product and to T.
template <typename T>
__device__ __forceinline__ uint2 widen4(uint32_t w, float s) {
    float f[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
        f[j] = __fmul_rn(__fsub_rn(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7540u + j)),
                                   8388736.0f),
                         s);
    return make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w)
                 : "memory");
}

// Byte offset of 16-byte chunk `ch` (8 features) of token row k in an operand tile.
__device__ __forceinline__ uint32_t chunk_at(uint32_t ch, uint32_t k) {
    return (ch >> 3) * kGroupBytes + k * 128u + (((ch ^ k) & 7u) << 4);
}

__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// 4 bytes global -> shared memory without a register (zeros where !there).
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, bool there) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src),
                 "r"(there ? 4 : 0)
                 : "memory");
}

// Arrive on `bar` when this thread's copies so far have landed.
__device__ __forceinline__ void arrive_after_copies(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar))
                 : "memory");
}

// A stage's codes to T: lane l of warp w takes columns 16*(l%8) .. of token rows 4w + l/8 and
// 32 + 4w + l/8.
template <typename T>
__device__ __forceinline__ void convert_stage(uint32_t raw, const float* scale, uint32_t tile,
                                              uint32_t lane, uint32_t w) {
    const uint32_t k0 = 4u * w + (lane >> 3), ch = 2u * (lane & 7u);
    // lanes of the second group of 64 features store their chunks in the other order: a quarter
    // warp then covers all eight 16-byte columns of the banks
    const uint32_t swap = (lane >> 2) & 1u;
    uint4 q[2];
    float s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        q[j] = ld_shared16(raw + (k0 + 32u * j) * kHalf + 8u * ch);
        s[j] = *(volatile const float*)(scale + k0 + 32u * j);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const uint32_t k = k0 + 32u * j;
        const uint2 a = widen4<T>(q[j].x, s[j]), b = widen4<T>(q[j].y, s[j]);
        const uint2 d = widen4<T>(q[j].z, s[j]), e = widen4<T>(q[j].w, s[j]);
        const uint4 lo = make_uint4(a.x, a.y, b.x, b.y), hi = make_uint4(d.x, d.y, e.x, e.y);
        st_shared16(tile + chunk_at(ch + swap, k), swap ? hi : lo);
        st_shared16(tile + chunk_at(ch + 1u - swap, k), swap ? lo : hi);
    }
}

// A's tile by plain loads, for a dy that TMA cannot address: 128 features x 64 tokens.
template <typename T>
__device__ __forceinline__ void store_dy(const WgradArgs& a, uint32_t tile, uint32_t o0,
                                         uint64_t t0, uint32_t thread) {
    const uint16_t* dy = reinterpret_cast<const uint16_t*>(a.dy.p);
#pragma unroll 1
    for (uint32_t e = thread; e < 16 * kTileK; e += 32 * kConvWarps) {
        const uint32_t ch = e & 15u, k = e >> 4, o = o0 + 8u * ch;
        const uint64_t t = t0 + k;
        uint32_t w[4] = {};
        if (t < a.tokens) {
            const uint16_t* src = dy + t * a.dy.ld + o;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (o + j < a.outf) w[j >> 1] |= (uint32_t)__ldg(src + j) << (16 * (j & 1));
        }
        st_shared16(tile + chunk_at(ch, k), make_uint4(w[0], w[1], w[2], w[3]));
    }
}

// 32 consecutive values of a row of dw, 16-byte aligned.
template <typename T>
__device__ __forceinline__ void store_row(T* p, const uint32_t (&v)[32], bool add) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) f[k] = __uint_as_float(v[8 * j + k]);
        if (add) {
            const uint4 o = *reinterpret_cast<const uint4*>(p + 8 * j);
            const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const uint16_t h = (uint16_t)(w[k >> 1] >> (16 * (k & 1)));
                T t;
                memcpy(&t, &h, 2);
                f[k] = __fadd_rn(to_f(t), f[k]);
            }
        }
        *reinterpret_cast<uint4*>(p + 8 * j) = make_uint4(
            pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]), pack2<T>(f[4], f[5]), pack2<T>(f[6], f[7]));
    }
}

// 32 rows (one per lane) x 32 columns of dw at any alignment: transposed between the lanes first,
// so that a store covers 32 neighbours of one row (lane by lane along its own row, the 2-byte
// stores took 77 us for 7085 x 668 outputs of 4 tokens, which now take 19).
template <typename T>
__device__ __forceinline__ void store_tile(T* p, uint64_t ld, uint32_t lane, uint32_t rows,
                                           uint32_t cols, uint32_t (&v)[32], bool add) {
#pragma unroll
    for (int s = 16; s > 0; s >>= 1) {
        const bool up = lane & s;
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (!(i & s)) {
                const uint32_t x = __shfl_xor_sync(0xffffffffu, up ? v[i] : v[i + s], s);
                if (up)
                    v[i] = x;
                else
                    v[i + s] = x;
            }
    }
    if (lane >= cols) return;
#pragma unroll
    for (int r = 0; r < 32; ++r)
        if (r < rows) {
            T* q = p + r * ld + lane;
            const float f = __uint_as_float(v[r]);
            *q = from_f<T>(add ? __fadd_rn(to_f(*q), f) : f);
        }
}

template <typename T, bool kTma, int kM>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kWgradThreads, 1)
    wgrad_kernel(const __grid_constant__ WgradCall p, const __grid_constant__ WgradMaps maps) {
    using S = Shape<kM>;
    constexpr int kStages = S::kStages, kAccs = S::kAccs;
    constexpr uint32_t kStageBytes = S::kStageBytes;
    extern __shared__ uint8_t raw[];
    uint8_t* base = raw + ((1024u - (smem_addr(raw) & 1023u)) & 1023u);   // swizzle atoms: 1024
    Head& hd = *reinterpret_cast<Head*>(base);
    const uint32_t tiles = smem_addr(base) + kHeadBytes;
    const int warp = threadIdx.x >> 5;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const uint64_t pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

    if (threadIdx.x == 32 * kTmaWarp) {
        if (kTma) prefetch_map(&maps.dy);
        prefetch_map(&maps.codes);
    }
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&hd.raw[s], 1 + 32);
            mbar_init(&hd.full[s], (kTma ? 1 : 0) + 2 * kConvWarps);
            mbar_init(&hd.empty[s], 1);
        }
        for (int b = 0; b < kAccs; ++b) {
            mbar_init(&hd.acc_full[b], 1);
            mbar_init(&hd.acc_empty[b], 2 * kEpiWarps);
        }
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                         smem_addr(&hd.tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
    const uint32_t tmem = hd.tmem;
    grid_wait();

    bool ok = true;
    if (warp == kTmaWarp) {
        if (lane == 0) {
            uint32_t it = 0;
            for (uint64_t n = pair; ok && n < p.plan.units; n += pairs) {
                const Unit u = unit_at(p.plan, n);
                for (uint32_t kb = u.kb0; kb < u.kb1; ++kb, ++it) {
                    const uint32_t s = it % kStages, use = it / kStages;
                    ok = wait_on(&hd.empty[s], (use & 1u) ^ 1u);
                    if (!ok) break;
                    const uint32_t dst = tiles + s * kStageBytes;
                    const int y = (int)(kb * kTileK), col = (int)(u.i0 + rank * kHalf);
                    mbar_arrive_expect_tx(&hd.raw[s], kCodeBytes);
                    tma_own(dst + S::kRawAt, &maps.codes, col, y, &hd.raw[s]);
                    if (kTma) {
                        const uint32_t full = map_to(smem_addr(&hd.full[s]), 0);
                        if (rank == 0) mbar_arrive_expect_tx(&hd.full[s], 2 * kM * kOpBytes);
#pragma unroll
                        for (int m = 0; m < kM; ++m) {
                            const int x = (int)(u.o0 + m * 256 + rank * kHalf);
                            const uint32_t at = dst + m * kOpBytes;
                            tma_tile(at, &maps.dy, x, y, full);
                            tma_tile(at + kGroupBytes, &maps.dy, x + 64, y, full);
                        }
                    }
                }
            }
        }
    } else if (warp == kScaleWarp) {
        uint32_t it = 0;
        for (uint64_t n = pair; ok && n < p.plan.units; n += pairs) {
            const Unit u = unit_at(p.plan, n);
            const uint32_t block = (u.i0 + rank * kHalf) / 128u;
            const uint32_t at = p.a.ck.code_bytes + 4u * min(block, p.a.ck.blocks - 1);
            for (uint32_t kb = u.kb0; kb < u.kb1; ++kb, ++it) {
                const uint32_t s = it % kStages;
                ok = __all_sync(0xffffffffu, wait_on(&hd.empty[s], ((it / kStages) & 1u) ^ 1u));
                if (!ok) break;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint32_t k = lane + 32u * j;
                    const uint64_t t = (uint64_t)kb * kTileK + k;
                    const bool there = t < p.a.tokens;
                    copy4(smem_addr(&hd.scale[s][k]),
                          p.a.ckpt + (there ? t : 0) * p.a.ck.row_bytes + at, there);
                }
                arrive_after_copies(&hd.raw[s]);
            }
        }
    } else if (warp == kMmaWarp) {
        if (rank == 0 && lane == 0) {
            uint32_t it = 0, tile = 0;
            for (uint64_t n = pair; ok && n < p.plan.units; n += pairs, ++tile) {
                const Unit u = unit_at(p.plan, n);
                const uint32_t b = tile % kAccs;
                ok = wait_on(&hd.acc_empty[b], ((tile / kAccs) & 1u) ^ 1u);
                if (!ok) break;
                asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                const uint32_t d = tmem + b * kTileI;
                for (uint32_t kb = u.kb0; kb < u.kb1; ++kb, ++it) {
                    const uint32_t s = it % kStages;
                    ok = wait_on(&hd.full[s], (it / kStages) & 1u);
                    if (!ok) break;
                    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
                    const uint32_t st = tiles + s * kStageBytes;
#pragma unroll
                    for (uint32_t k = 0; k < kTileK / 16; ++k)   // 16 tokens = 2048 bytes
#pragma unroll
                        for (uint32_t m = 0; m < kM; ++m)
                            mma_pair(d + m * kTileI, tile_desc(st + m * kOpBytes + k * 2048u),
                                     tile_desc(st + S::kBAt + k * 2048u), mma_desc<T>(),
                                     kb > u.kb0 || k > 0);
                    commit_pair(&hd.empty[s]);
                }
                if (ok) commit_pair(&hd.acc_full[b]);
            }
        }
    } else if (warp >= kConvWarp0) {
        const uint32_t w = warp - kConvWarp0;
        uint32_t it = 0;
        for (uint64_t n = pair; ok && n < p.plan.units; n += pairs) {
            const Unit u = unit_at(p.plan, n);
            for (uint32_t kb = u.kb0; kb < u.kb1; ++kb, ++it) {
                const uint32_t s = it % kStages, st = tiles + s * kStageBytes;
                // the stage's codes were asked for after its last products ended
                ok = __all_sync(0xffffffffu, wait_on(&hd.raw[s], (it / kStages) & 1u));
                if (!ok) break;
                convert_stage<T>(st + S::kRawAt, hd.scale[s], st + S::kBAt, lane, w);
                if (!kTma)
                    for (uint32_t m = 0; m < kM; ++m)
                        store_dy<T>(p.a, st + m * kOpBytes, u.o0 + m * 256u + rank * kHalf,
                                    (uint64_t)kb * kTileK, w * 32u + lane);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) arrive_at(map_to(smem_addr(&hd.full[s]), 0));
            }
        }
        // the last use of every stage: no arrival may reach a CTA that has left
        for (uint32_t j = it < kStages ? 0 : it - kStages; ok && j < it; ++j)
            ok = __all_sync(0xffffffffu, wait_on(&hd.empty[j % kStages], (j / kStages) & 1u));
    } else {   // write the results: lanes 32*(warp%4) .. of tensor memory, half of the columns
        const uint32_t quarter = warp & 3u, first = (warp >> 2) * kM * kTileI / 2;
        uint32_t tile = 0;
        for (uint64_t n = pair; ok && n < p.plan.units; n += pairs, ++tile) {
            const Unit u = unit_at(p.plan, n);
            const uint32_t b = tile % kAccs;
            ok = __all_sync(0xffffffffu, wait_on(&hd.acc_full[b], (tile / kAccs) & 1u));
            if (!ok) break;
            asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
#pragma unroll 1
            for (uint32_t c = first; c < first + kM * kTileI / 2; c += 32) {
                const uint32_t row0 = c / kTileI * 256u + rank * kHalf + 32u * quarter;
                const uint32_t row = row0 + lane, o = u.o0 + row0, i = u.i0 + c % kTileI;
                uint32_t v[32];
                tmem_load(tmem + b * kTileI + c + (quarter << 21), v);
                if (p.partial) {
                    float4* out = reinterpret_cast<float4*>(
                        p.partial + (n * S::kTileO + row) * kTileI + c % kTileI);
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        out[j] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                             __uint_as_float(v[4 * j + 2]),
                                             __uint_as_float(v[4 * j + 3]));
                } else if (o < p.a.outf && i < p.a.inf) {
                    T* dw = (T*)p.a.dw.p + o * p.a.dw.ld + i;
                    const uint32_t cols = p.a.inf - i, rows = p.a.outf - o;
                    if (p.vec == 16 && cols >= 32) {
                        if (lane < rows)
                            store_row<T>(dw + lane * p.a.dw.ld, v, p.a.accumulate != 0);
                    } else {
                        store_tile<T>(dw, p.a.dw.ld, lane, rows, cols, v, p.a.accumulate != 0);
                    }
                }
            }
            asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
            __syncwarp();
            if (lane == 0) arrive_at(map_to(smem_addr(&hd.acc_empty[b]), 0));
        }
    }
    if (!ok) {   // a wait gave up: flag it, and let the copies in flight land before leaving
        if (lane == 0) atomicOr(p.a.status, ZERO_FLAG_TIMEOUT);
        const uint64_t t0 = globaltimer_ns();
        while (globaltimer_ns() - t0 < 20000000ull) __nanosleep(1000);
    }
    __syncwarp();
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
    __syncthreads();
    cluster_sync();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem)
                     : "memory");
    }
    cluster_sync();
    if (p.partial) grid_launch_next();   // the kernel that adds the parts: this call's own
}

// dw = the parts of each tile added in order (+ dw), or zeros where there is no token.
template <typename T>
__global__ void __launch_bounds__(256) wgrad_join_kernel(WgradArgs a, WgradPlan plan,
                                                         const float* partial, int vec) {
    grid_wait();
    const uint32_t cols = (a.inf + 3) / 4;
    const uint64_t total = (uint64_t)a.outf * cols;
    for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < total;
         e += (uint64_t)gridDim.x * 256) {
        const uint32_t o = (uint32_t)(e / cols), i = (uint32_t)(e - (uint64_t)o * cols) * 4;
        float f[4] = {};
        if (partial) {
            const uint32_t tile_o = 256 * plan.m, to = o / tile_o, ti = i / kTileI;
            const uint32_t band = ti / 8, width = min(8u, plan.tiles_i - band * 8);
            const uint64_t tile = (uint64_t)band * 8 * plan.tiles_o + (uint64_t)to * width + ti % 8;
            const float* src = partial + (tile * plan.splits * tile_o + o % tile_o) * kTileI + i % kTileI;
            for (uint32_t s = 0; s < plan.splits; ++s) {
                const float4 v = *reinterpret_cast<const float4*>(src + (uint64_t)s * tile_o * kTileI);
                f[0] = __fadd_rn(f[0], v.x);
                f[1] = __fadd_rn(f[1], v.y);
                f[2] = __fadd_rn(f[2], v.z);
                f[3] = __fadd_rn(f[3], v.w);
            }
        }
        T* d = (T*)a.dw.p + o * a.dw.ld + i;
        if (vec >= 8 && i + 4 <= a.inf) {
            if (a.accumulate) {
                const uint2 old = *reinterpret_cast<const uint2*>(d);
                T t[4];
                memcpy(t, &old, 8);
#pragma unroll
                for (int j = 0; j < 4; ++j) f[j] = __fadd_rn(to_f(t[j]), f[j]);
            }
            *reinterpret_cast<uint2*>(d) = make_uint2(pack2<T>(f[0], f[1]), pack2<T>(f[2], f[3]));
            continue;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i + j < a.inf)
                d[j] = from_f<T>(a.accumulate ? __fadd_rn(to_f(d[j]), f[j]) : f[j]);
    }
}

// dy's rows to aligned rows of `pitch` (a multiple of 8) values; the values behind a row are not
// read later. A thread moves eight values: five 4-byte loads shifted together where the source is
// not 4-byte aligned (four where it is), single loads at a row's ends.
__global__ void __launch_bounds__(256) align_rows_kernel(uint64_t rows, uint32_t cols, Mat src,
                                                         uint16_t* dst, uint32_t pitch) {
    grid_wait();
    grid_launch_next();
    const uint32_t chunks = pitch / 8;
    const uint64_t total = rows * chunks;
    for (uint64_t e = (uint64_t)blockIdx.x * 256 + threadIdx.x; e < total;
         e += (uint64_t)gridDim.x * 256) {
        const uint64_t r = e / chunks;
        const uint32_t c = (uint32_t)(e - r * chunks) * 8;
        const uint16_t* p = (const uint16_t*)src.p + r * src.ld + c;
        uint32_t w[4];
        if (c > 0 && c + 8 < cols) {
            const uint32_t* q = reinterpret_cast<const uint32_t*>((uintptr_t)p & ~(uintptr_t)3);
            const uint32_t shift = ((uintptr_t)p & 2u) * 8u;   // 0 or 16 bits
            uint32_t v[5];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = __ldg(q + j);
            v[4] = shift ? __ldg(q + 4) : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = __funnelshift_r(v[j], v[j + 1], shift);
        } else {
            uint32_t v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = c + j < cols ? __ldg(p + j) : 0u;
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = v[2 * j] | v[2 * j + 1] << 16;
        }
        *reinterpret_cast<uint4*>(dst + r * pitch + c) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                              const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                              const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

cudaError_t encode_fn(EncodeFn* out) {
    static std::atomic<void*> fn{nullptr};
    void* f = fn.load(std::memory_order_relaxed);
    if (!f) {
        cudaDriverEntryPointQueryResult q;
        const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                               cudaEnableDefault, &q);
        if (e != cudaSuccess) return e;
        if (q != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
        fn.store(f, std::memory_order_relaxed);
    }
    *out = reinterpret_cast<EncodeFn>(f);
    return cudaSuccess;
}

cudaError_t encode_2d(EncodeFn encode, CUtensorMap* map, CUtensorMapDataType type, void* p,
                      uint64_t cols, uint64_t rows, uint64_t pitch, uint32_t box_cols,
                      CUtensorMapSwizzle swizzle) {
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {pitch};
    const cuuint32_t box[2] = {box_cols, kTileK}, step[2] = {1, 1};
    const CUresult r = encode(map, type, 2, p, dims, strides, box, step,
                              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// dy in boxes of 64 features x 64 tokens, swizzled; the checkpoint's bytes in boxes of 128 codes
// x 64 tokens. Zeros outside.
cudaError_t make_maps(const WgradArgs& a, int dtype, bool tma, WgradMaps* m) {
    EncodeFn encode;
    cudaError_t e = encode_fn(&encode);
    if (e == cudaSuccess && tma)
        e = encode_2d(encode, &m->dy,
                      dtype == ZERO_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
                      a.dy.p, a.outf, a.tokens, a.dy.ld * 2, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    void* ck = const_cast<uint8_t*>(a.ckpt);
    const uint64_t rb = a.ck.row_bytes;
    if (e == cudaSuccess)
        e = encode_2d(encode, &m->codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, ck, rb, a.tokens, rb,
                      kHalf, CU_TENSOR_MAP_SWIZZLE_NONE);
    return e;
}

template <typename T, bool kTma, int kM>
cudaError_t run_pairs(const WgradCall& c, const WgradMaps& maps, int sms, cudaStream_t stream) {
    auto kernel = wgrad_kernel<T, kTma, kM>;
    constexpr size_t smem = Shape<kM>::kSmem;
    thread_local int ready_on = -1;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (ready_on != dev) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)smem);
        if (e != cudaSuccess) return e;
        ready_on = dev;
    }
    const uint64_t most = (uint64_t)(sms / 2);
    const uint64_t pairs = c.plan.units < most ? c.plan.units : most;
    return launch_act(kernel, dim3((unsigned)(2 * pairs)), kWgradThreads, smem, stream, c,
                      maps);
}

template <typename T>
cudaError_t run_wgrad(const WgradArgs& a, int dtype, void* ws, cudaStream_t stream) {
    DevInfo di;
    cudaError_t e = dev_info(&di);
    if (e != cudaSuccess) return e;
    WgradCall c = {};
    c.a = a;
    c.plan = wgrad_plan(a.tokens, a.outf, a.inf);
    c.partial = c.plan.splits > 1 ? (float*)ws : nullptr;
    c.vec = aligned16(a.dw.p) && a.dw.ld % 8 == 0 ? 16 : 2;
    if (a.tokens) {
        // (a single row's stride is used for nothing: any, also one too large for a tensor map)
        if (a.tokens == 1) c.a.dy.ld = ((uint64_t)a.outf + 7) / 8 * 8;
        bool tma = aligned16(a.dy.p) && c.a.dy.ld % 8 == 0;
        if (!tma && a.outf % 8 != 0) {
            const uint32_t pitch = (a.outf + 7) / 8 * 8;
            uint16_t* copy = reinterpret_cast<uint16_t*>((char*)ws + partial_bytes(c.plan));
            e = launch_act(align_rows_kernel, dim3(plain_grid(a.tokens * (pitch / 8), di.sms, 16)),
                           256, 0, stream, a.tokens, a.outf, a.dy, copy, pitch);
            if (e != cudaSuccess) return e;
            c.a.dy = Mat{copy, pitch};
            tma = true;
        }
        WgradMaps maps = {};
        e = make_maps(c.a, dtype, tma, &maps);
        if (e != cudaSuccess) return e;
        e = c.plan.m == 2 ? (tma ? run_pairs<T, true, 2>(c, maps, di.sms, stream)
                                 : run_pairs<T, false, 2>(c, maps, di.sms, stream))
                          : (tma ? run_pairs<T, true, 1>(c, maps, di.sms, stream)
                                 : run_pairs<T, false, 1>(c, maps, di.sms, stream));
        if (e != cudaSuccess || !c.partial) return e;
    }
    const uint64_t quads = (uint64_t)a.outf * ((a.inf + 3) / 4);
    return launch_act(wgrad_join_kernel<T>, dim3(plain_grid(quads, di.sms)), 256, 0, stream, a,
                      c.plan, (const float*)c.partial, c.vec);
}

}  // namespace

cudaError_t launch_wgrad(const WgradArgs& a, int dtype, void* ws, cudaStream_t stream) {
    return dtype == ZERO_F16 ? run_wgrad<__half>(a, dtype, ws, stream)
                             : run_wgrad<bf16>(a, dtype, ws, stream);
}

}  // namespace zk
