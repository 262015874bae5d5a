// Product of two microscaled 4-bit matrices on the 5th-generation tensor cores.
//
//   acc[i,j] = sum_k (Xq[i,k] bx[i,k/B]) (Wq[j,k] bw[j,k/B])     fp32 sum
//   Y[i,j]   = acc * ((1/qs_x[i]) (1/qs_w[j])) (+ bias[j]), one rounding
// with E2M1 codes and block scales b (NVFP4: blocks of 16, E4M3; MXFP4: blocks
// of 32, E8M0). The tensor core multiplies by the block scales itself
// (tcgen05.mma kind::mxf4nvf4 / kind::mxf4, K = 64 an instruction).
//
// Design: that of the int8 GEMM (a persistent, warp-specialised CTA per SM; one
// TMA producer thread, one MMA issuer, eight epilogue warps), with
//   - stages of 256 codes of K (128 bytes a row, 128-byte swizzle), and beside
//     them the stage's block scales: the scale tiles are in global memory as
//     tensor memory wants them, so a stage's scales of 128 rows are 2 KB (1 KB)
//     in one piece;
//   - four scale warps bring each stage's scales from shared to tensor memory
//     (tcgen05.st, each its lane quarter) into one of two sets of columns, while
//     the MMAs of the stage before run. (tcgen05.cp copies them without warps,
//     but runs in one queue with the MMAs, about 50 cycles for each of a pair
//     stage's 12: 4096 x 12288 x 12288 took 408 us so, in any order of issue.)
//   - CTA pairs (256 x 256 tiles): two accumulators of 256 columns and the
//     scales' two sets of 48 (24) columns exceed the 512 of tensor memory, so the
//     accumulators share 96 (48): the epilogue reads the shared columns first
//     and hands them back, and the next tile's MMAs start while the rest is read;
//   - a last wave of pair tiles that is not full: its tiles are cut by k-blocks
//     into one contiguous range per pair, run before the whole tiles; a piece's
//     sums are parked in the workspace, and the piece that completes a tile adds
//     them in range order (1024 x 7168 x 28672, 112 tiles on 74 pairs: 106 us in
//     two waves, 92 so);
//   - few tiles (decode batches): a kernel of its own, one 128 x 128 tile (or one
//     part of its k-loop) per CTA, two CTAs per SM; the parts of a tile are a
//     cluster, which adds them up through its shared memory, in part order.
//     (Parked in global memory and counted by atomics, the parts cost 2.5 us
//     more: 16 x 4096 x 4096 9.9 us, so 6.2 us.)
// What bounds it at 4096 x 12288 x 12288 (NVFP4 253-280 us over devices, ten calls in
// a row, 4.4-4.9 PFLOP/s): called without end, the power cap (990 W, the SM clock at
// 1.59 of 1.965 GHz, 311 us). In short runs the tensor cores are active 55 % of the
// cycles and nothing that was measured is full: L2 delivers 11.4 TB/s, where the
// int8 pair kernel takes 12.0 with its tensor cores active 89 %; and MXFP4, with half
// the scale bytes, is no faster (250-268 us). The scales' way to tensor memory starts
// only when the MMAs of two stages before are complete. Few rows: the weight's bytes
// and latency (16 x 12288 x 12288 18.4 us, 13.1 of bytes; 16 x 16384 x 4096 9.4, 5.9).
// Every wait is bounded (about 2 s), code 0x8E1 + role in the status word.
#include <cstring>
#include <type_traits>

#include "sq_common.cuh"
#include "sq_fp4.cuh"
#include "sq_internal.h"
#include "sq_tc.cuh"

namespace sq {
namespace {

constexpr int BM = 128;
constexpr int BN = 256, CG = 2;  // the pair kernel's tile: 2 x BM rows, BN columns
constexpr int BK = 256;        // codes per stage: 128 bytes, one swizzle row
constexpr int UMMA_K = 64;     // codes per MMA: 32 bytes
constexpr int kEpiWarps = 8;   // two per TMEM lane quarter, each on half the tile's columns
constexpr int kScaleWarps = 4;  // one per TMEM lane quarter
constexpr int kThreads = 64 + 32 * (kEpiWarps + kScaleWarps);
constexpr int kStgRow = 80;    // staging: 32 rows x 64 B + 16 B pad (the TMA-store box uses the first 2 KB)
constexpr int kStgWarpBytes = 32 * kStgRow;
static_assert(kStgWarpBytes % 512 == 0, "staging slots must keep the 64-byte swizzle's 512-byte alignment");
enum OutKind { kOutBF16 = 0, kOutF16 = 1, kOutF32 = 2 };

// Instruction descriptor: E2M1 operands (format 1 at bits 7 and 10), K-major,
// N >> 3 at bit 17, scale format at bit 23 (0 E4M3, 1 E8M0), M >> 4 at bit
// 24; which byte of a scale word to start from: bit 4 (B), bit 29 (A).
template <int FMT>
__device__ constexpr uint32_t idesc_fp4(int m, int n, int sf) {
    return (1u << 7) | (1u << 10) | ((uint32_t)(n >> 3) << 17) | ((FMT == SQ_MXFP4 ? 1u : 0u) << 23) |
           ((uint32_t)(m >> 4) << 24) | ((uint32_t)sf << 4) | ((uint32_t)sf << 29);
}

template <int FMT>
struct Cfg {
    static constexpr int STAGES = 5;
    static constexpr int CHUNKS = FMT == SQ_NVFP4 ? 4 : 2;  // scale tiles (4 blocks) per stage and row group
    static constexpr int NG = BN / 128;                     // row groups of the weight's scales
    static constexpr uint32_t A_BYTES = BM * BK / 2;
    static constexpr uint32_t B_BYTES = (BN / CG) * BK / 2;
    static constexpr uint32_t SA_BYTES = CHUNKS * kFp4TileBytes;
    static constexpr uint32_t SB_BYTES = NG * CHUNKS * kFp4TileBytes;
    static constexpr uint32_t A_OFF = 0;
    static constexpr uint32_t B_OFF = A_OFF + STAGES * A_BYTES;
    static constexpr uint32_t SA_OFF = B_OFF + STAGES * B_BYTES;
    static constexpr uint32_t SB_OFF = SA_OFF + STAGES * SA_BYTES;
    static constexpr uint32_t BAR_OFF = SB_OFF + STAGES * SB_BYTES;  // full[S], empty[S], tfull[2], tempty[2], drain, sfull[S], sready[S]
    static constexpr uint32_t MISC_OFF = BAR_OFF + (4 * STAGES + 5) * 8;
    static constexpr uint32_t RW_OFF = (MISC_OFF + 16 + 15) / 16 * 16;
    static constexpr uint32_t RW_BYTES = kEpiWarps * 2 * (BN / 2) * 4;
    static constexpr uint32_t STG_OFF = (RW_OFF + RW_BYTES + 1023) / 1024 * 1024;
    static constexpr uint32_t SMEM = STG_OFF + kEpiWarps * kStgWarpBytes;
    static constexpr uint32_t SMEM_ALLOC = SMEM + 1024;
    static_assert(SMEM_ALLOC <= 232448, "over the 227 KB of shared memory a block may use");
    // tensor memory: two sets of scales (the weight's, then X's) in the last
    // columns, the accumulators before them
    static constexpr uint32_t TMEM_COLS = 512;
    static constexpr uint32_t SB_COLS = CHUNKS * NG * 4;
    static constexpr uint32_t SET_COLS = SB_COLS + CHUNKS * 4;
    static constexpr uint32_t SF_COL = TMEM_COLS - 2 * SET_COLS;
    static constexpr uint32_t ACC1 = SF_COL - BN;  // first column of the second accumulator
    // 32-column chunks of a half accumulator that the next tile waits for
    static constexpr int SHARED = (int)(BN - ACC1 + 31) / 32;
    static_assert(SHARED <= BN / 64, "the shared columns lie in one half of the accumulator");
    static __device__ constexpr uint32_t idesc(int sf) { return idesc_fp4<FMT>(BM * CG, BN, sf); }
};

struct Params {
    int M, N, K;
    int num_m, num_n, num_kb;
    int group_m;
    int vec_store, tma_store;
    const float* qs_x;
    const float* qs_w;
    const float* bias;
    int x_per_token, w_per_channel;
    void* Y;
    int64_t ldy;
    int* status;
    // the last wave's split: the first dp_tiles tiles run whole; the k-blocks of
    // the other sk_tiles, sk_iters in all, are dealt to the pairs
    int dp_tiles, sk_tiles, sk_iters, sk_units;
    int sk_cnt_bytes;
    int* sk_cnt;     // [sk_tiles][CG][kEpiWarps] k-blocks counted in (zero between launches)
    float* sk_part;  // [CTA][2][kEpiWarps][NCH][8][32] float4
};

// First k-block of unit c's range, and the unit whose range holds k-block x
// (every unit has at least one: sk_iters >= sk_units).
__device__ __forceinline__ int sk_start(int c, const Params& p) {
    return (int)((int64_t)c * p.sk_iters / p.sk_units);
}
__device__ __forceinline__ int sk_owner(int x, const Params& p) {
    return (int)((((int64_t)x + 1) * p.sk_units + p.sk_iters - 1) / p.sk_iters - 1);
}

// A unit's work, the same sequence for all its roles: the pieces of its range
// (the part inside one tile each; slot 0 for the first, 1 for the last, -1 where
// a piece is a whole tile), then its whole tiles.
template <bool SK>
struct Segments {
    int tile_dp, it, end;
    bool first;
    __device__ __forceinline__ explicit Segments(const Params& p) {
        tile_dp = blockIdx.x / CG;
        it = SK ? sk_start(blockIdx.x / CG, p) : 0;
        end = SK ? sk_start(blockIdx.x / CG + 1, p) : 0;
        first = true;
    }
    __device__ __forceinline__ bool next(const Params& p, int& tile, int& k0, int& k1, int& slot) {
        if (SK && it < end) {
            const int u = it / p.num_kb;
            k0 = it - u * p.num_kb;
            k1 = min(p.num_kb, k0 + (end - it));
            tile = p.dp_tiles + u;
            slot = (k0 == 0 && k1 == p.num_kb) ? -1 : (first ? 0 : 1);
            first = false;
            it += k1 - k0;
            return true;
        }
        tile = tile_dp;
        k0 = 0;
        k1 = p.num_kb;
        slot = -1;
        tile_dp += gridDim.x / CG;
        return tile < p.dp_tiles;
    }
};

__device__ __forceinline__ void tile_coords(int tile, const Params& p, int bm, int bn, int& m0, int& n0) {
    const int per_group = p.group_m * p.num_n;
    const int g = tile / per_group;
    const int r = tile - g * per_group;
    const int gm0 = g * p.group_m;
    const int gsize = min(p.group_m, p.num_m - gm0);
    const int nb = r / gsize;
    m0 = (gm0 + (r - nb * gsize)) * bm;
    n0 = nb * bn;
}

template <int FMT, int GROUP>
__device__ __forceinline__ void umma_fp4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa, uint32_t sfb,
                                         uint32_t acc) {
    if constexpr (FMT == SQ_NVFP4 && GROUP == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb));
    else if constexpr (FMT == SQ_NVFP4)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4nvf4.block_scale.block16 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb));
    else if constexpr (GROUP == 1)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb));
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::mxf4.block_scale.block32 [%0], %1, %2, %3, [%5], [%6], p;\n\t}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc), "r"(sfa), "r"(sfb));
}

// N words per lane (one of 32 lanes) to N columns of tensor memory.
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t* r) {
    static_assert(N == 8 || N == 16, "columns per store");
    if constexpr (N == 8)
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]),
                     "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    else
        asm volatile(
            "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
                taddr),
            "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
            "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
            : "memory");
}

template <int OUT>
__device__ __forceinline__ uint32_t pack2(float a, float b) {
    if constexpr (OUT == kOutBF16) {
        __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    } else {
        __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<uint32_t*>(&h);
    }
}

// One 32-column chunk of one warp's 32 rows: scale, add the bias, round, stage
// in shared memory and write out (by TMA store, or whole 64-byte row segments).
template <int OUT>
__device__ __forceinline__ void epi_chunk(const Params& p, const uint32_t* r, int cw, int col0, int row0, float rx,
                                          const float* rw_w, const float* bias_w, uint8_t* stg, int lane,
                                          const CUtensorMap* tmap_y) {
    float y[32];
    const float4* rw4 = reinterpret_cast<const float4*>(rw_w + cw);
    const uint64_t rx2 = pk2(rx, rx);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const float4 w = rw4[e];
        const uint64_t d01 = mul2(rx2, pk2(w.x, w.y)), d23 = mul2(rx2, pk2(w.z, w.w));
        upk2(mul2(pk2(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1])), d01), y[4 * e], y[4 * e + 1]);
        upk2(mul2(pk2(__uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3])), d23), y[4 * e + 2], y[4 * e + 3]);
    }
    if (p.bias) {
        const float4* b4 = reinterpret_cast<const float4*>(bias_w + cw);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const float4 b = b4[e];
            y[4 * e + 0] = __fadd_rn(y[4 * e + 0], b.x);
            y[4 * e + 1] = __fadd_rn(y[4 * e + 1], b.y);
            y[4 * e + 2] = __fadd_rn(y[4 * e + 2], b.z);
            y[4 * e + 3] = __fadd_rn(y[4 * e + 3], b.w);
        }
    }
    if constexpr (OUT != kOutF32) {
        if (p.tma_store) {
            if (lane == 0) bulk_wait_read_all();
            __syncwarp();
            uint8_t* rowp = stg + lane * 64;
            const int sw = (lane >> 1) & 3;
#pragma unroll
            for (int e = 0; e < 4; ++e)
                *reinterpret_cast<uint4*>(rowp + ((e ^ sw) << 4)) =
                    make_uint4(pack2<OUT>(y[8 * e], y[8 * e + 1]), pack2<OUT>(y[8 * e + 2], y[8 * e + 3]),
                               pack2<OUT>(y[8 * e + 4], y[8 * e + 5]), pack2<OUT>(y[8 * e + 6], y[8 * e + 7]));
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (lane == 0) tma_store_3d(tmap_y, smem_u32(stg), col0, row0, 0);
            return;
        }
    }
    constexpr int HALVES = OUT == kOutF32 ? 2 : 1;
    constexpr int EB = OUT == kOutF32 ? 4 : 2, EPV = 16 / EB;  // bytes per element, elements per 16 bytes
#pragma unroll
    for (int hh = 0; hh < HALVES; ++hh) {
        uint4* dst = reinterpret_cast<uint4*>(stg + lane * kStgRow);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if constexpr (OUT == kOutF32)
                dst[e] = make_uint4(__float_as_uint(y[16 * hh + 4 * e]), __float_as_uint(y[16 * hh + 4 * e + 1]),
                                    __float_as_uint(y[16 * hh + 4 * e + 2]), __float_as_uint(y[16 * hh + 4 * e + 3]));
            else
                dst[e] = make_uint4(pack2<OUT>(y[8 * e], y[8 * e + 1]), pack2<OUT>(y[8 * e + 2], y[8 * e + 3]),
                                    pack2<OUT>(y[8 * e + 4], y[8 * e + 5]), pack2<OUT>(y[8 * e + 6], y[8 * e + 7]));
        }
        __syncwarp();
        if (p.vec_store) {
            const int part = lane & 3;
#pragma unroll
            for (int it = 0; it < 4; ++it) {
                const int rr = it * 8 + (lane >> 2);
                const int64_t grow = (int64_t)row0 + rr;
                const int col = col0 + 16 * hh + part * EPV;
                const uint4 v = *reinterpret_cast<const uint4*>(stg + rr * kStgRow + part * 16);
                if (grow < p.M && col < p.N) {
                    uint8_t* out = static_cast<uint8_t*>(p.Y) + (grow * p.ldy + col) * EB;
                    if (col + EPV <= p.N) {
                        *reinterpret_cast<uint4*>(out) = v;
                    } else {
                        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int e = 0; e < EPV; ++e)
                            if (col + e < p.N) {
                                if constexpr (OUT == kOutF32) reinterpret_cast<uint32_t*>(out)[e] = w[e];
                                else reinterpret_cast<uint16_t*>(out)[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                            }
                    }
                }
            }
        } else {
            // rows that start anywhere: an element a lane, neighbours together
            constexpr int W = 64 / EB;      // elements of a staged row
            constexpr int RPI = 32 / W;     // rows a store
            const int cc = lane % W;
            const int col = col0 + 16 * hh + cc;
#pragma unroll 4
            for (int rr = lane / W; rr < 32; rr += RPI) {
                const int64_t grow = (int64_t)row0 + rr;
                if (grow < p.M && col < p.N) {
                    if constexpr (OUT == kOutF32)
                        static_cast<uint32_t*>(p.Y)[grow * p.ldy + col] =
                            *reinterpret_cast<const uint32_t*>(stg + rr * kStgRow + cc * 4);
                    else
                        static_cast<uint16_t*>(p.Y)[grow * p.ldy + col] =
                            *reinterpret_cast<const uint16_t*>(stg + rr * kStgRow + cc * 2);
                }
            }
        }
        __syncwarp();
    }
}

template <int FMT, int OUT, bool SK>
__global__ void __launch_bounds__(kThreads, 1)
gemm_fp4_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                const __grid_constant__ CUtensorMap tmap_sa, const __grid_constant__ CUtensorMap tmap_sb,
                const __grid_constant__ CUtensorMap tmap_y, const Params p) {
    using C = Cfg<FMT>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + C::BAR_OFF;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto tfull_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + a); };
    auto tempty_bar = [&](int a) { return bar0 + 8u * (2 * STAGES + 2 + a); };
    const uint32_t drain_bar = bar0 + 8u * (2 * STAGES + 4);
    auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + 5 + s); };
    auto sready_bar = [&](int s) { return bar0 + 8u * (3 * STAGES + 5 + s); };
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            mbar_init(sfull_bar(s), 1);
            mbar_init(sready_bar(s), kScaleWarps * CG);
        }
        for (int a = 0; a < 2; ++a) {
            mbar_init(tfull_bar(a), 1);
            mbar_init(tempty_bar(a), kEpiWarps * CG);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_holder)), "r"(C::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    if (warp == 0 && lane == 0) {
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_a)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_b)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_sa)) : "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap_sb)) : "memory");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_holder;
    pdl_wait();
    pdl_trigger();

    if (SK && blockIdx.x == 0 && threadIdx.x == 0) p.status[3] = p.sk_cnt_bytes;
    Segments<SK> seg(p);
    int tile, k0, k1, slot;
    if (warp == 0) {
        if (lane == 0) {
            // ---------------------------------------------------- TMA producer
            int stage = 0;
            uint32_t phase = 0, issued = 0, issued_phase = 0;
            bool ok = true;
            while (ok && seg.next(p, tile, k0, k1, slot)) {
                int m0, n0;
                tile_coords(tile, p, BM * CG, BN, m0, n0);
                const int gn = n0 / 128;
                m0 += (int)rank * BM;
                n0 += (int)rank * (BN / CG);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!wait_fast(empty_bar(stage), phase ^ 1u, abort_flag, p.status, 0x8E1)) {
                        ok = false;
                        break;
                    }
                    const uint32_t fb = map_to_rank(full_bar(stage), 0);
                    if (rank == 0) mbar_expect_tx(full_bar(stage), CG * (C::A_BYTES + C::B_BYTES));
                    mbar_expect_tx(sfull_bar(stage), C::SA_BYTES + C::SB_BYTES);
                    tma_load_3d<CG>(sbase + C::A_OFF + stage * C::A_BYTES, &tmap_a, fb, kb * (BK / 2), m0, 0);
                    tma_load_3d<CG>(sbase + C::B_OFF + stage * C::B_BYTES, &tmap_b, fb, kb * (BK / 2), n0, 0);
                    // the scales count on this CTA's own barrier: its scale warps wait for them
                    tma_load_3d<1>(sbase + C::SA_OFF + stage * C::SA_BYTES, &tmap_sa, sfull_bar(stage),
                                   kb * (int)(C::SA_BYTES / 8), m0 / 128, 0);
                    tma_load_3d<1>(sbase + C::SB_OFF + stage * C::SB_BYTES, &tmap_sb, sfull_bar(stage),
                                   kb * (int)(C::SA_BYTES / 8), gn, 0);
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
            }
            if (!ok)
                for (int s = 0; s < STAGES; ++s)
                    if (issued >> s & 1u) {
                        if (rank == 0) wait_drain(full_bar(s), issued_phase >> s & 1u);
                        wait_drain(sfull_bar(s), issued_phase >> s & 1u);
                    }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ---------------------------------------------------- MMA issuer
            int stage = 0, local = 0;
            uint32_t phase = 0, set = 0;
            bool ok = true;
            for (; ok && seg.next(p, tile, k0, k1, slot); ++local) {
                const int acc = local & 1;
                // the previous tile's shared columns (and all of the tile before it)
                // have been read
                const int prev = local - 1;
                if (prev >= 0 &&
                    !wait_fast(tempty_bar(prev & 1), (uint32_t)(prev >> 1) & 1u, abort_flag, p.status, 0x8E2)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + (acc ? C::ACC1 : 0u);
                for (int kb = k0; kb < k1; ++kb) {
                    if (!wait_fast(full_bar(stage), phase, abort_flag, p.status, 0x8E3) ||
                        !wait_fast(sready_bar(stage), phase, abort_flag, p.status, 0x8E5)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t a_addr = sbase + C::A_OFF + stage * C::A_BYTES;
                    const uint32_t b_addr = sbase + C::B_OFF + stage * C::B_BYTES;
                    const uint32_t sfb = tmem_base + C::SF_COL + set * C::SET_COLS, sfa = sfb + C::SB_COLS;
                    set ^= 1u;
                    // (codes past K are zero, but so may be all of an MMA's: skip those)
                    const int steps = min(BK / UMMA_K, (p.K - kb * BK + UMMA_K - 1) / UMMA_K);
#pragma unroll
                    for (int k = 0; k < BK / UMMA_K; ++k) {
                        if (k >= steps) break;
                        const int c = FMT == SQ_NVFP4 ? k : k >> 1;       // scale tile of this MMA
                        const int sf = FMT == SQ_NVFP4 ? 0 : (k & 1) * 2;  // first byte of its words
                        umma_fp4<FMT, CG>(d_tmem, sdesc(a_addr + k * (UMMA_K / 2)), sdesc(b_addr + k * (UMMA_K / 2)),
                                          C::idesc(sf), sfa + c * 4, sfb + c * C::NG * 4, (kb != k0 || k != 0) ? 1u : 0u);
                    }
                    umma_commit<CG>(empty_bar(stage));
                    if (++stage == STAGES) stage = 0, phase ^= 1u;
                }
                if (!ok) break;
                umma_commit<CG>(tfull_bar(acc));
            }
            umma_commit<CG>(drain_bar, 1);
            wait_drain(drain_bar, 0);
        }
    } else if (warp >= 2 + kEpiWarps) {
        // -------------------------------------------------- scale warps
        // Each stage's scales, shared to tensor memory: a scale tile is four
        // words per lane, the same in every lane quarter.
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        int stage = 0, before = -2;  // `before`: the stage two stages ago, whose MMAs read this stage's set
        uint32_t phase = 0, before_phase = 0, set = 0;
        bool ok = true;
        while (ok && seg.next(p, tile, k0, k1, slot)) {
            for (int kb = k0; kb < k1; ++kb) {
                ok = wait_fast(sfull_bar(stage), phase, abort_flag, p.status, 0x8E6);
                if (ok && before >= 0) ok = wait_fast(empty_bar(before), before_phase, abort_flag, p.status, 0x8E7);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                tc_fence_after();
                uint32_t r[C::SET_COLS];
                const uint4* sb = reinterpret_cast<const uint4*>(smem + C::SB_OFF + stage * C::SB_BYTES) + lane;
                const uint4* sa = reinterpret_cast<const uint4*>(smem + C::SA_OFF + stage * C::SA_BYTES) + lane;
#pragma unroll
                for (int c = 0; c < C::CHUNKS; ++c) {
#pragma unroll
                    for (int g = 0; g < C::NG; ++g)
                        *reinterpret_cast<uint4*>(r + (c * C::NG + g) * 4) = sb[(g * C::CHUNKS + c) * 32];
                    *reinterpret_cast<uint4*>(r + C::SB_COLS + c * 4) = sa[c * 32];
                }
                const uint32_t to = tmem_base + quarter + C::SF_COL + set * C::SET_COLS;
#pragma unroll
                for (uint32_t i = 0; i + 16 <= C::SET_COLS; i += 16) tmem_st<16>(to + i, r + i);
                if constexpr (C::SET_COLS % 16 == 8) tmem_st<8>(to + C::SET_COLS - 8, r + C::SET_COLS - 8);
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_remote(map_to_rank(sready_bar(stage), 0));
                set ^= 1u;
                if (++before == STAGES) before = 0, before_phase ^= 1u;
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
        }
    } else {
        // -------------------------------------------------------- epilogue
        const int q = warp & 3;
        const int half = (warp - 2) >> 2;
        constexpr int HC = BN / 2, NCH = HC / 32;
        float* rw_w = reinterpret_cast<float*>(smem + C::RW_OFF) + (warp - 2) * 2 * HC;
        float* bias_w = rw_w + HC;
        uint8_t* stg = smem + C::STG_OFF + (warp - 2) * kStgWarpBytes;
        auto release_acc = [&](int a) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(map_to_rank(tempty_bar(a), 0));
        };
        int local = 0;
        for (; seg.next(p, tile, k0, k1, slot); ++local) {
            int m0, n0;
            tile_coords(tile, p, BM * CG, BN, m0, n0);
            m0 += (int)rank * BM;
            const int c_base = n0 + half * HC;
            const int row0 = m0 + q * 32;
            const int64_t row = (int64_t)row0 + lane;
            const bool row_ok = row < p.M;
            float qv[HC / 32], bv[HC / 32], qxv = 1.0f;
#pragma unroll
            for (int i = 0; i < HC / 32; ++i) {
                const int col = c_base + lane + 32 * i;
                qv[i] = 1.0f;
                bv[i] = 0.0f;
                if (col < p.N) {
                    if (p.qs_w) qv[i] = p.qs_w[p.w_per_channel ? col : 0];
                    if (p.bias) bv[i] = p.bias[col];
                }
            }
            if (row_ok && p.qs_x) qxv = p.qs_x[p.x_per_token ? row : 0];
            __syncwarp();
#pragma unroll
            for (int i = 0; i < HC / 32; ++i) {
                rw_w[lane + 32 * i] = __frcp_rn(qv[i]);
                bias_w[lane + 32 * i] = bv[i];
            }
            __syncwarp();
            const int acc = local & 1;
            // a warp that reads no shared column hands the buffer back at once
            // (the tile before this one is read in full by now)
            const bool shares = half == 1 - acc;
            if (!shares) release_acc(acc);
            const bool ok = wait_fast(tfull_bar(acc), (uint32_t)(local >> 1) & 1u, abort_flag, p.status, 0x8E4);
            if (!__all_sync(0xffffffffu, ok)) break;
            tc_fence_after();
            const float rx = __frcp_rn(qxv);
            const uint32_t t_row =
                tmem_base + ((uint32_t)(q * 32) << 16) + (acc ? C::ACC1 : 0u) + (uint32_t)(half * HC);
            uint32_t r[32];
            // shared columns first: the upper half's last chunks of the first
            // accumulator, the lower half's first ones of the second
            const int turn = acc == 0 && half == 1 ? NCH - C::SHARED : 0;
            if constexpr (SK) {
                if (slot >= 0) {
                    // a piece: park the sums; the one that completes the tile's
                    // k-blocks adds every piece's in range order
                    const int wr = warp - 2;
                    constexpr int REGION = NCH * 8 * 32;  // float4 per warp
                    float4* parts = reinterpret_cast<float4*>(p.sk_part);
                    float4* mine = parts + ((int64_t)(blockIdx.x * 2 + slot) * kEpiWarps + wr) * REGION;
#pragma unroll 1
                    for (int i = 0; i < NCH; ++i) {
                        const int c = (i + turn) & (NCH - 1);
                        tmem_ld32(t_row + (uint32_t)(c * 32), r);
                        if (shares && i == C::SHARED - 1) release_acc(acc);
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            __stcg(mine + (c * 8 + e) * 32 + lane,
                                   make_float4(__uint_as_float(r[4 * e]), __uint_as_float(r[4 * e + 1]),
                                               __uint_as_float(r[4 * e + 2]), __uint_as_float(r[4 * e + 3])));
                    }
                    __threadfence();
                    __syncwarp();
                    const int u = tile - p.dp_tiles;
                    int before = 0;
                    int* cnt = p.sk_cnt + (u * CG + (int)rank) * kEpiWarps + wr;
                    if (lane == 0) before = atomicAdd(cnt, k1 - k0);
                    before = __shfl_sync(0xffffffffu, before, 0);
                    if (before + (k1 - k0) != p.num_kb) continue;
                    __threadfence();
                    if (lane == 0) *cnt = 0;  // ready for the next launch
                    const int x0 = u * p.num_kb;
                    const int c_lo = sk_owner(x0, p), c_hi = sk_owner(x0 + p.num_kb - 1, p);
#pragma unroll 1
                    for (int c = 0; c < NCH; ++c) {
                        if (row0 >= p.M || c_base + c * 32 >= p.N) break;
#pragma unroll
                        for (int e = 0; e < 32; ++e) r[e] = 0u;
#pragma unroll 1
                        for (int cc = c_lo; cc <= c_hi; ++cc) {
                            const int sl = sk_start(cc, p) >= x0 ? 0 : 1;
                            const float4* src =
                                parts + ((int64_t)((cc * CG + (int)rank) * 2 + sl) * kEpiWarps + wr) * REGION;
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const float4 v = __ldcg(src + (c * 8 + e) * 32 + lane);
                                r[4 * e] = __float_as_uint(__uint_as_float(r[4 * e]) + v.x);
                                r[4 * e + 1] = __float_as_uint(__uint_as_float(r[4 * e + 1]) + v.y);
                                r[4 * e + 2] = __float_as_uint(__uint_as_float(r[4 * e + 2]) + v.z);
                                r[4 * e + 3] = __float_as_uint(__uint_as_float(r[4 * e + 3]) + v.w);
                            }
                        }
                        epi_chunk<OUT>(p, r, c * 32, c_base + c * 32, row0, rx, rw_w, bias_w, stg, lane, &tmap_y);
                    }
                    continue;
                }
            }
#pragma unroll 1
            for (int i = 0; i < NCH; ++i) {
                const int c = (i + turn) & (NCH - 1);
                tmem_ld32(t_row + (uint32_t)(c * 32), r);
                if (shares && i == C::SHARED - 1) release_acc(acc);
                if (row0 < p.M && c_base + c * 32 < p.N)
                    epi_chunk<OUT>(p, r, c * 32, c_base + c * 32, row0, rx, rw_w, bias_w, stg, lane, &tmap_y);
            }
        }
        if (p.tma_store && lane == 0) bulk_wait_all();
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(C::TMEM_COLS));
    }
}

// ---------------------------------------------------------------- few tiles
// One 128 x 128 tile, or one part of its k-loop (the cluster holds the parts), per
// CTA. MB: rows of X that are loaded (the tensor core reads whatever is in the
// others; they only reach rows that are not written). Warp 0 loads, warp 1 issues
// the MMAs, warps 2..5 bring the scales to tensor memory and then the sums from
// there to shared memory; all six add the parts and write.
template <int FMT, int MB>
struct SCfg {
    static constexpr int CHUNKS = FMT == SQ_NVFP4 ? 4 : 2;
    static constexpr int STAGES = MB == 32 ? 4 : 3;
    // (an MMA reads 128 rows from its stage on: at MB = 32 those of later stages
    // and of the weight's, inside this block's memory)
    static constexpr uint32_t A_BYTES = MB * BK / 2;
    static constexpr uint32_t B_BYTES = 128 * BK / 2;
    static constexpr uint32_t S_BYTES = CHUNKS * kFp4TileBytes;  // of one operand
    static constexpr uint32_t TX = A_BYTES + B_BYTES;
    static constexpr uint32_t B_OFF = STAGES * A_BYTES;
    static constexpr uint32_t S_OFF = B_OFF + STAGES * B_BYTES;
    static constexpr uint32_t BAR_OFF = S_OFF + STAGES * 2 * S_BYTES;  // full[S], empty[S], sfull[S], sready[S], done
    static constexpr uint32_t MISC_OFF = BAR_OFF + (4 * STAGES + 1) * 8;
    static constexpr uint32_t RX_OFF = MISC_OFF + 16;  // 1 / qs_x of the rows
    static constexpr uint32_t SMEM_ALLOC = RX_OFF + MB * 4 + 1024;
    static constexpr int LDP = 132;  // floats per row of the sums (in the ring, once it is drained)
    static_assert(MB * LDP * 4 <= S_OFF && BM * BK / 2 <= STAGES * B_BYTES, "the sums and an MMA's reads fit in the ring");
    static_assert(2 * (SMEM_ALLOC + 1024) <= 233472, "two CTAs per SM");
    static constexpr uint32_t SET_COLS = 2 * CHUNKS * 4;
    static constexpr uint32_t SF_COL = 128, TMEM_COLS = 256;
    static_assert(SF_COL + 2 * SET_COLS <= TMEM_COLS, "tensor memory");
    static constexpr uint32_t idesc(int sf) { return idesc_fp4<FMT>(BM, 128, sf); }
};
constexpr int kSplitThreads = 6 * 32;

template <int FMT, int MB, int OUT>
__global__ void __launch_bounds__(kSplitThreads, 2)
gemm_fp4_split_kernel(const __grid_constant__ CUtensorMap tmap_a, const __grid_constant__ CUtensorMap tmap_b,
                      const __grid_constant__ CUtensorMap tmap_sa, const __grid_constant__ CUtensorMap tmap_sb,
                      const Params p, const int splits) {
    using C = SCfg<FMT, MB>;
    constexpr int STAGES = C::STAGES;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + C::BAR_OFF;
    auto full_bar = [&](int s) { return bar0 + 8u * s; };
    auto empty_bar = [&](int s) { return bar0 + 8u * (STAGES + s); };
    auto sfull_bar = [&](int s) { return bar0 + 8u * (2 * STAGES + s); };
    auto sready_bar = [&](int s) { return bar0 + 8u * (3 * STAGES + s); };
    const uint32_t done_bar = bar0 + 8u * (4 * STAGES);
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), 1);
            mbar_init(sfull_bar(s), 1);
            mbar_init(sready_bar(s), 4);
        }
        mbar_init(done_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_holder)),
                     "r"(C::TMEM_COLS));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    const int part = blockIdx.x % splits, tile = blockIdx.x / splits;
    const int nb = tile / p.num_m;
    const int m0 = (tile - nb * p.num_m) * BM, n0 = nb * 128;
    const int k0 = (int)((int64_t)part * p.num_kb / splits);
    const int k1 = (int)((int64_t)(part + 1) * p.num_kb / splits);
    const int rows = min(p.M - m0, MB);
    pdl_wait();
    pdl_trigger();
    // the scales and biases of the outputs this thread writes, fetched while the
    // k-loop runs: columns 4 l .. 4 l + 3 (lane l), or l, l + 32, .. where rows do
    // not start on 16-byte boundaries (a warp's stores then stay together)
    const int c0 = p.vec_store ? 4 * lane : lane, cs = p.vec_store ? 1 : 32;
    float rw[4], bias[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const int col = min(n0 + c0 + cs * e, p.N - 1);
        rw[e] = p.qs_w ? p.qs_w[p.w_per_channel ? col : 0] : 1.0f;
        bias[e] = p.bias ? p.bias[col] : 0.0f;
    }
    float* const rx_s = reinterpret_cast<float*>(smem + C::RX_OFF);
    if ((int)threadIdx.x < rows)
        rx_s[threadIdx.x] = p.qs_x ? __frcp_rn(p.qs_x[p.x_per_token ? m0 + (int)threadIdx.x : 0]) : 1.0f;
    if (warp == 0) {
        if (lane == 0) {
            int stage = 0, kb = k0;
            uint32_t phase = 0;
            for (; kb < k1; ++kb) {
                if (!wait_fast(empty_bar(stage), phase ^ 1u, abort_flag, p.status, 0x8F1)) break;
                mbar_expect_tx(full_bar(stage), C::TX);
                mbar_expect_tx(sfull_bar(stage), 2 * C::S_BYTES);
                tma_load_3d<1>(sbase + C::B_OFF + stage * C::B_BYTES, &tmap_b, full_bar(stage), kb * (BK / 2), n0, 0);
                tma_load_3d<1>(sbase + stage * C::A_BYTES, &tmap_a, full_bar(stage), kb * (BK / 2), m0, 0);
                const uint32_t sf = sbase + C::S_OFF + stage * 2 * C::S_BYTES;
                tma_load_3d<1>(sf, &tmap_sb, sfull_bar(stage), kb * (int)(C::S_BYTES / 8), n0 / 128, 0);
                tma_load_3d<1>(sf + C::S_BYTES, &tmap_sa, sfull_bar(stage), kb * (int)(C::S_BYTES / 8), m0 / 128, 0);
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
            // after an abort: the copies that are in flight land before the block leaves
            if (kb < k1)
                for (int i = max(k0, kb - STAGES); i < kb; ++i) {
                    wait_drain(full_bar((i - k0) % STAGES), (uint32_t)((i - k0) / STAGES) & 1u);
                    wait_drain(sfull_bar((i - k0) % STAGES), (uint32_t)((i - k0) / STAGES) & 1u);
                }
        }
    } else if (warp == 1) {
        if (lane == 0) {
            int stage = 0;
            uint32_t phase = 0, set = 0;
            for (int kb = k0; kb < k1; ++kb) {
                if (!wait_fast(full_bar(stage), phase, abort_flag, p.status, 0x8F2) ||
                    !wait_fast(sready_bar(stage), phase, abort_flag, p.status, 0x8F3))
                    break;
                tc_fence_after();
                const uint32_t a_addr = sbase + stage * C::A_BYTES, b_addr = sbase + C::B_OFF + stage * C::B_BYTES;
                const uint32_t sfb = tmem + C::SF_COL + set * C::SET_COLS, sfa = sfb + C::CHUNKS * 4;
                set ^= 1u;
                const int steps = min(BK / UMMA_K, (p.K - kb * BK + UMMA_K - 1) / UMMA_K);
#pragma unroll
                for (int k = 0; k < BK / UMMA_K; ++k) {
                    if (k >= steps) break;
                    const int c = FMT == SQ_NVFP4 ? k : k >> 1;
                    const int sf = FMT == SQ_NVFP4 ? 0 : (k & 1) * 2;
                    umma_fp4<FMT, 1>(tmem, sdesc(a_addr + k * (UMMA_K / 2)), sdesc(b_addr + k * (UMMA_K / 2)), C::idesc(sf),
                                     sfa + c * 4, sfb + c * 4, (kb != k0 || k != 0) ? 1u : 0u);
                }
                umma_commit<1>(empty_bar(stage));
                if (++stage == STAGES) stage = 0, phase ^= 1u;
            }
            umma_commit<1>(done_bar);
            wait_drain(done_bar, 0);  // (no MMA is in flight when tensor memory is freed)
        }
    } else {
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        int stage = 0, before = -2;
        uint32_t phase = 0, before_phase = 0, set = 0;
        bool ok = true;
        for (int kb = k0; kb < k1; ++kb) {
            ok = wait_fast(sfull_bar(stage), phase, abort_flag, p.status, 0x8F4);
            if (ok && before >= 0) ok = wait_fast(empty_bar(before), before_phase, abort_flag, p.status, 0x8F5);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            tc_fence_after();
            uint32_t r[C::SET_COLS];
            const uint4* sf = reinterpret_cast<const uint4*>(smem + C::S_OFF + stage * 2 * C::S_BYTES) + lane;
#pragma unroll
            for (int c = 0; c < 2 * C::CHUNKS; ++c) *reinterpret_cast<uint4*>(r + 4 * c) = sf[c * 32];
            const uint32_t to = tmem + quarter + C::SF_COL + set * C::SET_COLS;
#pragma unroll
            for (uint32_t i = 0; i < C::SET_COLS; i += 16) tmem_st<16>(to + i, r + i);
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(sready_bar(stage));
            set ^= 1u;
            if (++before == STAGES) before = 0, before_phase ^= 1u;
            if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        if (ok) ok = wait_fast(done_bar, 0, abort_flag, p.status, 0x8F6);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        // this warp's 32 rows to shared memory, over the drained ring
        const int row = (warp & 3) * 32 + lane;
        if (ok && (warp & 3) * 32 < rows) {
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {
                uint32_t r[32];
                tmem_ld32(tmem + quarter + c * 32, r);
                if (row < rows) {
                    uint4* to = reinterpret_cast<uint4*>(smem + (row * C::LDP + c * 32) * 4);
#pragma unroll
                    for (int e = 0; e < 8; ++e) to[e] = make_uint4(r[4 * e], r[4 * e + 1], r[4 * e + 2], r[4 * e + 3]);
                }
            }
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (splits > 1) cluster_sync_all();  // every part's sums are in its shared memory
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(C::TMEM_COLS));
    }
    // this part's share of the rows, a warp each
#pragma unroll
    for (int e = 0; e < 4; ++e) rw[e] = __frcp_rn(rw[e]);
    const int r1 = (int)((int64_t)(part + 1) * rows / splits);
#pragma unroll 2
    for (int row = (int)((int64_t)part * rows / splits) + warp; row < r1; row += kSplitThreads / 32) {
        const uint32_t at = sbase + (uint32_t)(row * C::LDP + c0) * 4;
        float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < splits; ++s) {
            float v[4];
            // (a lone CTA is rank 0 of a cluster of one)
            const uint32_t from = map_to_rank(at, (uint32_t)s);
            if (p.vec_store) {
                asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
                             : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
                             : "r"(from)
                             : "memory");
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v[e]) : "r"(from + 128u * e) : "memory");
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[e] += v[e];
        }
        const float rx = rx_s[row];
        float y[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            y[e] = __fmul_rn(acc[e], __fmul_rn(rx, rw[e]));
            if (p.bias) y[e] = __fadd_rn(y[e], bias[e]);
        }
        constexpr int EB = OUT == kOutF32 ? 4 : 2;
        uint8_t* out = static_cast<uint8_t*>(p.Y) + (((int64_t)m0 + row) * p.ldy + n0 + c0) * EB;
        uint32_t w[4];
        if constexpr (OUT == kOutF32) {
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(y[e]);
        } else {
            w[0] = pack2<OUT>(y[0], y[1]), w[1] = pack2<OUT>(y[2], y[3]);
        }
        if (p.vec_store && n0 + c0 + 4 <= p.N) {
            if constexpr (OUT == kOutF32) *reinterpret_cast<uint4*>(out) = make_uint4(w[0], w[1], w[2], w[3]);
            else *reinterpret_cast<uint2*>(out) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n0 + c0 + cs * e < p.N) {
                    if constexpr (OUT == kOutF32) *reinterpret_cast<uint32_t*>(out + 4 * cs * e) = w[e];
                    else *reinterpret_cast<uint16_t*>(out + 2 * cs * e) = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
                }
        }
    }
    if (splits > 1) cluster_sync_all();  // nobody leaves while its sums are read
}

// ---------------------------------------------------------------- host side
// Codes [rows, K / 2] bytes, box 128 bytes x box_rows, 128-byte swizzle.
bool make_map_codes(CUtensorMap* m, const uint8_t* base, int64_t rows, int64_t K, int box_rows) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)(K / 2), (cuuint64_t)rows, 1};
    cuuint64_t strides[2] = {(cuuint64_t)(K / 2), (cuuint64_t)(rows * K / 2)};
    cuuint32_t box[3] = {BK / 2, (cuuint32_t)box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<uint8_t*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Scale tiles as [row groups, tiles_k * 64] 8-byte words, box chunks * 64 x groups.
bool make_map_scales(CUtensorMap* m, const uint8_t* base, int64_t groups, int64_t tiles_k, int chunks, int box_groups) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)(tiles_k * 64), (cuuint64_t)groups, 1};
    cuuint64_t strides[2] = {(cuuint64_t)(tiles_k * kFp4TileBytes), (cuuint64_t)(groups * tiles_k * kFp4TileBytes)};
    cuuint32_t box[3] = {(cuuint32_t)(chunks * 64), (cuuint32_t)box_groups, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 3, const_cast<uint8_t*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Plan {
    bool pairs = false;
    int tiles = 0, splits = 1, grid = 0;
    int sk_tiles = 0;     // trailing pair tiles that are cut by k-blocks
    size_t sk_bytes = 0;  // their counters and parked sums
};

// Counters at a fixed place for every shape: one per warp region of the split
// tiles, of which there are fewer than pairs.
constexpr int kMaxSplitTiles = 128;
constexpr size_t kSkCntBytes = (size_t)kMaxSplitTiles * 2 * kEpiWarps * sizeof(int);
static_assert(kSkCntBytes % 256 == 0, "the parked sums start 256-byte aligned");

Plan plan_fp4(int64_t M, int64_t N, int64_t K) {
    Plan pl;
    const int sms = num_sms();
    const int64_t kb = (K + BK - 1) / BK;
    const int64_t ptiles = ((M + 255) / 256) * ((N + 255) / 256);
    const int64_t tiles = ((M + 127) / 128) * ((N + 127) / 128);
    // Pairs above 128 rows and 64 tiles. Measured on B200 (us, one tile or part
    // per CTA / pairs): 16 x 16384 x 4096 9.4 / 12.6, 1 x 28672 x 7168 23 / 40,
    // 128 x 4096 x 4096 8.6 / 11.9, 256 x 4096 x 4096 (64 tiles) 11.1 / 11.9,
    // 512 x 4096 x 4096 (128 tiles) 13.1 / 12.1, 256 x 12288 x 4096 (192) 17.1 / 12.6.
    if (M > 128 && tiles > 64) {
        pl.pairs = true;
        pl.tiles = (int)ptiles;
        const int64_t pairs = sms / 2;
        pl.grid = (int)(2 * (ptiles < pairs ? ptiles : pairs));
        // Split where the last wave would be at most three quarters full and the
        // waves under 95 % busy, for k-loops of 48 blocks or more, with eight or
        // more for every pair: parking and adding the pieces takes about 10 us.
        // Whole / split (us): 1024 x 7168 x 28672 (112 blocks) 106 / 92, 4096 x
        // 12288 x 12288 (48, where the two are even) 255 / 253, 1024 x 7168 x 7168 (28)
        // 31.6 / 33.8, 2048 x 4096 x 4096 (16) 21.4 / 31.2.
        const int64_t rem = ptiles % pairs, waves = (ptiles + pairs - 1) / pairs;
        if (ptiles > pairs && rem > 0 && 4 * rem <= 3 * pairs && 20 * ptiles < 19 * waves * pairs &&
            kb >= 48 && rem * kb >= 8 * pairs && rem * kb < (1ll << 31) && rem <= kMaxSplitTiles) {
            pl.sk_tiles = (int)rem;
            pl.sk_bytes = kSkCntBytes + (size_t)pl.grid * 2 * BM * 256 * sizeof(float);
        }
        return pl;
    }
    pl.tiles = (int)tiles;
    // The k-loop in two or four parts while all of them fit at once (two CTAs per
    // SM), in eight while they leave every CTA an SM of its own; two stages or
    // more each. 16 x 4096 x 4096 (32 tiles): 10.1 us whole, 8.0 in two parts,
    // 6.2 in four, 6.7 in eight; 16 x 12288 x 4096 (96 tiles): 10.4, 9.5, 13.4.
    for (int s = 2; s <= 8; s *= 2)
        if (tiles * s <= (s == 8 ? sms : 2 * sms) && kb >= 2 * s) pl.splits = s;
    pl.grid = (int)tiles * pl.splits;
    return pl;
}

struct Call {
    const uint8_t *Xq, *Xs, *Wq, *Ws;
    int64_t M, N, K;
    sq_dtype_t out_dt;
};

sq_status_t map_failed(const char* name) {
    return set_error(SQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", name);
}

template <int FMT, int OUT>
sq_status_t launch_pairs(const char* name, const Call& c, const Plan& pl, Params& p, cudaStream_t stream) {
    using C = Cfg<FMT>;
    const int64_t tk = fp4_tiles_k(FMT, c.K);
    CUtensorMap ta, tb, tsa, tsb, ty;
    memset(&ty, 0, sizeof(ty));
    if (!make_map_codes(&ta, c.Xq, c.M, c.K, BM) || !make_map_codes(&tb, c.Wq, c.N, c.K, BN / CG) ||
        !make_map_scales(&tsa, c.Xs, fp4_tiles_m(c.M), tk, C::CHUNKS, 1) ||
        !make_map_scales(&tsb, c.Ws, fp4_tiles_m(c.N), tk, C::CHUNKS, C::NG))
        return map_failed(name);
    if (OUT != kOutF32 && p.vec_store)
        p.tma_store = make_map_y(&ty, p.Y, c.M, c.N, p.ldy, 1, c.M * p.ldy, OUT == kOutBF16) ? 1 : 0;
    p.num_m = (int)((c.M + BM * CG - 1) / (BM * CG));
    p.num_n = (int)((c.N + BN - 1) / BN);
    // rows of X per raster group within about 48 MB of L2
    const int64_t per = (int64_t)BM * CG * c.K / 2;
    const int64_t g = (48ll << 20) / per;
    p.group_m = (int)(g < 1 ? 1 : g > p.num_m ? p.num_m : g);
    auto fn = p.sk_tiles > 0 ? gemm_fp4_kernel<FMT, OUT, true> : gemm_fp4_kernel<FMT, OUT, false>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_ALLOC) != cudaSuccess)
        return check_launch(name);
    launch_pdl_cluster(fn, dim3(pl.grid), dim3(kThreads), C::SMEM_ALLOC, stream, 2, ta, tb, tsa, tsb, ty, p);
    return check_launch(name);
}

template <int FMT, int MB, int OUT>
sq_status_t launch_split(const char* name, const Call& c, const Plan& pl, Params& p, cudaStream_t stream) {
    using C = SCfg<FMT, MB>;
    const int64_t tk = fp4_tiles_k(FMT, c.K);
    CUtensorMap ta, tb, tsa, tsb;
    if (!make_map_codes(&ta, c.Xq, c.M, c.K, MB) || !make_map_codes(&tb, c.Wq, c.N, c.K, 128) ||
        !make_map_scales(&tsa, c.Xs, fp4_tiles_m(c.M), tk, C::CHUNKS, 1) ||
        !make_map_scales(&tsb, c.Ws, fp4_tiles_m(c.N), tk, C::CHUNKS, 1))
        return map_failed(name);
    p.num_m = (int)((c.M + BM - 1) / BM);
    auto fn = gemm_fp4_split_kernel<FMT, MB, OUT>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_ALLOC) != cudaSuccess)
        return check_launch(name);
    if (pl.splits > 1)
        launch_pdl_cluster(fn, dim3(pl.grid), dim3(kSplitThreads), C::SMEM_ALLOC, stream, pl.splits, ta, tb, tsa, tsb, p,
                           pl.splits);
    else
        launch_pdl(fn, dim3(pl.grid), dim3(kSplitThreads), C::SMEM_ALLOC, stream, ta, tb, tsa, tsb, p, 1);
    return check_launch(name);
}

template <int FMT, int OUT>
sq_status_t launch_plan(const char* name, const Call& c, const Plan& pl, Params& p, cudaStream_t stream) {
    if (pl.pairs) return launch_pairs<FMT, OUT>(name, c, pl, p, stream);
    if (c.M <= 32) return launch_split<FMT, 32, OUT>(name, c, pl, p, stream);
    return launch_split<FMT, 128, OUT>(name, c, pl, p, stream);
}

template <int FMT>
sq_status_t launch_out(const char* name, const Call& c, const Plan& pl, Params& p, cudaStream_t stream) {
    if (c.out_dt == SQ_BF16) return launch_plan<FMT, kOutBF16>(name, c, pl, p, stream);
    if (c.out_dt == SQ_F16) return launch_plan<FMT, kOutF16>(name, c, pl, p, stream);
    return launch_plan<FMT, kOutF32>(name, c, pl, p, stream);
}

}  // namespace

size_t gemm_fp4_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (M <= 0 || N <= 0 || K <= 0) return kStatusBytes;
    return kStatusBytes + plan_fp4(M, N, K).sk_bytes;
}

}  // namespace sq

extern "C" sq_status_t sq_gemm_fp4(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws,
                                   sq_fp4_t fmt, int64_t M, int64_t N, int64_t K, const float* qs_x, int x_per_token,
                                   const float* qs_w, int w_per_channel, const float* bias, sq_dtype_t out_dt, void* Y,
                                   int64_t ldy, void* workspace, size_t ws_bytes, sq_stream_t stream) {
    const char* name = "sq_gemm_fp4";
    SQ_REQUIRE(fmt == SQ_NVFP4 || fmt == SQ_MXFP4, SQ_ERR_INVALID_ARG, "%s: bad format", name);
    SQ_REQUIRE(out_dt == SQ_F32 || out_dt == SQ_F16 || out_dt == SQ_BF16, SQ_ERR_INVALID_ARG,
               "%s: out dtype must be F32, F16 or BF16", name);
    SQ_REQUIRE(M >= 0 && N > 0 && K > 0 && ldy >= N, SQ_ERR_UNSUPPORTED_SHAPE, "%s: need N > 0, K > 0, ldy >= N", name);
    SQ_REQUIRE(K % 32 == 0, SQ_ERR_UNSUPPORTED_SHAPE, "%s: K must be a multiple of 32", name);
    SQ_REQUIRE(M < (1ll << 30) && N < (1ll << 30) && K < (1ll << 30) &&
                   ((M + 127) / 128) * ((N + 127) / 128) < (1ll << 31),
               SQ_ERR_UNSUPPORTED_SHAPE, "%s: M, N, K must be < 2^30 and the tiles < 2^31", name);
    if (M == 0) return SQ_OK;
    SQ_REQUIRE(Xq && Xs && Wq && Ws && Y, SQ_ERR_INVALID_ARG, "%s: null codes, block scales or Y", name);
    SQ_REQUIRE(sq::aligned16(Xq) && sq::aligned16(Xs) && sq::aligned16(Wq) && sq::aligned16(Ws), SQ_ERR_ALIGNMENT,
               "%s: codes and block scales must be 16-byte aligned", name);
    SQ_REQUIRE(workspace && ws_bytes >= sq::kStatusBytes, SQ_ERR_INVALID_ARG, "%s: needs a workspace of %zu bytes", name,
               sq::kStatusBytes);
    SQ_REQUIRE(sq::aligned16(workspace), SQ_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", name);
    const sq::Plan pl = sq::plan_fp4(M, N, K);
    const int eb = sq::dtype_bytes(out_dt);
    sq::Params p;
    memset(&p, 0, sizeof(p));
    p.M = (int)M;
    p.N = (int)N;
    p.K = (int)K;
    p.num_kb = (int)((K + sq::BK - 1) / sq::BK);
    p.vec_store = sq::aligned16(Y) && (ldy * eb) % 16 == 0;
    p.qs_x = qs_x;
    p.qs_w = qs_w;
    p.bias = bias;
    p.x_per_token = x_per_token;
    p.w_per_channel = w_per_channel;
    p.Y = Y;
    p.ldy = ldy;
    p.status = static_cast<int*>(workspace);
    // a workspace without room for the split runs whole tiles only
    p.sk_tiles = ws_bytes >= sq::kStatusBytes + pl.sk_bytes ? pl.sk_tiles : 0;
    p.dp_tiles = pl.tiles - p.sk_tiles;
    p.sk_iters = p.sk_tiles * p.num_kb;
    p.sk_units = pl.grid / 2;
    p.sk_cnt_bytes = (int)sq::kSkCntBytes;
    uint8_t* after = static_cast<uint8_t*>(workspace) + sq::kStatusBytes;
    p.sk_cnt = reinterpret_cast<int*>(after);
    p.sk_part = reinterpret_cast<float*>(after + sq::kSkCntBytes);
    const sq::Call c = {Xq, Xs, Wq, Ws, M, N, K, out_dt};
    cudaStream_t s = sq::as_cuda(stream);
    return fmt == SQ_NVFP4 ? sq::launch_out<SQ_NVFP4>(name, c, pl, p, s) : sq::launch_out<SQ_MXFP4>(name, c, pl, p, s);
}
