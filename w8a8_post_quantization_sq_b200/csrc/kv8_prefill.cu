// Attention over the paged int8 K/V cache for prompts: the sequences of a batch
// whose rows (new token x query head of a K/V head's group) are many.
//
// The same formula, scales and rounding as for single tokens (kv8_attention.cu):
// int8 codes as fp16, the K scale on the fp32 scores, the V scale in the
// softmax's exponent, P in fp16 below 2^8, a running maximum that moves only
// when a score passes it by 2^8. Here both products run on tcgen05 (kind::f16):
//   S = Q K^T   128 rows x 128 keys, both from shared memory
//   O += P V    P from tensor memory (it overwrites S's columns), V from shared
//               memory with the columns contiguous (MN-major), as it lies in
//               the cache
// A CTA (one per SM, persistent) takes 256 rows of one sequence and K/V head as
// two tiles; while one tile's scores are on the tensor core, the other's are
// exponentiated. Tensor memory: S (128 columns) and O (D) of both tiles, 512 at
// D = 128. Roles:
//   warps 0..3, 4..7   softmax of tile 0, 1: a thread per row; also loads Q,
//                      rescales O and writes Y
//   warps 8..11        int8 K and V tiles to fp16 tiles (128-byte swizzle): 128
//                      x D codes are converted once for 256 rows
//   warp 12            TMA of the int8 tiles, warp 13 the MMAs
// Items are (sequence, 256 rows, head), the rows with the most keys first.
// What bounds it: 128 x 128 scores take 512 cycles of the tensor core for each
// product at D = 128 and 1024 of the exponential unit, two tiles 2048 of either.
// Every wait is bounded (about 2 s), code 0x9E1 + role in the status word.
#include <climits>
#include <cstring>

#include "sq_internal.h"
#include "sq_kv8.cuh"
#include "sq_tc.cuh"

namespace sq {
namespace {

constexpr int kKeys = 128;
constexpr int kTileRows = 128;
constexpr int kItemRows = 2 * kTileRows;
constexpr int kRaw = 3, kF16 = 3;  // ring stages: int8 tiles, fp16 tiles
constexpr int kThreadsP = 14 * 32;

template <int D>
struct PCfg {
    static constexpr uint32_t HALF = kKeys * 128;           // 128 rows of 64 fp16
    static constexpr uint32_t TILE = D / 64 * HALF;         // 128 x D fp16
    static constexpr uint32_t RAW = kKeys * D;              // 128 x D int8
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t F_OFF = Q_OFF + 2 * TILE;
    static constexpr uint32_t R_OFF = F_OFF + kF16 * TILE;
    static constexpr uint32_t BAR_OFF = R_OFF + kRaw * RAW;
    // raw_full[3], raw_empty[3], f_full[3], f_empty[3], q_ready[2], s_full[2], p_full[2], o_full[2], drain
    static constexpr uint32_t NBAR = 2 * kRaw + 2 * kF16 + 9;
    static constexpr uint32_t MISC_OFF = BAR_OFF + NBAR * 8;  // tmem base, abort flag
    static constexpr uint32_t SMEM_ALLOC = MISC_OFF + 16 + 1024;
    static_assert(SMEM_ALLOC <= 232448, "over the 227 KB of shared memory a block may use");
    static constexpr uint32_t O_COL = 256;  // O of tile x at O_COL + x * D, S and P at x * 128
    // fp16 x fp16 -> fp32, M = 128: N = 128 keys, both K-major; N = D, V MN-major (bit 16)
    static constexpr uint32_t IDESC_S = (1u << 4) | ((uint32_t)(kKeys >> 3) << 17) | ((uint32_t)(kTileRows >> 4) << 24);
    static constexpr uint32_t IDESC_O =
        (1u << 4) | (1u << 16) | ((uint32_t)(D >> 3) << 17) | ((uint32_t)(kTileRows >> 4) << 24);
};

// Descriptor of an MN-major operand with 128-byte swizzle: 8 rows (of the
// summed axis) of 64 elements are 1024 bytes, the next 64 columns `lbo` bytes on.
__device__ __forceinline__ uint64_t sdesc_mn(uint32_t saddr, uint32_t lbo) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) |
           ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
__device__ __forceinline__ void umma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(acc));
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
        "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// The CTA's items in turn: item index -> sequence, head, rows, key tiles. Every
// warp walks them together (32 sequences a look).
struct Items {
    int64_t next_item, before, total_in;  // items before the sequences of `base`, and in them
    int base;
    Seq s;
    int b, h, r0;
    int tiles[2];  // key tiles of each row tile
    int vis;       // keys that the item's last row sees
    int64_t inc, mine;

    __device__ __forceinline__ void look(const AttnArgs& a, int lane) {
        mine = 0;
        if (base + lane < a.B) {
            const Seq t = seq_of<kItemRows, kKeys>(a, base + lane);
            if ((int64_t)t.n * a.G > a.row_limit) mine = (int64_t)t.rt * a.Hkv;
        }
        inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += up;
        }
        total_in = __shfl_sync(0xffffffffu, inc, 31);
    }
    __device__ __forceinline__ void init(const AttnArgs& a, int lane) {
        next_item = blockIdx.x;
        before = 0;
        base = 0;
        look(a, lane);
    }
    __device__ __forceinline__ bool next(const AttnArgs& a, int lane) {
        while (next_item >= before + total_in) {
            before += total_in;
            base += 32;
            if (base >= a.B) return false;
            look(a, lane);
        }
        const int l = __ffs(__ballot_sync(0xffffffffu, before + inc > next_item)) - 1;
        b = base + l;
        const int64_t first = before + __shfl_sync(0xffffffffu, inc - mine, l);
        s = seq_of<kItemRows, kKeys>(a, b);
        const int idx = (int)(next_item - first);
        const int back = idx / a.Hkv;
        h = idx - back * a.Hkv;
        r0 = (s.rt - 1 - back) * kItemRows;
        const int rows = s.n * a.G;
        vis = seen_by(a, s, min(r0 + kItemRows, rows) - 1);
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            const int f = r0 + x * kTileRows;
            tiles[x] = f < rows ? (seen_by(a, s, min(f + kTileRows, rows) - 1) + kKeys - 1) / kKeys : 0;
        }
        next_item += gridDim.x;
        return true;
    }
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreadsP, 1)
kv8_prefill_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                   const AttnArgs a) {
    using C = PCfg<D>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t bar0 = sbase + C::BAR_OFF;
    auto raw_full = [&](int s) { return bar0 + 8u * s; };
    auto raw_empty = [&](int s) { return bar0 + 8u * (kRaw + s); };
    auto f_full = [&](int s) { return bar0 + 8u * (2 * kRaw + s); };
    auto f_empty = [&](int s) { return bar0 + 8u * (2 * kRaw + kF16 + s); };
    const uint32_t bar1 = bar0 + 8u * (2 * kRaw + 2 * kF16);
    auto q_ready = [&](int x) { return bar1 + 8u * x; };
    auto s_full = [&](int x) { return bar1 + 8u * (2 + x); };
    auto p_full = [&](int x) { return bar1 + 8u * (4 + x); };
    auto o_full = [&](int x) { return bar1 + 8u * (6 + x); };
    const uint32_t drain_bar = bar1 + 8u * 8;
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(smem + C::MISC_OFF);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kRaw; ++s) {
            mbar_init(raw_full(s), 1);
            mbar_init(raw_empty(s), 4);
        }
        for (int s = 0; s < kF16; ++s) {
            mbar_init(f_full(s), 4);
            mbar_init(f_empty(s), 1);
        }
        for (int x = 0; x < 2; ++x) {
            mbar_init(q_ready(x), 4);
            mbar_init(s_full(x), 1);
            mbar_init(p_full(x), 4);
            mbar_init(o_full(x), 1);
        }
        mbar_init(drain_bar, 1);
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 13) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_holder)));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_holder;
    pdl_wait();
    pdl_trigger();
    Items it;
    it.init(a, lane);
    bool ok = true;
    if (warp < 8) {
        // ------------------------------------------------------ softmax
        const int x = warp >> 2;
        const int row = (warp & 3) * 32 + lane;  // row of the tile, and lane of tensor memory
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + quarter + (uint32_t)(x * 128), t_o = tmem + quarter + C::O_COL + (uint32_t)(x * D);
        uint32_t s_phase = 0, o_phase = 0;
        while (ok && it.next(a, lane)) {
            const int rows = it.s.n * a.G;
            const int r = it.r0 + x * kTileRows + row;
            const bool live = r < rows;
            const int i = live ? r / a.G : 0;
            const int64_t at = (it.s.lo + i) * 1;  // token
            const int64_t head = (int64_t)(it.h * a.G + (live ? r - i * a.G : 0)) * D;
            // Q: scaled by a power of two per row to [1, 2), the score scale's
            // sign in it, as fp16 to the swizzled tile
            float crow;
            {
                const T* q = static_cast<const T*>(a.Q) + at * a.ldq + head;
                uint4 w[D / 8];
                uint32_t m2 = 0;
#pragma unroll
                for (int e = 0; e < D / 8; ++e) {
                    w[e] = live ? ldg_nc_v4(q + 8 * e) : make_uint4(0, 0, 0, 0);
                    m2 = __vmaxu2(m2, __vmaxu2(w[e].x & 0x7fff7fffu, w[e].y & 0x7fff7fffu));
                    m2 = __vmaxu2(m2, __vmaxu2(w[e].z & 0x7fff7fffu, w[e].w & 0x7fff7fffu));
                }
                float top[8];
                unpack<T>(make_uint4(max(m2 & 0xffffu, m2 >> 16), 0, 0, 0), top);
                const uint32_t field = min(max(__float_as_uint(top[0]) >> 23, 1u), 253u);
                const float down = copysignf(__uint_as_float((254u - field) << 23), a.scale);
                crow = fabsf(a.scale) * kLog2e * __uint_as_float(field << 23);
                uint8_t* base = smem + C::Q_OFF + x * C::TILE + row * 128;
#pragma unroll
                for (int e = 0; e < D / 8; ++e) {
                    float v[8];
                    unpack<T>(w[e], v);
                    *reinterpret_cast<uint4*>(base + (e >> 3) * C::HALF + (((e & 7) ^ (row & 7)) << 4)) =
                        make_uint4(pack_half2(v[0] * down, v[1] * down), pack_half2(v[2] * down, v[3] * down),
                                   pack_half2(v[4] * down, v[5] * down), pack_half2(v[6] * down, v[7] * down));
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready(x));
            // (rows past the sequence's end are computed unmasked and not written)
            const int vis = live ? seen_by(a, it.s, r) : INT_MAX;
            const int32_t* table = a.table + (int64_t)it.b * a.ldb;
            // lane e < 8 looks after the scales of keys 16 e .. of a tile, one tile ahead
            auto scales_of = [&](int j) {
                float kq = __uint_as_float(0x7fffffffu), vq = kq;
                const int key = j * kKeys + (lane & 7) * 16;
                if (key < it.vis) {
                    const int64_t blk = __ldg(table + key / a.block);
                    if (blk >= 0 && blk < a.num_blocks) {
                        kq = __ldg(a.kqs + blk * a.Hkv + it.h);
                        vq = __ldg(a.vqs + blk * a.Hkv + it.h);
                    }
                }
                return make_float2(kq, vq);
            };
            const int tiles = it.tiles[x];
            float m = -INFINITY, l = 0.0f;
            float2 next = scales_of(0);
            for (int j = 0; j < tiles; ++j) {
                const float my_k = __frcp_rn(next.x), my_v = next.y, my_lv = -__log2f(next.y);
                if (j + 1 < tiles) next = scales_of(j + 1);
                ok = wait_fast(s_full(x), s_phase, abort_flag, a.status, 0x9E1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                s_phase ^= 1u;
                tc_fence_after();
                const int key0 = j * kKeys;
                const bool masked = __any_sync(0xffffffffu, key0 + kKeys > vis);
                float tm = -INFINITY;
                uint32_t s[32];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld32(t_s + c * 32, s);
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        const float f = crow * __shfl_sync(0xffffffffu, my_k, 2 * c + hb);
                        const float lv = __shfl_sync(0xffffffffu, my_lv, 2 * c + hb);
                        float q = -INFINITY;
                        if (!masked) {
#pragma unroll
                            for (int e = 0; e < 16; ++e) q = fmaxf(q, __uint_as_float(s[16 * hb + e]));
                            tm = fmaxf(tm, fmaf(q, f, lv));
                        } else {
#pragma unroll
                            for (int e = 0; e < 16; ++e)
                                if (key0 + 32 * c + 16 * hb + e < vis)
                                    q = fmaxf(q, fmaf(__uint_as_float(s[16 * hb + e]), f, lv));
                            tm = fmaxf(tm, q);
                        }
                    }
                }
                if (__any_sync(0xffffffffu, tm > m + kSlack)) {
                    const float to = tm > m + kSlack ? tm : m;
                    const float f = to == -INFINITY ? 1.0f : ex2(m - to);
                    m = to;
                    l *= f;
                    if (j > 0) {
                        // (the scores' barrier says that the product before them is complete)
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            tmem_ld32(t_o + c * 32, s);
#pragma unroll
                            for (int e = 0; e < 32; ++e) s[e] = __float_as_uint(__uint_as_float(s[e]) * f);
                            tmem_st16(t_o + c * 32, s);
                            tmem_st16(t_o + c * 32 + 16, s + 16);
                        }
                    }
                }
                const float mu = m == -INFINITY ? 0.0f : m;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    tmem_ld32(t_s + c * 32, s);
                    uint32_t p[16];
#pragma unroll
                    for (int hb = 0; hb < 2; ++hb) {
                        const float f = crow * __shfl_sync(0xffffffffu, my_k, 2 * c + hb);
                        const float lv = __shfl_sync(0xffffffffu, my_lv, 2 * c + hb) - mu;
                        const float vq = __shfl_sync(0xffffffffu, my_v, 2 * c + hb);
                        float sum = 0.0f;
#pragma unroll
                        for (int e = 0; e < 16; e += 2) {
                            float p0 = ex2(fmaf(__uint_as_float(s[16 * hb + e]), f, lv));
                            float p1 = ex2(fmaf(__uint_as_float(s[16 * hb + e + 1]), f, lv));
                            if (masked) {
                                if (key0 + 32 * c + 16 * hb + e >= vis) p0 = 0.0f;
                                if (key0 + 32 * c + 16 * hb + e + 1 >= vis) p1 = 0.0f;
                            }
                            sum += p0 + p1;
                            p[8 * hb + e / 2] = pack_half2(p0, p1);
                        }
                        // (a row that sees none of these keys takes nothing from their scale)
                        if (!masked || key0 + 32 * c + 16 * hb < vis) l = fmaf(sum, vq, l);
                    }
                    tmem_st16(t_s + c * 16, p);
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(x));
            }
            if (!ok) break;
            const float inv = (m == -INFINITY && l == 0.0f) ? 0.0f : __frcp_rn(l);
            T* y = static_cast<T*>(a.Y) + at * a.ldy + head;
            if (tiles > 0) {
                ok = wait_fast(o_full(x), o_phase, abort_flag, a.status, 0x9E2);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                o_phase ^= 1u;
                tc_fence_after();
            }
#pragma unroll 1
            for (int c = 0; c < D / 32; ++c) {
                uint32_t s[32];
                if (tiles > 0) {
                    tmem_ld32(t_o + c * 32, s);
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e) s[e] = 0u;
                }
                if (live) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t p[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            p[e] = (uint32_t)to16<T>(__uint_as_float(s[8 * q + 2 * e]) * inv) |
                                   ((uint32_t)to16<T>(__uint_as_float(s[8 * q + 2 * e + 1]) * inv) << 16);
                        *reinterpret_cast<uint4*>(y + c * 32 + 8 * q) = make_uint4(p[0], p[1], p[2], p[3]);
                    }
                }
            }
        }
    } else if (warp < 12) {
        // ------------------------------------------------------ conversion
        const int t = threadIdx.x - 256;
        int rs = 0, fs = 0;
        uint32_t rp = 0, fp = 0;
        while (ok && it.next(a, lane)) {
            const int n = 2 * max(it.tiles[0], it.tiles[1]);
            for (int j = 0; ok && j < n; ++j) {
                ok = wait_fast(raw_full(rs), rp, abort_flag, a.status, 0x9E3) &&
                     wait_fast(f_empty(fs), fp ^ 1u, abort_flag, a.status, 0x9E4);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint8_t* src = smem + C::R_OFF + rs * C::RAW;
                uint8_t* dst = smem + C::F_OFF + fs * C::TILE;
                constexpr int UPR = D / 16;  // 16-code units per key
#pragma unroll
                for (int k = 0; k < kKeys * UPR / 128; ++k) {
                    const int unit = k * 128 + t;
                    const int key = unit / UPR, u = unit % UPR;
                    const uint4 w = *reinterpret_cast<const uint4*>(src + unit * 16);
                    uint32_t o[8];
                    const uint32_t in[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        o[2 * e] = half2_of(in[e], 0x4140);
                        o[2 * e + 1] = half2_of(in[e], 0x4342);
                    }
                    // 16-byte chunks 2 u, 2 u + 1 of the key's row, 8 to a half;
                    // at D = 128 units of the two halves store in opposite order, so that
                    // eight lanes cover all banks
                    uint8_t* row = dst + (u >> 2) * C::HALF + key * 128;
                    const int c0 = (2 * u) & 7, sw = key & 7;
                    const uint4 a0 = make_uint4(o[0], o[1], o[2], o[3]), a1 = make_uint4(o[4], o[5], o[6], o[7]);
                    const bool swap = D == 128 && u >= 4;
                    *reinterpret_cast<uint4*>(row + (((swap ? c0 + 1 : c0) ^ sw) << 4)) = swap ? a1 : a0;
                    *reinterpret_cast<uint4*>(row + (((swap ? c0 : c0 + 1) ^ sw) << 4)) = swap ? a0 : a1;
                }
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(f_full(fs));
                    mbar_arrive(raw_empty(rs));
                }
                if (++rs == kRaw) rs = 0, rp ^= 1u;
                if (++fs == kF16) fs = 0, fp ^= 1u;
            }
        }
    } else if (warp == 12) {
        // ------------------------------------------------------ TMA
        int rs = 0;
        uint32_t rp = 0, issued = 0, issued_phase = 0;
        const int box = a.box, per_box = box / 16;
        while (ok && it.next(a, lane)) {
            const int n = max(it.tiles[0], it.tiles[1]);
            const int32_t* table = a.table + (int64_t)it.b * a.ldb;
            // lane e looks after part e % 8 (16 keys) of tile j0 + e / 8
            auto block_of = [&](int j0) {
                const int key = j0 * kKeys + lane * 16;
                const int blk = key < it.vis ? __ldg(table + key / a.block) : -1;
                return blk >= 0 && blk < a.num_blocks ? blk : -1;
            };
            int next = block_of(0);
            for (int j0 = 0; ok && j0 < n; j0 += 4) {
                const int blk = next;
                if (j0 + 4 < n) next = block_of(j0 + 4);
                const int y = it.h * a.block + ((j0 * kKeys + lane * 16) & (a.block - 1));
                for (int j = j0; ok && j < min(j0 + 4, n); ++j) {
                    const int part = lane - (j - j0) * 8;
                    const bool copy = part >= 0 && part < 8 && blk >= 0 && part % per_box == 0;
                    const int boxes = __popc(__ballot_sync(0xffffffffu, copy));
#pragma unroll
                    for (int v = 0; v < 2; ++v) {
                        ok = wait_fast(raw_empty(rs), rp ^ 1u, abort_flag, a.status, 0x9E5);
                        ok = __all_sync(0xffffffffu, ok);
                        if (!ok) break;
                        if (lane == 0) mbar_expect_tx(raw_full(rs), (uint32_t)(boxes * box * D));
                        __syncwarp();
                        if (copy)
                            tma_load_3d<1>(sbase + C::R_OFF + rs * C::RAW + part * 16 * D, v ? &map_v : &map_k,
                                           raw_full(rs), 0, y, blk);
                        issued |= 1u << rs;
                        issued_phase = (issued_phase & ~(1u << rs)) | (rp << rs);
                        if (++rs == kRaw) rs = 0, rp ^= 1u;
                    }
                }
            }
        }
        if (!ok)
            for (int s = 0; s < kRaw; ++s)
                if (issued >> s & 1u) wait_drain(raw_full(s), issued_phase >> s & 1u);
    } else {
        // ------------------------------------------------------ MMA
        int fs = 0;  // stage of the next fp16 tile in the order K0 V0 K1 V1 ...
        uint32_t fp = 0, q_phase = 0, p_phase[2] = {0, 0};
        while (ok && it.next(a, lane)) {
            if (lane == 0) {
                const int n0 = it.tiles[0], n1 = it.tiles[1], n = max(n0, n1);
                auto take = [&](int& stage) {  // waits for the next fp16 tile
                    stage = fs;
                    const bool got = wait_fast(f_full(fs), fp, abort_flag, a.status, 0x9E6);
                    if (++fs == kF16) fs = 0, fp ^= 1u;
                    tc_fence_after();
                    return got;
                };
                auto score = [&](int x, int st) {
                    const uint32_t qa = sbase + C::Q_OFF + x * C::TILE, kb = sbase + C::F_OFF + st * C::TILE;
#pragma unroll
                    for (int k = 0; k < D / 16; ++k) {
                        const uint32_t off = (k >> 2) * C::HALF + (k & 3) * 32;
                        umma_ss(tmem + x * 128, sdesc(qa + off), sdesc(kb + off), C::IDESC_S, k != 0);
                    }
                    umma_commit<1>(s_full(x));
                };
                ok = wait_fast(q_ready(0), q_phase, abort_flag, a.status, 0x9E7) &&
                     wait_fast(q_ready(1), q_phase, abort_flag, a.status, 0x9E7);
                tc_fence_after();
                int ks = 0, vs = 0;
                if (ok && n > 0) {
                    ok = take(ks);
                    if (ok) {
                        if (n0 > 0) score(0, ks);
                        if (n1 > 0) score(1, ks);
                        umma_commit<1>(f_empty(ks));
                    }
                }
                for (int j = 0; ok && j < n; ++j) {
                    ok = take(vs);
                    const bool more = j + 1 < n;
                    bool have_k = false;
                    for (int x = 0; ok && x < 2; ++x) {
                        const int nx = x ? n1 : n0;
                        if (j < nx) {
                            ok = wait_fast(p_full(x), p_phase[x], abort_flag, a.status, 0x9E8);
                            if (!ok) break;
                            p_phase[x] ^= 1u;
                            tc_fence_after();
                            const uint32_t vb = sbase + C::F_OFF + vs * C::TILE;
#pragma unroll
                            for (int k = 0; k < kKeys / 16; ++k)
                                umma_ts(tmem + C::O_COL + x * D, tmem + x * 128 + k * 8,
                                        sdesc_mn(vb + k * 16 * 128, C::HALF), C::IDESC_O, (j != 0 || k != 0) ? 1u : 0u);
                            if (j + 1 == nx) umma_commit<1>(o_full(x));
                        }
                        if (more && !have_k) {
                            ok = take(ks);
                            have_k = true;
                        }
                        if (ok && j + 1 < nx) score(x, ks);
                    }
                    if (!ok) break;
                    umma_commit<1>(f_empty(vs));
                    if (more) umma_commit<1>(f_empty(ks));
                }
                q_phase ^= 1u;
            }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0) != 0;
        }
        if (lane == 0) {
            umma_commit<1>(drain_bar);
            wait_drain(drain_bar, 0);
        }
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

template <typename T, int D>
sq_status_t launch_prefill(const char* name, const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a,
                           cudaStream_t stream) {
    auto fn = kv8_prefill_kernel<T, D>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PCfg<D>::SMEM_ALLOC) != cudaSuccess)
        return check_launch(name);
    // items: at most one per 256 rows and one more per sequence, for every head
    const int64_t items = ((a.T * a.G + kItemRows - 1) / kItemRows + a.B) * a.Hkv;
    const int64_t sms = num_sms();
    launch_pdl(fn, dim3((unsigned)(items < sms ? items : sms)), dim3(kThreadsP), PCfg<D>::SMEM_ALLOC, stream, mk, mv, a);
    return check_launch(name);
}

}  // namespace

sq_status_t launch_kv8_prefill(const char* name, sq_dtype_t dt, int64_t D, const int8_t* Kc, const int8_t* Vc,
                               const AttnArgs& args, cudaStream_t stream) {
    AttnArgs a = args;
    a.box = a.block < kKeys ? a.block : kKeys;
    CUtensorMap mk, mv;
    if (!make_map_kv(&mk, Kc, a.num_blocks, (int64_t)a.Hkv * a.block, D, a.box, false) ||
        !make_map_kv(&mv, Vc, a.num_blocks, (int64_t)a.Hkv * a.block, D, a.box, false))
        return set_error(SQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", name);
    if (dt == SQ_BF16)
        return D == 128 ? launch_prefill<__nv_bfloat16, 128>(name, mk, mv, a, stream)
                        : launch_prefill<__nv_bfloat16, 64>(name, mk, mv, a, stream);
    return D == 128 ? launch_prefill<__half, 128>(name, mk, mv, a, stream)
                    : launch_prefill<__half, 64>(name, mk, mv, a, stream);
}

}  // namespace sq
