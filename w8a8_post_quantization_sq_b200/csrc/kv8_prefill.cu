// Attention over the paged int8 K/V cache for prompts: the sequences of a batch
// whose rows (new token x query head of a K/V head's group) are many.
//
// The same formula, scales and rounding as for single tokens (kv8_attention.cu):
// int8 codes as fp16, the K scale on the fp32 scores, the V scale in the
// softmax's exponent, P in fp16 below 2^15, a running maximum that moves only
// when a score passes it by 2^8. Here both products run on tcgen05 (kind::f16):
//   S = Q K^T   128 rows x 128 keys, both from shared memory
//   O += P V    P from tensor memory (it overwrites half of S), V from shared
//               memory with the columns contiguous (MN-major), as it lies in
//               the cache
// A CTA (one per SM, persistent) takes 256 rows of one sequence and K/V head as
// two tiles; while one tile's scores are on the tensor core, the other's are
// exponentiated. Tensor memory: S (128 columns) and O (D) of both tiles, 512 at
// D = 128. Roles:
//   warps 0..3, 4..7   softmax of tile 0, 1: a thread per row; also fetches Q,
//                      rescales O, writes Y and joins pieces
//   warps 8..11        int8 K and V tiles to fp16 tiles (128-byte swizzle): 128
//                      x D codes are converted once for 256 rows
//   warp 12            TMA of the int8 tiles
//   warp 13            the MMAs
//   warp 14            the CTA's items, worked out ahead and left in a ring
// Items are (sequence, 256 rows, head), the last rows of every sequence first (they
// see the most keys), dealt to the CTAs forth and back; few items are cut by
// their keys (see Items). The loops are rolled where the roles' code together
// would leave the instruction cache (unrolled throughout it took 120 KB, and a
// change of items 15,000 cycles of instruction fetches).
// What bounds it: 128 x 128 scores take 512 cycles of the tensor core for each
// product at D = 128 and 1024 of the exponential unit, two tiles 2048 of either.
// A step of two tiles takes 4700: a tile's chain of scores (two reads of tensor
// memory, the maximum, 128 exponentials per thread), product, next scores is
// sequential and two tiles are all that tensor memory holds; a change of items
// takes 11,000 more. 2 prompts of 1440 and 1380 tokens on 3300 keys, 32 heads over
// 8, D 128: 188 us, 630 TFLOP/s; 8 of 1024 on 4096: 586 us, 820; the same tokens and
// keys with 16 heads over 16, D 64: 309 us, 390.
// Every wait is bounded (about 2 s), code 0x9E1 + role in the status word.
#include <climits>

#include "sq_internal.h"
#include "sq_kv8.cuh"
#include "sq_tc.cuh"

namespace sq {
namespace {

constexpr int kKeys = 128;
constexpr int kTileRows = 128;
constexpr int kItemRows = 2 * kTileRows;
constexpr int kRaw = 2, kF16 = 4;  // ring stages: int8 tiles, fp16 tiles
constexpr int kThreadsP = 16 * 32;
// Registers per thread: 128 at launch, dealt out again by warpgroup (two softmax
// groups, conversion, TMA and MMA).
constexpr int kRegsSoftmax = 168, kRegsConvert = 96, kRegsIssue = 80;
static_assert(2 * kRegsSoftmax + kRegsConvert + kRegsIssue <= 4 * 128, "more registers than the block was launched with");

template <int D>
struct PCfg {
    static constexpr uint32_t HALF = kKeys * 128;           // 128 rows of 64 fp16
    static constexpr uint32_t TILE = D / 64 * HALF;         // 128 x D fp16
    static constexpr uint32_t RAW = kKeys * D;              // 128 x D int8
    static constexpr uint32_t Q_OFF = 0;
    static constexpr uint32_t F_OFF = Q_OFF + 2 * TILE;
    static constexpr uint32_t R_OFF = F_OFF + kF16 * TILE;
    static constexpr uint32_t BAR_OFF = R_OFF + kRaw * RAW;
    // raw_full[R], raw_empty[R], f_full[F], f_empty[F], q_ready[2], s_full[2], p_full[2], o_full[2], drain
    // item_full[2], item_empty[2]
    static constexpr uint32_t NBAR = 2 * kRaw + 2 * kF16 + 9 + 4;
    static constexpr uint32_t MISC_OFF = BAR_OFF + (NBAR + 1) / 2 * 16;  // tmem base, abort flag
    static constexpr uint32_t ITEM_OFF = MISC_OFF + 16;                  // Item[2]
    static constexpr uint32_t SMEM_ALLOC = ITEM_OFF + 2 * 64 + 1024;
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
// One lane of a converged warp: the MMA warp runs whole and its elected lane
// issues (216 -> 210 us at 2 prompts of some 1400 tokens, 32 heads, against a
// single lane in the role).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(p));
    return p != 0;
}
// 16 columns, with the wait in the same statement.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t* r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(taddr)
        : "memory");
}
__device__ __forceinline__ float max3(float a, float b, float c) {
    float y;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}
__device__ __forceinline__ float max3(uint32_t a, uint32_t b, uint32_t c) {
    return max3(__uint_as_float(a), __uint_as_float(b), __uint_as_float(c));
}
// The larger one, NaN if either is (fmaxf drops NaN).
__device__ __forceinline__ float max_nan(float a, float b) {
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}
// 16 bytes to shared memory (zeros without `live`), not waited for.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(live ? 16 : 0) : "memory");
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// An item, or a piece of one, as the scheduling warp leaves it for the others.
struct Item {
    int64_t lo;        // first new token of the sequence
    int b, h, r0;      // sequence (-1: no more), head, first row
    int n, len;        // new tokens and length of the sequence
    int k0;            // first key tile
    int tiles[2];      // key tiles of each row tile, from k0 (0: none here)
    int vis;           // keys that the item's last row sees
    int first, parts;  // the CTAs first .. first + parts - 1 have a piece each (1: whole)
};

// The CTA's items in turn. Level k of the order holds the k-th row block from
// the end of every sequence that has one, for every head. One warp walks them
// (32 sequences a look).
// Where there are fewer items than CTAs, their keys are cut too, into pieces of
// `cut` key tiles or fewer, such that every CTA has one piece at most. (One
// prompt of 64 tokens on 8192 keys, 8 heads: 182 us whole, 57 so. Where there are
// more, a cut costs what it balances: 360 items of 26 tiles and fewer, in equal
// shares of all key tiles, took 191 us, whole 185.) An item of kMinCut tiles or
// fewer stays whole: a join of two pieces costs as much as some four tiles.
constexpr int kMinCut = 8, kWhole = INT_MAX;
constexpr int kMaxGridP = 255;  // pieces of an item are counted in 8 bits
template <bool SPLIT>
struct Items {
    int64_t before, count;  // items (or pieces) of the levels before `level`, and of it
    int level, round, cut;
    Seq mine;  // sequence `lane` (the first 32 are kept)

    // lane's sequence of the 32 from `base`, its row blocks in rt (0: not a prompt)
    __device__ __forceinline__ static Seq load(const AttnArgs& a, int i) {
        Seq t;
        t.lo = 0;
        t.n = t.len = t.rt = 0;
        if (i < a.B) t = seq_of<kItemRows, kKeys>(a, i);
        if ((int64_t)t.n * a.G <= a.row_limit) t.rt = 0;
        return t;
    }
    __device__ __forceinline__ Seq seq(const AttnArgs& a, int base, int lane) const {
        return base ? load(a, base + lane) : mine;
    }
    __device__ __forceinline__ static Seq from_lane(const Seq& s, int l) {
        Seq t;
        t.lo = __shfl_sync(0xffffffffu, s.lo, l);
        t.n = __shfl_sync(0xffffffffu, s.n, l);
        t.len = __shfl_sync(0xffffffffu, s.len, l);
        t.rt = __shfl_sync(0xffffffffu, s.rt, l);
        return t;
    }
    // key tiles of a row block, and the pieces that they are cut into
    __device__ __forceinline__ static int tiles_of(const AttnArgs& a, const Seq& s, int blk) {
        const int last = (int)(min((int64_t)(blk + 1) * kItemRows, (int64_t)s.n * a.G) - 1);
        return max((seen_by(a, s, last) + kKeys - 1) / kKeys, 1);
    }
    __device__ __forceinline__ int pieces_of(const AttnArgs& a, const Seq& s, int blk) const {
        if (blk < 0) return 0;
        if (!SPLIT || cut == kWhole) return 1;
        return (tiles_of(a, s, blk) + cut - 1) / cut;
    }
    __device__ __forceinline__ void look(const AttnArgs& a, int lane) {
        int n = 0;
#pragma unroll 1
        for (int base = 0; base < a.B; base += 32) {
            const Seq s = seq(a, base, lane);
            n += __reduce_add_sync(0xffffffffu, pieces_of(a, s, s.rt - 1 - level));
        }
        count = (int64_t)n * a.Hkv;
    }
    // row blocks of all sequences, pieces of `cut` key tiles, or tiles (cut = 1)
    __device__ __forceinline__ int64_t sum(const AttnArgs& a, int lane) const {
        int64_t n = 0;
#pragma unroll 1
        for (int base = 0; base < a.B; base += 32) {
            const Seq s = seq(a, base, lane);
            if (cut == kWhole) {
                n += s.rt;
                continue;
            }
            unsigned left = __ballot_sync(0xffffffffu, s.rt > 0);
#pragma unroll 1
            while (left) {
                const Seq t = from_lane(s, __ffs(left) - 1);
                left &= left - 1;
#pragma unroll 1
                for (int blk = lane; blk < t.rt; blk += 32) n += pieces_of(a, t, blk);
            }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
        return n * a.Hkv;
    }
    __device__ __forceinline__ void begin(const AttnArgs& a, int lane) {
        before = 0;
        level = round = 0;
        mine = load(a, lane);
        cut = kWhole;
        if (SPLIT && sum(a, lane) < gridDim.x) {
            cut = 1;
            cut = (int)max(sum(a, lane) / gridDim.x, (int64_t)kMinCut);
#pragma unroll 1
            while (sum(a, lane) > gridDim.x) cut += max(cut >> 3, 1);
        }
        look(a, lane);
    }
    __device__ __forceinline__ bool next(const AttnArgs& a, int lane, Item& it) {
        const int64_t at = (int64_t)round * gridDim.x + ((round & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
        ++round;
#pragma unroll 1
        while (at >= before + count) {
            if (count == 0) return false;
            before += count;
            ++level;
            look(a, lane);
        }
        int off = (int)(at - before), pieces = 1, blk = 0;
        Seq s;
#pragma unroll 1
        for (int base = 0;; base += 32) {
            s = seq(a, base, lane);
            const int mb = s.rt - 1 - level;
            const unsigned has = __ballot_sync(0xffffffffu, mb >= 0);
            int mp = mb >= 0, up = __popc(has & (0xffffffffu >> (31 - lane)));  // with the sequences before
            if (SPLIT && cut != kWhole) {
                up = mp = pieces_of(a, s, mb);
#pragma unroll 1
                for (int o = 1; o < 32; o <<= 1) {
                    const int u = __shfl_up_sync(0xffffffffu, up, o);
                    if (lane >= o) up += u;
                }
            }
            const unsigned past = __ballot_sync(0xffffffffu, up * a.Hkv > off);
            if (past) {
                const int l = __ffs(past) - 1;
                pieces = __shfl_sync(0xffffffffu, mp, l);
                off -= (__shfl_sync(0xffffffffu, up, l) - pieces) * a.Hkv;
                blk = __shfl_sync(0xffffffffu, mb, l);
                it.b = base + l;
                s = from_lane(s, l);
                break;
            }
            off -= __shfl_sync(0xffffffffu, up, 31) * a.Hkv;
        }
        it.h = !SPLIT || pieces == 1 ? off : off / pieces;
        const int piece = off - it.h * pieces;
        it.first = (int)at - piece;
        it.parts = pieces;
        it.lo = s.lo;
        it.n = s.n;
        it.len = s.len;
        it.r0 = blk * kItemRows;
        const int rows = s.n * a.G;
        int k1 = INT_MAX;
        it.k0 = 0;
        if (SPLIT && pieces > 1) {
            const int64_t n = tiles_of(a, s, blk);
            it.k0 = (int)(n * piece / pieces);
            k1 = (int)(n * (piece + 1) / pieces);
        }
        it.vis = seen_by(a, s, min(it.r0 + kItemRows, rows) - 1);
#pragma unroll 1
        for (int x = 0; x < 2; ++x) {
            const int f = it.r0 + x * kTileRows;
            const int tiles = f < rows ? (seen_by(a, s, min(f + kTileRows, rows) - 1) + kKeys - 1) / kKeys : 0;
            it.tiles[x] = max(min(tiles, k1) - it.k0, 0);
        }
        return true;
    }
};

template <typename T, int D, bool SPLIT>
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
    auto item_full = [&](int s) { return bar1 + 8u * (9 + s); };
    auto item_empty = [&](int s) { return bar1 + 8u * (11 + s); };
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
            mbar_init(item_full(x), 1);
            mbar_init(item_empty(x), 14);  // warps 0..13
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
    auto wait = [&](uint32_t bar, uint32_t parity, int code) {
        return wait_suspended(bar, parity, abort_flag, a.status, code, kTimeoutNs);
    };
    bool ok = true;
    int is = 0;  // items taken from the ring
    // the next item (whole warps; false when there are no more)
    auto take_item = [&](Item& it) {
        ok = wait(item_full(is & 1), (uint32_t)(is >> 1) & 1u, 0x9E9);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) return false;
        it = *reinterpret_cast<const Item*>(smem + C::ITEM_OFF + (is & 1) * 64);
        __syncwarp();
        if (lane == 0) mbar_arrive(item_empty(is & 1));
        ++is;
        return it.b >= 0;
    };
    if (warp < 8) {
        // ------------------------------------------------------ softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        const int x = warp >> 2;
        const int row = (warp & 3) * 32 + lane;  // row of the tile, and lane of tensor memory
        const uint32_t quarter = (uint32_t)((warp & 3) * 32) << 16;
        const uint32_t t_s = tmem + quarter + (uint32_t)(x * 128), t_o = tmem + quarter + C::O_COL + (uint32_t)(x * D);
        uint32_t s_phase = 0, o_phase = 0;
        // The warp's 32 rows of q are copied to their places in the Q tile, 16 bytes a
        // lane and whole rows an access, and then scaled in place by a thread per row.
        // (Through registers, a row a lane, an access touched 32 lines: 8000 cycles
        // per item.)
        constexpr int LPR = D / 8, RPI = 32 / LPR;
        const uint32_t q_tile = sbase + C::Q_OFF + x * C::TILE;
        // 16 bytes `u` of row r (halves of 64 elements, swizzled)
        auto unit_of = [&](int r, int u) { return (uint32_t)((u >> 3) * C::HALF + r * 128 + (((u & 7) ^ (r & 7)) << 4)); };
        Item it = {};
        int blk0 = -1, blk1 = -1;
        // lane e < 8 looks after the scales of keys 16 e .. of a key tile: the block
        // number two tiles ahead, the scales one
        auto block_of = [&](int j) {
            const int key = (it.k0 + j) * kKeys + (lane & 7) * 16;
            return key < it.vis ? __ldg(a.table + (int64_t)it.b * a.ldb + (key >> a.block_log2)) : -1;
        };
        auto fetch = [&]() {
            blk0 = block_of(0);
            blk1 = block_of(1);
            const int rows = it.n * a.G, di = RPI / a.G, dg = RPI - di * a.G;
            int rl = (warp & 3) * 32 + lane / LPR;
            int r = it.r0 + x * kTileRows + rl, i = r / a.G, g = r - i * a.G;
            const T* q = static_cast<const T*>(a.Q) + it.lo * a.ldq + (int64_t)it.h * a.G * D + lane % LPR * 8;
#pragma unroll 1
            for (int e = 0; e < 32 / RPI; ++e) {
                cp_async16(q_tile + unit_of(rl, lane % LPR), r < rows ? q + i * a.ldq + g * D : a.Q, r < rows);
                rl += RPI;
                r += RPI;
                i += di;
                g += dg;
                if (g >= a.G) g -= a.G, ++i;
            }
        };
        // a CTA's part in the workspace: O in columns of four, m and l of the tile's rows
        auto part_of = [&](int cta) { return a.part + ((int64_t)cta * 2 + x) * ((D + 2) * kTileRows); };
        // a part's share of a sum under the maximum of all (no part of a row that saw
        // no key; NaN scores leave its m at -inf and its l NaN)
        auto share_of = [&](float mp, float lp, float top) {
            return lp == 0.0f ? 0.0f : mp == -INFINITY ? lp : lp * ex2(mp - top);
        };
        bool more = take_item(it);
        if (more) fetch();
#pragma unroll 1
        while (more) {
            const int rows = it.n * a.G, r = it.r0 + x * kTileRows + row;
            const bool live = r < rows;
            const int i = live ? r / a.G : 0;
            T* const y = static_cast<T*>(a.Y) + (it.lo + i) * a.ldy + (int64_t)(it.h * a.G + (live ? r - i * a.G : 0)) * D;
            // keys that the row sees (rows past the end: all, computed and not written)
            const int vis = !live ? INT_MAX : a.causal ? max(min(it.len - it.n + i + 1, it.len), 0) : it.len;
            // Q: scaled by a power of two per row to [1, 2), the score scale's
            // sign in it, as fp16
            float crow;
            {
                asm volatile("cp.async.wait_all;" ::: "memory");
                __syncwarp();
                uint32_t m2 = 0;
#pragma unroll 8
                for (int e = 0; e < D / 8; ++e) {
                    const uint4 w = *reinterpret_cast<const uint4*>(smem + C::Q_OFF + x * C::TILE + unit_of(row, e));
                    m2 = __vmaxu2(m2, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
                    m2 = __vmaxu2(m2, __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu));
                }
                float top[8];
                unpack<T>(make_uint4(max(m2 & 0xffffu, m2 >> 16), 0, 0, 0), top);
                const uint32_t field = min(max(__float_as_uint(top[0]) >> 23, 1u), 253u);
                const float down = copysignf(__uint_as_float((254u - field) << 23), a.scale);
                crow = fabsf(a.scale) * kLog2e * __uint_as_float(field << 23);
#pragma unroll 4
                for (int e = 0; e < D / 8; ++e) {
                    uint4* at = reinterpret_cast<uint4*>(smem + C::Q_OFF + x * C::TILE + unit_of(row, e));
                    float v[8];
                    unpack<T>(*at, v);
                    *at = make_uint4(pack_half2(v[0] * down, v[1] * down), pack_half2(v[2] * down, v[3] * down),
                                     pack_half2(v[4] * down, v[5] * down), pack_half2(v[6] * down, v[7] * down));
                }
            }
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(q_ready(x));
            auto scales_of = [&](int blk) {
                float2 s = make_float2(__uint_as_float(0x7fffffffu), __uint_as_float(0x7fffffffu));
                if (blk >= 0 && blk < a.num_blocks) {
                    s.x = __ldg(a.kqs + (int64_t)blk * a.Hkv + it.h);
                    s.y = __ldg(a.vqs + (int64_t)blk * a.Hkv + it.h);
                }
                return s;
            };
            const int tiles = it.tiles[x];
            float m = -INFINITY, l = 0.0f;
            int next_blk = blk1;
            float2 next = scales_of(blk0);
#pragma unroll 1
            for (int j = 0; j < tiles; ++j) {
                const float my_k = __frcp_rn(next.x), my_v = next.y, my_lv = -__log2f(next.y);
                next = scales_of(next_blk);
                next_blk = block_of(j + 2);
                ok = wait(s_full(x), s_phase, 0x9E1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                s_phase ^= 1u;
                tc_fence_after();
                const int key0 = (it.k0 + j) * kKeys;
                const bool masked = __any_sync(0xffffffffu, key0 + kKeys > vis);
                // per 16 keys: score factor and -log2 of the V scale; of keys that
                // this row does not see nothing is taken, whatever their scales.
                // The factor is never 0 (a row of zeros times a block of zeros, whose
                // 1 / kqs is 8e-11, would be): masked scores are -inf before they
                // are multiplied, and -inf x 0 is NaN. A NaN scale stays NaN.
                auto factors = [&](int k, float& f, float& lv) {
                    f = max_nan(crow * __shfl_sync(0xffffffffu, my_k, k), 1.17549435e-38f);
                    lv = __shfl_sync(0xffffffffu, my_lv, k);
                    if (key0 + 16 * k >= vis) f = 1.0f, lv = 0.0f;
                };
                uint32_t s[64];
                float f[4], lv[4];
                // 64 keys and their factors
                auto load = [&](int c) {
                    tmem_ld32_async(t_s + c * 64, s);
                    tmem_ld32_async(t_s + c * 64 + 32, s + 32);
#pragma unroll
                    for (int q = 0; q < 4; ++q) factors(4 * c + q, f[q], lv[q]);
                    tmem_wait(s);
                    tmem_wait(s + 32);
                };
                float tm = -INFINITY;
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    load(c);
                    if (masked) {
#pragma unroll
                        for (int e = 0; e < 64; ++e)
                            if (key0 + 64 * c + e >= vis) s[e] = 0xff800000u;
                        // (read again below)
#pragma unroll
                        for (int e = 0; e < 4; ++e) tmem_st16(t_s + c * 64 + 16 * e, s + 16 * e);
                        tmem_wait_st();
                    }
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t* v = s + 16 * q;
                        const float lo = max3(max3(v[0], v[1], v[2]), max3(v[3], v[4], v[5]), max3(v[6], v[7], v[8]));
                        const float hi = max3(max3(v[9], v[10], v[11]), max3(v[12], v[13], v[14]), __uint_as_float(v[15]));
                        const float top = fmaxf(lo, hi);
                        tm = fmaxf(tm, fmaf(top, f[q], lv[q]));
                    }
                }
                tm -= kLift;
                const bool move = tm > m + kSlack;
                if (__any_sync(0xffffffffu, move)) {
                    const float to = move ? tm : m;
                    const float r = to == -INFINITY ? 1.0f : ex2(m - to);
                    m = to;
                    l *= r;
                    if (j > 0) {
                        // (the scores' barrier says that the product before them is complete)
#pragma unroll 1
                        for (int c = 0; c < D / 16; ++c) {
                            uint32_t o[16];
                            tmem_ld16(t_o + c * 16, o);
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * r);
                            tmem_st16(t_o + c * 16, o);
                        }
                    }
                }
                const float mu = m == -INFINITY ? 0.0f : m;
                // weights, 64 keys at a time: P of 32 keys goes to the first half of their own
                // columns
#pragma unroll 1
                for (int c = 0; c < 2; ++c) {
                    load(c);
#pragma unroll
                    for (int hf = 0; hf < 2; ++hf) {
                        uint32_t p[16];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            const int g = 2 * hf + q;
                            const uint32_t* sg = s + 16 * g;
                            const uint64_t f2 = pk2(f[g], f[g]), c2 = pk2(lv[g] - mu, lv[g] - mu);
                            uint64_t w2[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                w2[e] = fma2(pk2(__uint_as_float(sg[2 * e]), __uint_as_float(sg[2 * e + 1])), f2, c2);
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                float p0, p1;
                                upk2(w2[e], p0, p1);
                                p0 = ex2(p0);
                                p1 = ex2(p1);
                                w2[e] = pk2(p0, p1);
                                p[8 * q + e] = pack_half2(p0, p1);
                            }
#pragma unroll
                            for (int e = 4; e > 0; e >>= 1)
#pragma unroll
                                for (int z = 0; z < e; ++z) w2[z] = add2(w2[z], w2[z + e]);
                            float a0, a1;
                            upk2(w2[0], a0, a1);
                            const int k = 4 * c + g;
                            const float vq = __shfl_sync(0xffffffffu, my_v, k);
                            l = fmaf(a0 + a1, key0 + 16 * k < vis ? vq : 0.0f, l);
                        }
                        tmem_st16(t_s + c * 64 + hf * 32, p);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(p_full(x));
            }
            if (!ok) break;
            const int first = it.first, parts = it.parts;
            // the next item's q is fetched while this one's last product runs
            more = take_item(it);
            if (!ok) break;
            if (more) fetch();
            ok = wait(o_full(x), o_phase, 0x9E2);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            o_phase ^= 1u;
            tc_fence_after();
            bool write = true;
            if (SPLIT && parts > 1) {
                // m, l and O (not yet divided) go to the workspace, a lane per row; the warp
                // that completes the count of its 32 rows joins the parts, in key order
                float* part = part_of(blockIdx.x);
                __stcg(part + D * kTileRows + row, m);
                __stcg(part + (D + 1) * kTileRows + row, l);
                if (tiles > 0) {
#pragma unroll 1
                    for (int c = 0; c < D / 16; ++c) {
                        uint32_t o[16];
                        tmem_ld16(t_o + c * 16, o);
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            __stcg(reinterpret_cast<uint4*>(part) + (4 * c + e) * kTileRows + row,
                                   make_uint4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]));
                    }
                }
                __threadfence();
                __syncwarp();
                const int shift = 8 * (warp & 3);
                unsigned* const cnt = reinterpret_cast<unsigned*>(a.cnt) + 2 * first + x;
                int count = 0;
                if (lane == 0) {
                    count = atomicAdd(cnt, 1u << shift) >> shift & 255;
                    if (count + 1 == parts) atomicSub(cnt, (unsigned)parts << shift);
                }
                write = __shfl_sync(0xffffffffu, count, 0) + 1 == parts;
                if (write) {
                    __threadfence();
                    m = -INFINITY;
                    l = 0.0f;
#pragma unroll 4
                    for (int i = 0; i < parts; ++i) m = fmaxf(m, __ldcg(part_of(first + i) + D * kTileRows + row));
#pragma unroll 4
                    for (int i = 0; i < parts; ++i) {
                        const float* from = part_of(first + i) + D * kTileRows + row;
                        l += share_of(__ldcg(from), __ldcg(from + kTileRows), m);
                    }
                }
            }
            const float inv = (m == -INFINITY && l == 0.0f) ? 0.0f : __frcp_rn(l);
#pragma unroll 1
            for (int c = 0; write && c < D / 16; ++c) {
                uint32_t s[16];
                if (SPLIT && parts > 1) {
                    float o[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = 0.0f;
#pragma unroll 4
                    for (int i = 0; i < parts; ++i) {
                        const float* from = part_of(first + i);
                        const float lp = __ldcg(from + (D + 1) * kTileRows + row);
                        const float r = share_of(__ldcg(from + D * kTileRows + row), 1.0f, m);
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float4 v = __ldcg(reinterpret_cast<const float4*>(from) + (4 * c + e) * kTileRows + row);
                            if (lp != 0.0f) {
                                o[4 * e] = fmaf(v.x, r, o[4 * e]);
                                o[4 * e + 1] = fmaf(v.y, r, o[4 * e + 1]);
                                o[4 * e + 2] = fmaf(v.z, r, o[4 * e + 2]);
                                o[4 * e + 3] = fmaf(v.w, r, o[4 * e + 3]);
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] = __float_as_uint(o[e]);
                } else if (tiles > 0) {
                    tmem_ld16(t_o + c * 16, s);
                } else {
#pragma unroll
                    for (int e = 0; e < 16; ++e) s[e] = 0u;
                }
                if (live) {
                    uint32_t p[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        p[e] = (uint32_t)to16<T>(__uint_as_float(s[2 * e]) * inv) |
                               ((uint32_t)to16<T>(__uint_as_float(s[2 * e + 1]) * inv) << 16);
                    *reinterpret_cast<uint4*>(y + c * 16) = make_uint4(p[0], p[1], p[2], p[3]);
                    *reinterpret_cast<uint4*>(y + c * 16 + 8) = make_uint4(p[4], p[5], p[6], p[7]);
                }
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp < 12) {
        // ------------------------------------------------------ conversion
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsConvert));
        const int t = threadIdx.x - 256;
        int rs = 0, fs = 0;
        uint32_t rp = 0, fp = 0;
        Item it;
#pragma unroll 1
        while (ok && take_item(it)) {
            const int n = 2 * max(it.tiles[0], it.tiles[1]);
#pragma unroll 1
            for (int j = 0; ok && j < n; ++j) {
                ok = wait(raw_full(rs), rp, 0x9E3) &&
                     wait(f_empty(fs), fp ^ 1u, 0x9E4);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                const uint8_t* src = smem + C::R_OFF + rs * C::RAW;
                uint8_t* dst = smem + C::F_OFF + fs * C::TILE;
                constexpr int UPR = D / 16;  // 16-code units per key
#pragma unroll 4
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
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        int rs = 0;
        uint32_t rp = 0, issued = 0, issued_phase = 0;
        const int box = a.box, per_box = box / 16;
        Item it;
#pragma unroll 1
        while (ok && take_item(it)) {
            const int n = max(it.tiles[0], it.tiles[1]);
            const int32_t* table = a.table + (int64_t)it.b * a.ldb;
            // lane e looks after part e % 8 (16 keys) of tile j0 + e / 8
            auto block_of = [&](int j0) {
                const int key = (it.k0 + j0) * kKeys + lane * 16;
                const int blk = key < it.vis ? __ldg(table + (key >> a.block_log2)) : -1;
                return blk >= 0 && blk < a.num_blocks ? blk : -1;
            };
            int next = block_of(0);
#pragma unroll 1
            for (int j0 = 0; ok && j0 < n; j0 += 4) {
                const int blk = next;
                if (j0 + 4 < n) next = block_of(j0 + 4);
                const int y = it.h * a.block + (((it.k0 + j0) * kKeys + lane * 16) & (a.block - 1));
#pragma unroll 1
                for (int j = j0; ok && j < min(j0 + 4, n); ++j) {
                    const int part = lane - (j - j0) * 8;
                    const bool copy = part >= 0 && part < 8 && blk >= 0 && part % per_box == 0;
                    const int boxes = __popc(__ballot_sync(0xffffffffu, copy));
#pragma unroll 1
                    for (int v = 0; v < 2; ++v) {
                        ok = wait(raw_empty(rs), rp ^ 1u, 0x9E5);
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
                if (issued >> s & 1u) wait_drain_inline(raw_full(s), issued_phase >> s & 1u);
    } else if (warp == 13) {
        // ------------------------------------------------------ MMA
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        int fs = 0;  // stage of the next fp16 tile in the order K0 V0 K1 V1 ...
        uint32_t fp = 0, q_phase = 0, p_phase[2] = {0, 0};
        // descriptors of the first tiles; others differ in the address field (16-byte
        // units, no carry: all of shared memory is 14 bits of them)
        const uint64_t q_desc = sdesc(sbase + C::Q_OFF), k_desc = sdesc(sbase + C::F_OFF),
                       v_desc = sdesc_mn(sbase + C::F_OFF, C::HALF);
        Item it;
#pragma unroll 1
        while (ok && take_item(it)) {
            const int n0 = __shfl_sync(0xffffffffu, it.tiles[0], 0), n1 = __shfl_sync(0xffffffffu, it.tiles[1], 0);
            const int n = max(n0, n1);
            auto take = [&](int& stage) {  // waits for the next fp16 tile
                stage = fs;
                const bool got = __all_sync(0xffffffffu, wait(f_full(fs), fp, 0x9E6));
                if (++fs == kF16) fs = 0, fp ^= 1u;
                tc_fence_after();
                return got;
            };
            auto score = [&](int x, int st) {
                const uint64_t qa = q_desc + (uint32_t)x * (C::TILE >> 4), kb = k_desc + (uint32_t)st * (C::TILE >> 4);
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t off = ((k >> 2) * C::HALF + (k & 3) * 32) >> 4;
                    if (elect_one()) umma_ss(tmem + x * 128, qa + off, kb + off, C::IDESC_S, k != 0);
                }
                if (elect_one()) umma_commit<1>(s_full(x));
            };
            int ks = 0, vs = 0;
            // step j: the products with V of tile j (from 0), then the scores of tile j + 1
#pragma unroll 1
            for (int j = -1; ok && j < n; ++j) {
                if (j >= 0) ok = take(vs);
                const bool more = j + 1 < n;
                bool have_k = false;
#pragma unroll 1
                for (int x = 0; ok && x < 2; ++x) {
                    const int nx = x ? n1 : n0;
                    if (j >= 0 && j < nx) {
                        ok = __all_sync(0xffffffffu, wait(p_full(x), p_phase[x], 0x9E8));
                        if (!ok) break;
                        p_phase[x] ^= 1u;
                        tc_fence_after();
                        const uint64_t vb = v_desc + (uint32_t)vs * (C::TILE >> 4);
#pragma unroll
                        for (int k = 0; k < kKeys / 16; ++k)
                            if (elect_one())
                                umma_ts(tmem + C::O_COL + x * D, tmem + x * 128 + (k >> 1) * 32 + (k & 1) * 8,
                                        vb + (k * 16 * 128 >> 4), C::IDESC_O, (j != 0 || k != 0) ? 1u : 0u);
                    }
                    if (x == 1 && j >= 0 && elect_one()) umma_commit<1>(f_empty(vs));  // both products with V are issued
                    if (more && !have_k) {
                        ok = take(ks);
                        have_k = true;
                    }
                    if (ok && j < 0) {
                        ok = __all_sync(0xffffffffu, wait(q_ready(x), q_phase, 0x9E7));
                        tc_fence_after();
                    }
                    if (ok && j + 1 < nx) score(x, ks);
                    // (with no tile at all too: the rows' warps are never a whole item ahead)
                    if (ok && j + 1 == nx && elect_one()) umma_commit<1>(o_full(x));
                }
                if (!ok) break;
                if (more && elect_one()) umma_commit<1>(f_empty(ks));
            }
            q_phase ^= 1u;
        }
        if (lane == 0) {
            umma_commit<1>(drain_bar);
            wait_drain_inline(drain_bar, 0);
        }
    } else {
        // ------------------------------------------------------ items
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsIssue));
        if (warp == 14) {
            Items<SPLIT> list;
            list.begin(a, lane);
            bool more = true;
#pragma unroll 1
            for (int n = 0; more; ++n) {
                Item it;
                more = list.next(a, lane, it);
                if (!more) it.b = -1;
                ok = wait(item_empty(n & 1), ((uint32_t)(n >> 1) & 1u) ^ 1u, 0x9EA);
                if (!__all_sync(0xffffffffu, ok)) break;
                if (lane == 0) {
                    *reinterpret_cast<Item*>(smem + C::ITEM_OFF + (n & 1) * 64) = it;
                    mbar_arrive(item_full(n & 1));
                }
            }
        }
    }
    // pieces that gave up leave their rows counted in: what is to be cleared with the status
    if (SPLIT && !ok) a.status[3] = a.cnt_bytes;
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
    }
}

int prefill_grid() { return num_sms() < kMaxGridP ? num_sms() : kMaxGridP; }

template <typename T, int D, bool SPLIT>
sq_status_t launch_prefill(const char* name, const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a,
                           cudaStream_t stream) {
    auto fn = kv8_prefill_kernel<T, D, SPLIT>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)PCfg<D>::SMEM_ALLOC) != cudaSuccess)
        return check_launch(name);
    launch_pdl(fn, dim3(prefill_grid()), dim3(kThreadsP), PCfg<D>::SMEM_ALLOC, stream, mk, mv, a);
    return check_launch(name);
}

template <typename T, int D>
sq_status_t launch_either(const char* name, bool split, const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a,
                          cudaStream_t stream) {
    return split ? launch_prefill<T, D, true>(name, mk, mv, a, stream) : launch_prefill<T, D, false>(name, mk, mv, a, stream);
}

}  // namespace

size_t kv8_prefill_part_bytes(int64_t D) {
    return (size_t)prefill_grid() * 2 * kTileRows * (size_t)(D + 2) * sizeof(float);
}

sq_status_t launch_kv8_prefill(const char* name, sq_dtype_t dt, int64_t D, const int8_t* Kc, const int8_t* Vc,
                               const AttnArgs& args, cudaStream_t stream) {
    AttnArgs a = args;
    a.box = a.block < kKeys ? a.block : kKeys;
    CUtensorMap mk, mv;
    if (!make_map_kv(&mk, Kc, a.num_blocks, (int64_t)a.Hkv * a.block, D, a.box, false) ||
        !make_map_kv(&mv, Vc, a.num_blocks, (int64_t)a.Hkv * a.block, D, a.box, false))
        return set_error(SQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", name);
    // Which sequences are prompts is on the device: their items are counted there, by
    // the kernel that can cut them. Where T or the table's width rules it out (or T
    // makes it unlikely) the other one is faster: 36 against 41 us at 4 x 128 tokens on
    // 1000 keys, 32 heads, 187 against 192 at 2 x 1400 on 3300.
    const bool split = a.T * a.G * a.Hkv < (int64_t)prefill_grid() * kItemRows &&
                       (int64_t)a.max_blocks * a.block > kMinCut * kKeys;
    if (dt == SQ_BF16)
        return D == 128 ? launch_either<__nv_bfloat16, 128>(name, split, mk, mv, a, stream)
                        : launch_either<__nv_bfloat16, 64>(name, split, mk, mv, a, stream);
    return D == 128 ? launch_either<__half, 128>(name, split, mk, mv, a, stream)
                    : launch_either<__half, 64>(name, split, mk, mv, a, stream);
}

}  // namespace sq
