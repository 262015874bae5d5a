// Attention over the paged int8 K/V cache (a scale per block of tokens and
// head), for any number of new tokens per sequence.
//
//   s_j = scale q . k_j,  k_j = K_j / kqs(j)      (K_j, V_j: int8 codes)
//   o   = sum_j w_j v_j,  w = softmax(s),  v_j = V_j / vqs(j)
// over the keys j < len - n + i + 1 of new token i of n (causal) or j < len.
//
// The codes go through the tensor cores as fp16, which holds every int8
// exactly; the two scales of a block multiply the 16 x 16 score tiles in fp32:
// the K scale multiplies the scores, and the V scale is folded into the
// softmax's exponent. With t_j = log2(e) s_j - log2(vqs(j)) and m, the running
// maximum of t (not of s) less 7,
//   P_j = 2^(t_j - m),  O = sum_j P_j V_j,  l = sum_j P_j vqs(j),  o = O / l,
// and V is never scaled. m is moved only when a t passes it by 15 (the rescaling
// of O then costs nothing on most tiles), so P, the only quantity rounded to
// fp16, stays below 2^15 whatever the scales. Its rounding is at most 2^-11
// relative, as that of an fp16 output, down to 2^-21 of the largest P of the keys
// that share m; below that it is an fp16 subnormal, off by 2^-32 of the largest.
// m, l, O are fp32.
// q is scaled by a power of two per row to [1, 2) before it becomes fp16, so it
// keeps its bits, but for elements that are then below 2^-14 (fp16 subnormals,
// off by 2^-25 at most).
//
// Work: rows (new token, query head of the group) of one sequence and K/V head
// make row tiles of 8 or 16; the keys of each row tile are cut into tiles of 64 (128),
// and the list of all tiles is cut into one contiguous range per block (the
// lengths are on the device; every block works out its own range). A row tile
// whose keys fall into several ranges is joined by the block that finishes last,
// in range order, so results do not depend on timing.
// In a block, one warp brings a tile's K and V by TMA (swizzled, ring of stages),
// and four warps take 16 (32) keys each. A decode step has 1 to 16 rows per
// K/V head, an eighth of the smallest tcgen05 tile, and is bound by the cache's
// bytes and by the conversions, so the products are mma.m16n8k16 with the keys
// (K) and the columns (V) on the 16-wide side and 8 rows on the other: half the
// instructions and registers of the usual orientation.
// Measured (32 heads over 8, D 128): 64 sequences of up to 8192 keys 107 us, 5.4 TB/s
// (0.83 of the copy rate); one of 1000 keys 11.2 us, the chain of loads and the join.
// Rows past 16 of a head are further row tiles, which read and convert the keys
// again: 16 sequences on 4000 keys (20 us of bytes) take 48 us with 4 tokens each,
// 75 with 8 and 133 with 16. At D = 128 the kernel of two row groups spills (152
// bytes stored, 248 loaded per thread).
#include <cstring>

#include "sq_internal.h"
#include "sq_kv8.cuh"
#include "sq_tc.cuh"

namespace sq {

namespace {

constexpr int kSub = 16;      // keys that one MMA takes
// 16-key parts per warp and stage: a stage is 16 KB at either head width. (At D =
// 64 with one part, the per-stage work of a warp, waits, maximum and branches, was
// as long as the products: 16 sequences x 4 tokens of up to 4000 keys took 25.5 us,
// with two 21.5.)
constexpr int parts_of(int d) { return d == 64 ? 2 : 1; }
constexpr int kCWarps = 4;    // consumer warps
constexpr int kThreadsA = 32 * (kCWarps + 1);
constexpr int kStages = 3;
// Sequences of more rows than this go to the prompt kernel where one is launched.
// Here / there (us), D = 128, 8 heads: 1 sequence on 8192 keys, 16 rows 23.7 / 48.2, 64
// rows 32 / 48; 4 on 4000, 64 rows 44 / 45; 16 on 4000, 48 rows 106 / 112, 64 rows
// 133 / 112. D = 64, 4 heads, 64 rows: 1 on 8192 16 / 36, 16 on 4000 43 / 71.
constexpr int64_t kRowLimit = 64;
// blocks per SM by row groups of 8: registers (accumulators) and shared memory
constexpr int ctas_per_sm(int nr) { return nr == 1 ? 3 : 2; }

template <int D, int NR>
struct ACfg {
    static constexpr int ROWS = 8 * NR;
    static constexpr int PARTS = parts_of(D);
    static constexpr int TILE = kCWarps * kSub * PARTS;  // keys per stage
    static constexpr int NPART = TILE / kSub;            // 16-key parts per stage
    static constexpr uint32_t KV = TILE * D;             // bytes of one stage's K (and of its V)
    static constexpr uint32_t STAGE = 2 * KV;
    static constexpr uint32_t SC_OFF = kStages * STAGE;                  // float4 [stages][parts]: 1/kqs, -log2 vqs, vqs
    static constexpr uint32_t BAR_OFF = SC_OFF + kStages * NPART * 16;   // full[S], empty[S]
    static constexpr uint32_t MISC_OFF = BAR_OFF + 2 * kStages * 8;  // abort flag, last flag
    static constexpr uint32_t ML_OFF = MISC_OFF + 16;                // m, l [warps][rows]
    static constexpr int LDO = D + 4;                                // floats per row of a warp's O
    static constexpr uint32_t O_OFF = ML_OFF + kCWarps * ROWS * 2 * 4;
    static constexpr uint32_t SMEM = O_OFF + kCWarps * ROWS * LDO * 4;
    static constexpr uint32_t SMEM_ALLOC = SMEM + 1024;
};

__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
    return v;
}
// D += A B on 16 x 8 x 16 fp16 with fp32 sums
__device__ __forceinline__ void mma16816(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 tile of 16-bit elements transposed across the warp.
__device__ __forceinline__ uint32_t movmatrix(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// floor(a / b); a call, so that the 64-bit division is in the code once.
static __device__ __noinline__ int64_t div_floor(int64_t a, int b) {
    return a < (1ll << 31) ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

template <int ROWS, int KEYS>
__device__ __forceinline__ Seq short_seq(const AttnArgs& a, int b) {
    Seq s = seq_of<ROWS, KEYS>(a, b);
    if ((int64_t)s.n * a.G > a.row_limit) s.rt = 0;
    return s;
}

// A block's range of the list of key tiles, as pieces: the part of the range
// inside one row tile. Every warp walks the same sequence.
template <int ROWS, int KEYS>
struct Walk {
    int64_t it, end, total;
    int units, b, item, k0, k1;
    bool first;
    Seq s;
    __device__ __forceinline__ int64_t start_of(int c) const { return div_floor(c * total, units); }
    // the unit whose range holds x: the first c with start_of(c + 1) > x
    __device__ __forceinline__ int owner_of(int64_t x) const {
        // (units fits 11 bits, so (x + 1) * units stays inside 64; the quotient
        // by `total` is below units)
        const int64_t n = (x + 1) * units + total - 1;
        if (n < (1ll << 31)) return (int)((uint32_t)n / (uint32_t)total) - 1;
        return (int)(n / total - 1);
    }

    __device__ __forceinline__ void init(const AttnArgs& a, int lane) {
        // 32 sequences a look: their work, and the work up to each of them
        Seq mine;
        int64_t w, inc;
        auto look = [&](int base) {
            mine = short_seq<ROWS, KEYS>(a, min(base + lane, a.B - 1));
            w = base + lane < a.B ? mine.work(a.Hkv) : 0;
            inc = w;
#pragma unroll 1
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t up = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += up;
            }
        };
        total = 0;
        int base = 0;
#pragma unroll 1
        for (; base < a.B; base += 32) {
            look(base);
            total += __shfl_sync(0xffffffffu, inc, 31);
        }
        units = (int)min((int64_t)gridDim.x, total);
        it = end = 0;
        first = true;
        b = item = k0 = 0;
        if ((int)blockIdx.x >= units) return;
        it = start_of(blockIdx.x);
        end = start_of(blockIdx.x + 1);
        // the sequence that holds `it` (up to 32 sequences are still at hand)
        int64_t before = 0;
        unsigned past;
        base = 0;
#pragma unroll 1
        for (;; base += 32) {
            if (a.B > 32) look(base);
            past = __ballot_sync(0xffffffffu, before + inc > it);
            if (past) break;
            before += __shfl_sync(0xffffffffu, inc, 31);
        }
        const int l = __ffs(past) - 1;
        b = base + l;
        before += __shfl_sync(0xffffffffu, inc - w, l);
        s.lo = __shfl_sync(0xffffffffu, mine.lo, l);
        s.n = __shfl_sync(0xffffffffu, mine.n, l);
        s.len = __shfl_sync(0xffffffffu, mine.len, l);
        s.rt = __shfl_sync(0xffffffffu, mine.rt, l);
        s.tiles = __shfl_sync(0xffffffffu, mine.tiles, l);
        item = (int)div_floor(it - before, s.tiles);
        k0 = (int)(it - before - (int64_t)item * s.tiles);
    }
    // The next piece: tiles [k0, k1) of row tile `item` of sequence b.
    __device__ __forceinline__ bool next(const AttnArgs& a) {
        if (it >= end) return false;
        while (item >= a.Hkv * s.rt) {
            s = short_seq<ROWS, KEYS>(a, ++b);
            item = 0;
        }
        k1 = (int)min((int64_t)s.tiles, k0 + (end - it));
        return true;
    }
    __device__ __forceinline__ void done() {
        it += k1 - k0;
        first = false;
        k0 = 0;
        ++item;
    }
    __device__ __forceinline__ int seen(const AttnArgs& a, int row) const { return seen_by(a, s, row); }
};

template <typename T, int D, int NR>
__global__ void __launch_bounds__(kThreadsA, ctas_per_sm(NR))
kv8_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                     const AttnArgs a) {
    using C = ACfg<D, NR>;
    constexpr int ROWS = C::ROWS;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t sbase = smem_u32(smem);
    auto full_bar = [&](int s) { return sbase + C::BAR_OFF + 8u * s; };
    auto empty_bar = [&](int s) { return sbase + C::BAR_OFF + 8u * (kStages + s); };
    volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1);
            mbar_init(empty_bar(s), kCWarps);
        }
        *abort_flag = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    pdl_trigger();
    Walk<ROWS, C::TILE> w;
    w.init(a, lane);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    if (warp == kCWarps) {
        // ------------------------------------------------------ producer
        float4* sc = reinterpret_cast<float4*>(smem + C::SC_OFF);
        const int per_box = a.box / kSub;  // 16-key parts per copy
        uint32_t issued = 0, issued_phase = 0;
        for (; ok && w.next(a); w.done()) {
            const int h = w.item / w.s.rt, rt = w.item - h * w.s.rt;
            const int vis = w.seen(a, rt * ROWS + ROWS - 1);
            const int last = min(w.k1, (vis + C::TILE - 1) / C::TILE);
            const int32_t* row = a.table + (int64_t)w.b * a.ldb;
            // lane l looks after part l of the next few tiles' 32 parts; the block
            // numbers of those after them are on their way meanwhile
            constexpr int LOOK = 32 / C::NPART;
            auto block_of = [&](int t0) {
                const int key = t0 * C::TILE + lane * kSub;
                return key < vis ? __ldg(row + (key >> a.block_log2)) : -1;
            };
            int blk_next = block_of(w.k0);
            for (int t0 = w.k0; ok && t0 < last; t0 += LOOK) {
                const int key = t0 * C::TILE + lane * kSub;
                const int64_t blk = blk_next >= 0 && blk_next < a.num_blocks ? blk_next : -1;
                float kq = __uint_as_float(0x7fffffffu), vq = kq;  // no such block: NaN scales, nothing read
                if (blk >= 0) {
                    kq = __ldg(a.kqs + blk * a.Hkv + h);
                    vq = __ldg(a.vqs + blk * a.Hkv + h);
                }
                if (t0 + LOOK < last) blk_next = block_of(t0 + LOOK);
                const int y = h * a.block + (key & (a.block - 1));
                for (int t = t0; t < min(t0 + LOOK, last); ++t) {
                    ok = wait_fast(empty_bar(stage), phase ^ 1u, abort_flag, a.status, 0x7E1);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                    const int sub = lane - (t - t0) * C::NPART;
                    const bool mine_now = sub >= 0 && sub < C::NPART;
                    const bool copy = mine_now && blk >= 0 && sub % per_box == 0;
                    const int boxes = __popc(__ballot_sync(0xffffffffu, copy));
                    if (lane == 0) mbar_expect_tx_only(full_bar(stage), (uint32_t)(2 * boxes * a.box * D));
                    __syncwarp();
                    if (copy) {
                        const uint32_t dst = sbase + stage * C::STAGE + sub * kSub * D;
                        tma_load_3d<1>(dst, &map_k, full_bar(stage), 0, y, (int)blk);
                        tma_load_3d<1>(dst + C::KV, &map_v, full_bar(stage), 0, y, (int)blk);
                    }
                    // the scales arrive while the copies run
                    if (mine_now) sc[stage * C::NPART + sub] = make_float4(__frcp_rn(kq), -__log2f(vq), vq, 0.0f);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(full_bar(stage));
                    issued |= 1u << stage;
                    issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
                    if (++stage == kStages) stage = 0, phase ^= 1u;
                }
            }
        }
        if (!ok)
            for (int s = 0; s < kStages; ++s)
                if (issued >> s & 1u) wait_drain(full_bar(s), issued_phase >> s & 1u);
        return;
    }
    // ---------------------------------------------------------- consumers
    const int g = lane >> 2, c = lane & 3;
    constexpr int NK = D / 16;  // k-steps of a score
    constexpr int NO = D / 16;  // 16-column tiles of O
    constexpr int DG = D / 8;   // columns of O per lane group g
    float* ml = reinterpret_cast<float*>(smem + C::ML_OFF);  // m [warps][rows], l [warps][rows]
    float* osm = reinterpret_cast<float*>(smem + C::O_OFF);
    volatile int* last_flag = reinterpret_cast<volatile int*>(smem + C::MISC_OFF + 4);
    for (; w.next(a); w.done()) {
        const int h = w.item / w.s.rt, rt = w.item - h * w.s.rt;
        const int rows = w.s.n * a.G;  // rows of the sequence
        const int r0 = rt * ROWS;
        const int vis_last = w.seen(a, r0 + ROWS - 1), vis_first = w.seen(a, r0);
        const int last = min(w.k1, (vis_last + C::TILE - 1) / C::TILE);
        // q of row g of each group of 8: lane c holds columns [c D/4, (c + 1)
        // D/4), as the B operand of k-step j the columns 4 j .. 4 j + 3 of those
        // (the same permutation of the summed axis as K's below)
        uint32_t qf[NR][NK][2];
        float crow[NR][2];  // of this lane's rows 2 c, 2 c + 1: score of the codes -> log2
        int vis[NR][2];
#pragma unroll
        for (int z = 0; z < NR; ++z) {
            const int r = r0 + 8 * z + g;
            float v[D / 4];
#pragma unroll
            for (int e = 0; e < D / 4; ++e) v[e] = 0.0f;
            if (r < rows) {
                const int i = r / a.G;
                const T* q = static_cast<const T*>(a.Q) + (w.s.lo + i) * a.ldq + (int64_t)(h * a.G + r - i * a.G) * D +
                             c * (D / 4);
#pragma unroll
                for (int e = 0; e < D / 32; ++e) unpack<T>(ldg_nc_v4(q + 8 * e), v + 8 * e);
            }
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < D / 4; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
            m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
            const uint32_t field = min(max(m >> 23, 1u), 253u);
            const float down = __uint_as_float((254u - field) << 23);
            const float cr = a.scale * kLog2e * __uint_as_float(field << 23);
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                crow[z][x] = __shfl_sync(0xffffffffu, cr, (2 * c + x) * 4);
                const int rr = r0 + 8 * z + 2 * c + x;
                vis[z][x] = rr < rows ? w.seen(a, rr) : 0;
            }
#pragma unroll
            for (int j = 0; j < NK; ++j) {
                qf[z][j][0] = pack_half2(v[4 * j] * down, v[4 * j + 1] * down);
                qf[z][j][1] = pack_half2(v[4 * j + 2] * down, v[4 * j + 3] * down);
            }
        }
        // O transposed: tile j holds columns g DG + 2 j (elements 0, 1: rows 2 c,
        // 2 c + 1) and g DG + 2 j + 1 (elements 2, 3)
        float o[NR][NO][4];
        float m[NR][2], l[NR][2];
#pragma unroll
        for (int z = 0; z < NR; ++z) {
#pragma unroll
            for (int j = 0; j < NO; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) o[z][j][e] = 0.0f;
            m[z][0] = m[z][1] = -INFINITY;
            l[z][0] = l[z][1] = 0.0f;
        }
        for (int t = w.k0; t < last; ++t) {
            if (ok) ok = wait_fast(full_bar(stage), phase, abort_flag, a.status, 0x7E2);
            ok = __all_sync(0xffffffffu, ok);
            constexpr int PARTS = C::PARTS;
            const int key0 = t * C::TILE + warp * (kSub * PARTS);
            if (ok && key0 < vis_last) {
                const float4* scs = reinterpret_cast<const float4*>(smem + C::SC_OFF) + stage * C::NPART + warp * PARTS;
                const uint32_t kb0 = sbase + stage * C::STAGE + warp * (kSub * PARTS) * D;
                // scores: keys g (elements 0, 1), g + 8 (2, 3) of each part; rows 2 c, 2 c + 1
                float s[PARTS][NR][4];
#pragma unroll
                for (int u = 0; u < PARTS; ++u) {
                    // keys g and g + 8: lane c's D / 4 bytes are one or two 16-byte
                    // units, swizzled by row
                    const uint32_t kb = kb0 + u * kSub * D;
                    uint32_t kw[2][D / 16];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const int row = g + 8 * x;
                        if constexpr (D == 128) {
                            const uint4 u0 = lds128(kb + row * D + (((2 * c) ^ g) << 4));
                            const uint4 u1 = lds128(kb + row * D + (((2 * c + 1) ^ g) << 4));
                            kw[x][0] = u0.x, kw[x][1] = u0.y, kw[x][2] = u0.z, kw[x][3] = u0.w;
                            kw[x][4] = u1.x, kw[x][5] = u1.y, kw[x][6] = u1.z, kw[x][7] = u1.w;
                        } else {
                            const uint4 u0 = lds128(kb + row * D + ((c ^ (g >> 1)) << 4));
                            kw[x][0] = u0.x, kw[x][1] = u0.y, kw[x][2] = u0.z, kw[x][3] = u0.w;
                        }
                    }
#pragma unroll
                    for (int z = 0; z < NR; ++z)
#pragma unroll
                        for (int e = 0; e < 4; ++e) s[u][z][e] = 0.0f;
#pragma unroll
                    for (int j = 0; j < NK; ++j) {
                        const uint32_t u0 = kw[0][j] ^ 0x80808080u, u1 = kw[1][j] ^ 0x80808080u;
                        const uint32_t af[4] = {half2_of(u0, 0x4140), half2_of(u1, 0x4140), half2_of(u0, 0x4342),
                                                half2_of(u1, 0x4342)};
#pragma unroll
                        for (int z = 0; z < NR; ++z) mma16816(s[u][z], af, qf[z][j][0], qf[z][j][1]);
                    }
                }
                // scores in log2 with the V scale folded in
                const bool masked = key0 + kSub * PARTS > vis_first;
                float tm[NR][2];
                bool move = false;
#pragma unroll
                for (int z = 0; z < NR; ++z)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float q = -INFINITY;
#pragma unroll
                        for (int u = 0; u < PARTS; ++u) {
                            const float f = crow[z][x] * scs[u].x, lv = scs[u].y;
                            s[u][z][x] = fmaf(s[u][z][x], f, lv);
                            s[u][z][2 + x] = fmaf(s[u][z][2 + x], f, lv);
                            if (masked) {
                                if (key0 + u * kSub + g >= vis[z][x]) s[u][z][x] = -INFINITY;
                                if (key0 + u * kSub + g + 8 >= vis[z][x]) s[u][z][2 + x] = -INFINITY;
                            }
                            q = fmaxf(q, fmaxf(s[u][z][x], s[u][z][2 + x]));
                        }
                        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 4));
                        q = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 8));
                        tm[z][x] = fmaxf(q, __shfl_xor_sync(0xffffffffu, q, 16)) - kLift;
                        move |= tm[z][x] > m[z][x] + kSlack;
                    }
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int z = 0; z < NR; ++z)
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float to = fmaxf(m[z][x], tm[z][x]);
                            const float f = to == -INFINITY ? 1.0f : ex2(m[z][x] - to);
                            m[z][x] = to;
                            l[z][x] *= f;
#pragma unroll
                            for (int j = 0; j < NO; ++j) o[z][j][x] *= f, o[z][j][2 + x] *= f;
                        }
                }
#pragma unroll
                for (int u = 0; u < PARTS; ++u) {
                    const float vq = scs[u].z;
                    uint32_t pf[NR][2];
#pragma unroll
                    for (int z = 0; z < NR; ++z) {
                        float p[4];
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float mu = m[z][x] == -INFINITY ? 0.0f : m[z][x];
                            p[x] = ex2(s[u][z][x] - mu);
                            p[2 + x] = ex2(s[u][z][2 + x] - mu);
                            // (a row that sees none of these keys takes nothing from their scale)
                            if (!masked || key0 + u * kSub < vis[z][x]) l[z][x] = fmaf(p[x] + p[2 + x], vq, l[z][x]);
                        }
                        // rows to the lane groups, keys to the lanes: the B operand
                        pf[z][0] = movmatrix(pack_half2(p[0], p[1]));
                        pf[z][1] = movmatrix(pack_half2(p[2], p[3]));
                    }
                    // V: this lane's keys are 2 c, 2 c + 1, 2 c + 8, 2 c + 9, its
                    // columns [g DG, (g + 1) DG)
                    const uint32_t vb = kb0 + C::KV + u * kSub * D;
                    uint32_t vw[4][D / 32];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int row = 2 * c + (e & 1) + (e >> 1) * 8;
                        if constexpr (D == 128) {
                            const uint4 v = lds128(vb + row * D + ((g ^ (row & 7)) << 4));
                            vw[e][0] = v.x, vw[e][1] = v.y, vw[e][2] = v.z, vw[e][3] = v.w;
                        } else {
                            const uint2 v = lds64(vb + row * D + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8);
                            vw[e][0] = v.x, vw[e][1] = v.y;
                        }
                    }
#pragma unroll
                    for (int q = 0; q < D / 32; ++q) {
                        uint32_t b[2][4];
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t x0 = vw[2 * e][q] ^ 0x80808080u, x1 = vw[2 * e + 1][q] ^ 0x80808080u;
                            const uint32_t lo = __byte_perm(x0, x1, 0x5140), hi = __byte_perm(x0, x1, 0x7362);
                            b[e][0] = half2_of(lo, 0x4140);
                            b[e][1] = half2_of(lo, 0x4342);
                            b[e][2] = half2_of(hi, 0x4140);
                            b[e][3] = half2_of(hi, 0x4342);
                        }
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const uint32_t af[4] = {b[0][2 * e], b[0][2 * e + 1], b[1][2 * e], b[1][2 * e + 1]};
#pragma unroll
                            for (int z = 0; z < NR; ++z) mma16816(o[z][2 * q + e], af, pf[z][0], pf[z][1]);
                        }
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(empty_bar(stage));
            if (++stage == kStages) stage = 0, phase ^= 1u;
        }
        // ------------------------------------------------ join the four warps
#pragma unroll
        for (int z = 0; z < NR; ++z)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float s = l[z][x];
                s += __shfl_xor_sync(0xffffffffu, s, 4);
                s += __shfl_xor_sync(0xffffffffu, s, 8);
                s += __shfl_xor_sync(0xffffffffu, s, 16);
                const int row = 8 * z + 2 * c + x;
                if (g == 0) {
                    ml[warp * ROWS + row] = m[z][x];
                    ml[(kCWarps + warp) * ROWS + row] = s;
                }
                float* to = osm + (warp * ROWS + row) * C::LDO + g * DG;
#pragma unroll
                for (int j = 0; j < NO; j += 2)
                    *reinterpret_cast<float4*>(to + 2 * j) =
                        make_float4(o[z][j][x], o[z][j][2 + x], o[z][j + 1][x], o[z][j + 1][2 + x]);
            }
        asm volatile("bar.sync 1, 128;" ::: "memory");
        constexpr int CPT = ROWS * D / 128;  // columns per thread
        constexpr int TPR = D / CPT;
        const int row = threadIdx.x / TPR, col = (threadIdx.x % TPR) * CPT;
        float M = -INFINITY, L = 0.0f, acc[CPT];
#pragma unroll
        for (int e = 0; e < CPT; ++e) acc[e] = 0.0f;
#pragma unroll
        for (int x = 0; x < kCWarps; ++x) M = fmaxf(M, ml[x * ROWS + row]);
#pragma unroll
        for (int x = 0; x < kCWarps; ++x) {
            const float mx = ml[x * ROWS + row], lx = ml[(kCWarps + x) * ROWS + row];
            const float f = mx == -INFINITY ? 0.0f : ex2(mx - M);
            L += mx == -INFINITY ? lx : lx * f;
            const float* from = osm + (x * ROWS + row) * C::LDO + col;
#pragma unroll
            for (int e = 0; e < CPT; ++e) acc[e] = fmaf(from[e], f, acc[e]);
        }
        bool write = true;
        if (w.k0 != 0 || w.k1 != w.s.tiles) {
            // a part of the row tile's keys: leave it in the workspace; the
            // block that completes the count joins all parts, in range order
            constexpr int PART = ROWS * (D + 2);
            float* mine = a.part + (int64_t)(blockIdx.x * 2 + (w.first ? 0 : 1)) * PART;
#pragma unroll
            for (int e = 0; e < CPT; e += 4)
                __stcg(reinterpret_cast<float4*>(mine + row * D + col + e),
                       make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]));
            if (col == 0) {
                __stcg(mine + ROWS * D + row, M);
                __stcg(mine + ROWS * D + ROWS + row, L);
            }
            const int64_t i0 = w.it - w.k0;
            const int c_lo = w.owner_of(i0);
            asm volatile("bar.sync 1, 128;" ::: "memory");
            if (threadIdx.x == 0) {
                // (the barrier orders the block's stores before this fence, which
                // makes them visible before the count)
                __threadfence();
                const int before = atomicAdd(a.cnt + c_lo, w.k1 - w.k0);
                const bool is_last = before + (w.k1 - w.k0) == w.s.tiles;
                if (is_last) a.cnt[c_lo] = 0;  // ready for the next launch
                __threadfence();
                *last_flag = is_last;
            }
            asm volatile("bar.sync 1, 128;" ::: "memory");
            write = *last_flag != 0;
            if (write) {
                const int c_hi = w.owner_of(i0 + w.s.tiles - 1);
                // the row tile is the last piece of the range it starts in
                // (unless it starts that range), the first of the later ones
                const float* from = a.part + (int64_t)(c_lo * 2 + (w.start_of(c_lo) == i0 ? 0 : 1)) * PART;
                const int n = c_hi - c_lo + 1;
                M = -INFINITY;
                L = 0.0f;
#pragma unroll
                for (int e = 0; e < CPT; ++e) acc[e] = 0.0f;
                // four parts' loads at a time, joined in order
                constexpr int PB = 4;
#pragma unroll 1
                for (int x0 = 0; x0 < n; x0 += PB) {
                    float mp[PB], lp[PB];
                    float4 op[PB][CPT / 4];
#pragma unroll
                    for (int x = 0; x < PB; ++x) {
                        mp[x] = -INFINITY;
                        lp[x] = 0.0f;
                        if (x0 + x < n) {
                            const float* p = x0 + x == 0 ? from : a.part + (int64_t)(c_lo + x0 + x) * 2 * PART;
                            mp[x] = __ldcg(p + ROWS * D + row);
                            lp[x] = __ldcg(p + ROWS * D + ROWS + row);
#pragma unroll
                            for (int e = 0; e < CPT / 4; ++e)
                                op[x][e] = __ldcg(reinterpret_cast<const float4*>(p + row * D + col) + e);
                        } else {
#pragma unroll
                            for (int e = 0; e < CPT / 4; ++e) op[x][e] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        }
                    }
                    float to = M;
#pragma unroll
                    for (int x = 0; x < PB; ++x) to = fmaxf(to, mp[x]);
                    const float keep = M == -INFINITY ? 0.0f : ex2(M - to);
                    if (M != -INFINITY) L *= keep;  // (NaN scores leave m at -inf and l NaN)
                    M = to;
#pragma unroll
                    for (int e = 0; e < CPT; ++e) acc[e] *= keep;
#pragma unroll
                    for (int x = 0; x < PB; ++x) {
                        const float f = mp[x] == -INFINITY ? 0.0f : ex2(mp[x] - to);
                        L += mp[x] == -INFINITY ? lp[x] : lp[x] * f;
#pragma unroll
                        for (int e = 0; e < CPT / 4; ++e) {
                            acc[4 * e] = fmaf(op[x][e].x, f, acc[4 * e]);
                            acc[4 * e + 1] = fmaf(op[x][e].y, f, acc[4 * e + 1]);
                            acc[4 * e + 2] = fmaf(op[x][e].z, f, acc[4 * e + 2]);
                            acc[4 * e + 3] = fmaf(op[x][e].w, f, acc[4 * e + 3]);
                        }
                    }
                }
            }
        }
        const int r = r0 + row;
        if (write && r < rows) {
            const int i = r / a.G;
            T* y = static_cast<T*>(a.Y) + (w.s.lo + i) * a.ldy + (int64_t)(h * a.G + r - i * a.G) * D + col;
            // a row that sees no key is zero
            const float inv = (M == -INFINITY && L == 0.0f) ? 0.0f : __frcp_rn(L);
            uint32_t p[CPT / 2];
#pragma unroll
            for (int e = 0; e < CPT / 2; ++e)
                p[e] = (uint32_t)to16<T>(acc[2 * e] * inv) | ((uint32_t)to16<T>(acc[2 * e + 1] * inv) << 16);
            if constexpr (CPT == 4) {
                *reinterpret_cast<uint2*>(y) = make_uint2(p[0], p[1]);
            } else {
#pragma unroll
                for (int e = 0; e < CPT / 8; ++e)
                    reinterpret_cast<uint4*>(y)[e] = make_uint4(p[4 * e], p[4 * e + 1], p[4 * e + 2], p[4 * e + 3]);
            }
        }
        // the next piece writes the shared O and the flag again
        asm volatile("bar.sync 1, 128;" ::: "memory");
    }
}

// Counters at a fixed place for every size, one per block of the largest grid.
constexpr int kMaxGrid = 1024;
constexpr size_t kCntBytes = kMaxGrid * sizeof(int);
static_assert(kCntBytes % 256 == 0, "the parts start 256-byte aligned");

int attention_grid(int nr) {
    const int g = ctas_per_sm(nr) * num_sms();
    return g < kMaxGrid ? g : kMaxGrid;
}

template <typename T, int D, int NR>
sq_status_t launch_rows(const char* name, const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a,
                        cudaStream_t stream) {
    using C = ACfg<D, NR>;
    auto fn = kv8_attention_kernel<T, D, NR>;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)C::SMEM_ALLOC) != cudaSuccess)
        return check_launch(name);
    launch_pdl(fn, dim3(attention_grid(NR)), dim3(kThreadsA), C::SMEM_ALLOC, stream, mk, mv, a);
    return check_launch(name);
}

template <typename T, int D>
sq_status_t launch_attention(const char* name, const CUtensorMap& mk, const CUtensorMap& mv, const AttnArgs& a,
                             int64_t max_q, cudaStream_t stream) {
    if (max_q * a.G <= 8) return launch_rows<T, D, 1>(name, mk, mv, a, stream);
    return launch_rows<T, D, 2>(name, mk, mv, a, stream);
}

}  // namespace

size_t kv8_attention_workspace_bytes(int64_t T, int64_t Hq, int64_t D) {
    if (T <= 0 || Hq <= 0 || D <= 0) return kStatusBytes;
    size_t part = 0;
    for (int nr = 1; nr <= 2; ++nr) {
        const size_t n = (size_t)attention_grid(nr) * 2 * (8 * nr) * (size_t)(D + 2) * sizeof(float);
        part = n > part ? n : part;
    }
    // (a sequence has at most T * Hq rows of a head)
    if (T * Hq > kRowLimit) {
        const size_t n = kv8_prefill_part_bytes(D);
        part = n > part ? n : part;
    }
    return kStatusBytes + kCntBytes + part;
}

}  // namespace sq

extern "C" sq_status_t sq_kv8_attention(const void* Q, sq_dtype_t dt, int64_t T, int64_t Hq, int64_t Hkv, int64_t D,
                                        int64_t ldq, const int8_t* Kc, const int8_t* Vc, const float* kqs,
                                        const float* vqs, int64_t num_blocks, int64_t block, const int32_t* cu_q,
                                        const int32_t* seq_lens, int64_t B, const int32_t* block_table,
                                        int64_t max_blocks, int64_t ldb, float scale, int causal, int64_t max_q, void* Y,
                                        int64_t ldy, void* workspace, size_t ws_bytes, sq_stream_t stream) {
    const char* name = "sq_kv8_attention";
    SQ_REQUIRE(dt == SQ_F16 || dt == SQ_BF16, SQ_ERR_INVALID_ARG, "%s: dtype must be F16 or BF16", name);
    const sq_status_t st = sq::check_kv8(name, T, B, Hkv, D, block, num_blocks, max_blocks, ldb);
    if (st != SQ_OK) return st;
    SQ_REQUIRE(Hq > 0 && Hq % Hkv == 0 && Hq <= 65535, SQ_ERR_UNSUPPORTED_SHAPE,
               "%s: Hq must be a multiple of Hkv", name);
    SQ_REQUIRE(ldq >= Hq * D && ldy >= Hq * D, SQ_ERR_UNSUPPORTED_SHAPE, "%s: token strides must be >= Hq * D", name);
    SQ_REQUIRE(T * Hq < (1ll << 31) - 65536, SQ_ERR_UNSUPPORTED_SHAPE, "%s: tokens x heads must be < 2^31", name);
    SQ_REQUIRE(max_q >= 0, SQ_ERR_INVALID_ARG, "%s: max_q must be >= 0", name);
    if (T == 0 || B == 0) return SQ_OK;
    SQ_REQUIRE(Q && Kc && Vc && kqs && vqs && cu_q && seq_lens && block_table && Y, SQ_ERR_INVALID_ARG,
               "%s: null pointer", name);
    SQ_REQUIRE(sq::aligned16(Q) && sq::aligned16(Y) && sq::aligned16(Kc) && sq::aligned16(Vc) && ldq % 8 == 0 &&
                   ldy % 8 == 0,
               SQ_ERR_ALIGNMENT, "%s: Q, Y, the caches and token strides must be 16-byte aligned", name);
    SQ_REQUIRE(workspace && ws_bytes >= sq::kv8_attention_workspace_bytes(T, Hq, D), SQ_ERR_INVALID_ARG,
               "%s: needs a workspace of %zu bytes", name, sq::kv8_attention_workspace_bytes(T, Hq, D));
    SQ_REQUIRE(sq::aligned16(workspace), SQ_ERR_ALIGNMENT, "%s: the workspace must be 16-byte aligned", name);
    sq::AttnArgs a;
    memset(&a, 0, sizeof(a));
    a.Q = Q;
    a.Y = Y;
    a.ldq = ldq;
    a.ldy = ldy;
    a.T = T;
    a.ldb = ldb;
    a.num_blocks = num_blocks;
    a.cu = cu_q;
    a.lens = seq_lens;
    a.table = block_table;
    a.kqs = kqs;
    a.vqs = vqs;
    a.B = (int)B;
    a.Hkv = (int)Hkv;
    a.G = (int)(Hq / Hkv);
    a.block = (int)block;
    a.block_log2 = block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
    a.box = (int)(block < 64 ? block : 64);
    a.max_blocks = (int)max_blocks;
    a.causal = causal != 0;
    a.scale = scale;
    a.status = static_cast<int*>(workspace);
    a.cnt_bytes = (int)sq::kCntBytes;
    a.cnt = reinterpret_cast<int*>(static_cast<uint8_t*>(workspace) + sq::kStatusBytes);
    a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + sq::kStatusBytes + sq::kCntBytes);
    CUtensorMap mk, mv;
    if (!sq::make_map_kv(&mk, Kc, num_blocks, Hkv * block, D, a.box, true) ||
        !sq::make_map_kv(&mv, Vc, num_blocks, Hkv * block, D, a.box, true))
        return sq::set_error(SQ_ERR_CUDA, "%s: cuTensorMapEncodeTiled failed", name);
    cudaStream_t s = sq::as_cuda(stream);
    // prompts and single tokens may share a batch: each kernel takes its
    // sequences; without long ones (as the caller says) one kernel takes all
    a.row_limit = INT64_MAX;
    if (max_q > sq::kRowLimit / a.G) {
        a.row_limit = sq::kRowLimit;
        const sq_status_t ps = sq::launch_kv8_prefill(name, dt, D, Kc, Vc, a, s);
        if (ps != SQ_OK) return ps;
    }
    if (dt == SQ_BF16)
        return D == 128 ? sq::launch_attention<__nv_bfloat16, 128>(name, mk, mv, a, max_q, s)
                        : sq::launch_attention<__nv_bfloat16, 64>(name, mk, mv, a, max_q, s);
    return D == 128 ? sq::launch_attention<__half, 128>(name, mk, mv, a, max_q, s)
                    : sq::launch_attention<__half, 64>(name, mk, mv, a, max_q, s);
}
