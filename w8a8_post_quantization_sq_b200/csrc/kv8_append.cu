// New tokens' K and V into the paged int8 cache, one scale per block of tokens
// and head.
//
// For block j of a sequence and head h, with `kept` tokens in it before the
// call and a = max |x| over the new tokens that enter it:
//   qs' = fl(127 fl(1 / max(a, 1e-8))), and min(qs, that) where kept > 0
//   new codes      = rne(x qs') clipped to +-127
//   codes of kept  = rne(code fl(qs' / qs)) where qs' < qs, else as they were
// so a block's scale always covers every token in it, and a call that enters a
// fresh block (kept = 0) never looks at what its memory held before.
//
// One warp takes one (block, head, K or V): it is the only writer of that part,
// so there are no atomics and the result depends on nothing but the inputs.
// Warps are dealt to spans of `span` flattened tokens and pick the tokens that
// start a block (or a sequence) there; up to 8 x 512 bytes of the tokens stay in
// registers between the maximum and the codes.
// What bounds it: the chain of dependent loads (sequence range, length, block
// number, scale), all of it for single tokens (64 of them: 3.3 us); for prompts a
// warp's loads of its tokens wait behind it, and the copies run at half the copy
// rate (4 of up to 2048 tokens, 8 heads of 128: 10.6 us, 3.3 TB/s, 5.4 us of bytes).
#include "sq_common.cuh"
#include "sq_kv8.cuh"

namespace sq {
namespace {

constexpr int kWarps = 4;

struct AppendArgs {
    const void* src[2];  // K, V
    int64_t ld[2];
    int8_t* codes[2];
    float* qs[2];
    const int32_t* cu;
    const int32_t* lens;
    const int32_t* table;
    int64_t T, ldb, num_blocks;
    int B, Hkv, block, max_blocks, span;
};

template <typename T>
__device__ __forceinline__ float from_bits16(uint32_t b) {
    if constexpr (std::is_same<T, __nv_bfloat16>::value) return __uint_as_float(b << 16);
    else return __half2float(__ushort_as_half((unsigned short)b));
}

// The codes of `kept` tokens (contiguous bytes) times r.
__device__ __forceinline__ void rescale(int8_t* codes, int bytes, float r, int lane) {
    for (int i = lane * 16; i < bytes; i += 512) {
        uint4 w = *reinterpret_cast<const uint4*>(codes + i);
        uint32_t* p = reinterpret_cast<uint32_t*>(&w);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            uint32_t q[4];
#pragma unroll
            for (int b = 0; b < 4; ++b) q[b] = quant_bits_clip(__fmul_rn((float)(int8_t)(p[e] >> (8 * b)), r));
            p[e] = pack_low_bytes(q[0], q[1], q[2], q[3]);
        }
        *reinterpret_cast<uint4*>(codes + i) = w;
    }
}

// nt new tokens (rows of D elements, stride ld) into rows kept.. of one head's
// part of a block.
template <typename T, int D>
__device__ __forceinline__ void fill_block(const T* src, int64_t ld, int nt, int kept, int8_t* codes, float* qs, int lane) {
    constexpr int LPT = D / 8;     // lanes per token
    constexpr int TPP = 32 / LPT;  // tokens per pass
    constexpr int NP = 8;          // passes held in registers
    constexpr uint32_t kInf16 = std::is_same<T, __nv_bfloat16>::value ? 0x7f80u : 0x7c00u;
    const int sub = lane / LPT, col = (lane % LPT) * 8;
    const float old = kept > 0 ? *qs : 0.0f;
    uint4 r[NP];
    auto load = [&](int base) {
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int tok = base + i * TPP + sub;
            r[i] = tok < nt ? *reinterpret_cast<const uint4*>(src + (int64_t)tok * ld + col) : make_uint4(0, 0, 0, 0);
        }
    };
    uint32_t m2 = 0;
    for (int base = 0; base < nt; base += NP * TPP) {
        load(base);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            m2 = __vmaxu2(m2, __vmaxu2(r[i].x & 0x7fff7fffu, r[i].y & 0x7fff7fffu));
            m2 = __vmaxu2(m2, __vmaxu2(r[i].z & 0x7fff7fffu, r[i].w & 0x7fff7fffu));
        }
    }
    const uint32_t m = __reduce_max_sync(0xffffffffu, max(m2 & 0xffffu, m2 >> 16));
    float now = __fmul_rn(127.0f, __frcp_rn(fmaxf(from_bits16<T>(m), 1e-8f)));
    if (m >= kInf16 || (kept > 0 && old != old)) now = __uint_as_float(0x7fffffffu);
    else if (kept > 0) now = fminf(now, old);
    if (kept > 0 && now < old) rescale(codes, kept * D, __fdiv_rn(now, old), lane);
    for (int base = 0; base < nt; base += NP * TPP) {
        if (nt > NP * TPP) load(base);
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            const int tok = base + i * TPP + sub;
            if (tok < nt) {
                float v[8];
                unpack<T>(r[i], v);
                uint32_t b[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) b[e] = quant_bits_clip(__fmul_rn(v[e], now));
                *reinterpret_cast<uint2*>(codes + (int64_t)(kept + tok) * D + col) =
                    make_uint2(pack_low_bytes(b[0], b[1], b[2], b[3]), pack_low_bytes(b[4], b[5], b[6], b[7]));
            }
        }
    }
    if (lane == 0) *qs = now;
}

template <typename T, int D>
__global__ void __launch_bounds__(kWarps * 32) kv8_append_kernel(const AppendArgs a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31;
    const int64_t unit = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int per = 2 * a.Hkv;
    const int64_t t0 = unit / per * a.span;
    if (t0 >= a.T) return;
    const int hv = (int)(unit % per);
    const int h = hv >> 1, kv = hv & 1;
    const int64_t t1 = min(t0 + a.span, a.T);
    int b = kv8_sequence_of(a.cu, a.B, t0, lane);
    int64_t t = t0;
    while (t < t1 && b < a.B) {
        const int64_t lo = __ldg(a.cu + b), hi = min((int64_t)__ldg(a.cu + b + 1), a.T);
        if (t >= hi) {
            ++b;
            continue;
        }
        if (t < lo) {
            t = lo;
            continue;
        }
        const int64_t pos = __ldg(a.lens + b) - (hi - t);
        // a length that does not hold the sequence's new tokens: nothing is written
        if (pos < t - lo || pos >= (int64_t)a.max_blocks * a.block) {
            t = hi;
            continue;
        }
        const int j = (int)(pos / a.block), kept = (int)(pos - (int64_t)j * a.block);
        const int64_t end = min(hi, t + a.block - kept);
        if (t == lo || kept == 0) {
            const int64_t blk = __ldg(a.table + (int64_t)b * a.ldb + j);
            if (blk >= 0 && blk < a.num_blocks) {
                const int64_t part = blk * a.Hkv + h;
                fill_block<T, D>(static_cast<const T*>(a.src[kv]) + t * a.ld[kv] + (int64_t)h * D, a.ld[kv],
                                 (int)(end - t), kept, a.codes[kv] + part * a.block * D, a.qs[kv] + part, lane);
            }
        }
        t = end;
    }
}

}  // namespace

sq_status_t check_kv8(const char* name, int64_t T, int64_t B, int64_t Hkv, int64_t D, int64_t block, int64_t num_blocks,
                      int64_t max_blocks, int64_t ldb) {
    SQ_REQUIRE(T >= 0 && B >= 0 && Hkv > 0 && num_blocks > 0 && max_blocks > 0 && ldb >= max_blocks,
               SQ_ERR_UNSUPPORTED_SHAPE, "%s: need T, B >= 0, heads, blocks > 0, table stride >= max_blocks", name);
    SQ_REQUIRE(D == 64 || D == 128, SQ_ERR_UNSUPPORTED_SHAPE, "%s: head width must be 64 or 128", name);
    SQ_REQUIRE(block == 16 || block == 32 || block == 64 || block == 128, SQ_ERR_UNSUPPORTED_SHAPE,
               "%s: block must be 16, 32, 64 or 128 tokens", name);
    SQ_REQUIRE(T < (1ll << 31) && B < (1ll << 24) && Hkv <= 65535 && num_blocks < (1ll << 31) &&
                   max_blocks * block < (1ll << 31),
               SQ_ERR_UNSUPPORTED_SHAPE, "%s: tokens, blocks and a sequence's positions must be < 2^31", name);
    return SQ_OK;
}

}  // namespace sq

extern "C" sq_status_t sq_kv8_append(const void* Kn, const void* Vn, sq_dtype_t dt, int64_t T, int64_t Hkv, int64_t D,
                                     int64_t ldk, int64_t ldv, const int32_t* cu_q, const int32_t* seq_lens, int64_t B,
                                     const int32_t* block_table, int64_t max_blocks, int64_t ldb, int8_t* Kc,
                                     int8_t* Vc, float* kqs, float* vqs, int64_t num_blocks, int64_t block,
                                     sq_stream_t stream) {
    const char* name = "sq_kv8_append";
    SQ_REQUIRE(dt == SQ_F16 || dt == SQ_BF16, SQ_ERR_INVALID_ARG, "%s: dtype must be F16 or BF16", name);
    const sq_status_t st = sq::check_kv8(name, T, B, Hkv, D, block, num_blocks, max_blocks, ldb);
    if (st != SQ_OK) return st;
    SQ_REQUIRE(ldk >= Hkv * D && ldv >= Hkv * D, SQ_ERR_UNSUPPORTED_SHAPE, "%s: token strides must be >= Hkv * D", name);
    if (T == 0 || B == 0) return SQ_OK;
    SQ_REQUIRE(Kn && Vn && cu_q && seq_lens && block_table && Kc && Vc && kqs && vqs, SQ_ERR_INVALID_ARG,
               "%s: null pointer", name);
    SQ_REQUIRE(sq::aligned16(Kn) && sq::aligned16(Vn) && sq::aligned16(Kc) && sq::aligned16(Vc) && ldk % 8 == 0 &&
                   ldv % 8 == 0,
               SQ_ERR_ALIGNMENT, "%s: K, V, the caches and token strides must be 16-byte aligned", name);
    sq::AppendArgs a;
    a.src[0] = Kn;
    a.src[1] = Vn;
    a.ld[0] = ldk;
    a.ld[1] = ldv;
    a.codes[0] = Kc;
    a.codes[1] = Vc;
    a.qs[0] = kqs;
    a.qs[1] = vqs;
    a.cu = cu_q;
    a.lens = seq_lens;
    a.table = block_table;
    a.T = T;
    a.ldb = ldb;
    a.num_blocks = num_blocks;
    a.B = (int)B;
    a.Hkv = (int)Hkv;
    a.block = (int)block;
    a.max_blocks = (int)max_blocks;
    // a warp per token where sequences bring a few tokens each (every token
    // starts a part), spans of a block's length for prompts
    a.span = T <= 4 * B ? 1 : T < 256 * B ? 4 : 16;
    const int64_t units = (T + a.span - 1) / a.span * 2 * Hkv;
    const int64_t grid = (units + sq::kWarps - 1) / sq::kWarps;
    SQ_REQUIRE(grid < (1ll << 31), SQ_ERR_UNSUPPORTED_SHAPE, "%s: too many tokens and heads", name);
    const dim3 g((unsigned)grid), t(sq::kWarps * 32);
    cudaStream_t s = sq::as_cuda(stream);
    if (dt == SQ_BF16 && D == 64) sq::launch_pdl(sq::kv8_append_kernel<__nv_bfloat16, 64>, g, t, 0, s, a);
    else if (dt == SQ_BF16) sq::launch_pdl(sq::kv8_append_kernel<__nv_bfloat16, 128>, g, t, 0, s, a);
    else if (D == 64) sq::launch_pdl(sq::kv8_append_kernel<__half, 64>, g, t, 0, s, a);
    else sq::launch_pdl(sq::kv8_append_kernel<__half, 128>, g, t, 0, s, a);
    return sq::check_launch(name);
}
