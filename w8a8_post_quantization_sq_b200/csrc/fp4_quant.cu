// Microscaled 4-bit quantisation (NVFP4 and MXFP4) and its inverse.
//
// Quantisation of a row v (fp32; X, X / s or W * s):
//   NVFP4: qs = 2^(10 - floor(log2 max|v|)) over the row (or a given scale),
//          u = fl(v qs); per 16: b = E4M3(fl(max|u| / 6)), code = E2M1(fl(u / b))
//   MXFP4: per 32: b = 2^(floor(log2 max|v|) - 2), code = E2M1(v / b)
// every rounding to nearest, ties to even, magnitudes past the format's largest
// saturated. The row scale is a power of two because a power of two changes no
// mantissa: u and the code decisions are those of the unscaled row, and E4M3's
// range (2^-9 .. 448) is placed so that the row's largest block scale lies in
// [170, 342).
// A block holding a NaN or an infinity gets the NaN scale (0x7F, 0xFF) and zero
// codes, so a product with it gives NaN; the row scale looks at finite values.
//
// One pass over memory: TPR threads share a row, each holding up to four units
// of 16 elements in registers between the row maximum and the codes, 16-bit
// inputs as they came (held as fp32, three units took 109 registers and two
// blocks per SM: 4096 x 12288 bf16 65 us). Rows too wide for that (over 32768
// elements; 49152 of 16 bits) are read twice, the second time from L2.
// What bounds it, at 4096 x 12288 (us, of them the bytes at 6.54 TB/s): quantisation
// the bytes and the codes' arithmetic between them, bf16 to NVFP4 26.8 (19.7), to MXFP4
// 21.4 (19.5), fp32 44.8 (35.1) and 34.4 (34.9); with a smoothing scale the fp32
// values held and, for activations, a division each (bf16 to NVFP4 80.4 with 1 / s, 57.8
// with s; to MXFP4 54.1 and 39.5). Dequantisation to bf16 24.2 (19.7). Few rows: the
// launch and one chain of loads (16 x 4096: 2.9 and 1.6).
#include <cuda_fp8.h>

#include "sq_common.cuh"
#include "sq_fp4.cuh"

namespace sq {
namespace {

enum Smooth { kNone = 0, kMul = 1, kDiv = 2 };
constexpr uint32_t kInfBits = 0x7f800000u;
constexpr float kMaxF32 = 0x1.fffffep+127f;

// 32 bytes a lane: a warp's access then covers whole 32-byte sectors, which two
// accesses of 16 bytes touch twice (4096 x 12288: dequantisation 29.7 -> 25.5 us,
// quantisation of fp32 56.7 -> 49.0 us). `wide`: the address is 32-byte aligned.
__device__ __forceinline__ void load32(const void* p, bool wide, uint32_t* r) {
    if (wide) {
        asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p));
    } else {
        const uint4 a = ldg_nc_v4(p), b = ldg_nc_v4(static_cast<const uint8_t*>(p) + 16);
        r[0] = a.x, r[1] = a.y, r[2] = a.z, r[3] = a.w;
        r[4] = b.x, r[5] = b.y, r[6] = b.z, r[7] = b.w;
    }
}
__device__ __forceinline__ void store32(void* p, bool wide, const uint32_t* r) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]),
                     "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                     : "memory");
    } else {
        __stcs(static_cast<uint4*>(p), make_uint4(r[0], r[1], r[2], r[3]));
        __stcs(static_cast<uint4*>(p) + 1, make_uint4(r[4], r[5], r[6], r[7]));
    }
}

// 16 consecutive elements as they are held between the passes: the 16-bit
// words, or fp32 values (fp32 inputs, and smoothed ones, which have no 16-bit
// form).
template <typename T, int SM>
struct Unit {
    static constexpr bool RAW = sizeof(T) == 2 && SM == kNone;
    uint32_t w[RAW ? 8 : 16];

    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int e = 0; e < (RAW ? 8 : 16); ++e) w[e] = 0u;
    }
    __device__ __forceinline__ void load(const T* row, const float* s, int64_t k, bool wide) {
        if constexpr (RAW) {
            load32(row + k, wide, w);
        } else {
            float v[16];
            uint32_t r[16];
            load32(row + k, wide, r);
            if constexpr (sizeof(T) == 4) {
                load32(row + k + 8, wide, r + 8);
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(r[e]);
            } else {
                unpack<T>(make_uint4(r[0], r[1], r[2], r[3]), v);
                unpack<T>(make_uint4(r[4], r[5], r[6], r[7]), v + 8);
            }
            if constexpr (SM != kNone) {
                const float4* s4 = reinterpret_cast<const float4*>(s + k);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 f = __ldg(s4 + i);
                    const float sv[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        v[4 * i + e] = SM == kMul ? __fmul_rn(v[4 * i + e], sv[e]) : __fdiv_rn(v[4 * i + e], sv[e]);
                }
            }
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(v[e]);
        }
    }
    __device__ __forceinline__ void values(float* v) const {
        if constexpr (RAW) {
            unpack<T>(make_uint4(w[0], w[1], w[2], w[3]), v);
            unpack<T>(make_uint4(w[4], w[5], w[6], w[7]), v + 8);
        } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = __uint_as_float(w[e]);
        }
    }
    // Largest |v| as fp32 bits: kInfBits and above if a value is not finite (bit
    // patterns of non-negative floats order as the floats do, infinities and
    // NaN above every finite value).
    __device__ __forceinline__ uint32_t absmax_bits() const {
        if constexpr (RAW) {
            uint32_t m[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) m[e] = __vmaxu2(w[e] & 0x7fff7fffu, w[e + 4] & 0x7fff7fffu);
            m[0] = __vmaxu2(__vmaxu2(m[0], m[1]), __vmaxu2(m[2], m[3]));
            float f[8];
            unpack<T>(make_uint4(max(m[0] & 0xffffu, m[0] >> 16), 0, 0, 0), f);
            return __float_as_uint(f[0]);
        } else {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 16; ++e) m = max(m, w[e] & 0x7fffffffu);
            return m;
        }
    }
    // The same over the finite values alone.
    __device__ __forceinline__ uint32_t finite_bits() const {
        float v[16];
        values(v);
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 16; ++e) {
            const uint32_t b = __float_as_uint(v[e]) & 0x7fffffffu;
            if (b < kInfBits) m = max(m, b);
        }
        return m;
    }
};

// 2^(10 - floor(log2 m)); m below 2^-100 counts as 2^-100, so the scale and its
// reciprocal stay normal.
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
    const int field = max((int)(amax_bits >> 23), 27);
    return __uint_as_float((uint32_t)(264 - field) << 23);
}

// Eight values to the nearest E2M1 (ties to even, saturated), the first in the
// lowest four bits.
__device__ __forceinline__ uint32_t e2m1x8(const float* t) {
    uint32_t w;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}"
        : "=r"(w)
        : "f"(t[0]), "f"(t[1]), "f"(t[2]), "f"(t[3]), "f"(t[4]), "f"(t[5]), "f"(t[6]), "f"(t[7]));
    return w;
}

// Eight codes of fl(u / b), inv = fl(1 / b). The quotient is rounded correctly
// by one residual step (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990: with inv the correctly rounded
// reciprocal, q = fl(u inv), r = u - q b exactly, fl(q + r inv) is the rounded
// quotient), because a quotient that lies on the border between two codes is
// common (u and b have few bits) and must go to the even code.
__device__ __forceinline__ uint32_t codes8(const float* u, float b, float inv) {
    float t[8];
    const uint64_t nb2 = pk2(-b, -b), inv2 = pk2(inv, inv);
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
        const uint64_t u2 = pk2(u[e], u[e + 1]);
        const uint64_t q2 = mul2(u2, inv2);
        upk2(fma2(fma2(q2, nb2, u2), inv2, q2), t[e], t[e + 1]);
    }
    return e2m1x8(t);
}

struct QuantArgs {
    const void* X;
    const float* s;
    const float* static_qs;
    uint8_t* codes;
    uint8_t* scales;
    float* qs;
    int64_t rows, K, ld, tiles_k, pad_rows;
    int units;  // K / 16
    bool wide;  // rows start on 32-byte boundaries
};

// Codes and scale of one unit of the row whose codes and first scale tile's
// words are at `codes` and `scales`. bits: |v| maximum of the unit. Every lane of
// the warp calls this (valid = 0 past the row's end).
template <int FMT>
__device__ __forceinline__ void emit_unit(const QuantArgs& a, uint8_t* codes, uint8_t* scales, int unit, bool valid,
                                          float* v, uint32_t bits, float qs) {
    uint32_t byte;
    uint2 w;
    if constexpr (FMT == SQ_NVFP4) {
        // (a given scale may carry finite values past fp32's largest: held there,
        // they saturate below, where an infinity would make NaN of the residuals)
        const float top = fminf(__fmul_rn(__uint_as_float(bits), qs), kMaxF32);
        // fl(top / 6), the quotient rounded as in codes8
        float sixth = __fmul_rn(top, 0x1.555556p-3f);
        sixth = __fmaf_rn(__fmaf_rn(sixth, -6.0f, top), 0x1.555556p-3f, sixth);
        byte = __nv_cvt_float_to_fp8(sixth, __NV_SATFINITE, __NV_E4M3);
        const bool finite = bits < kInfBits;
        if (!finite) byte = 0x7Fu;
        float b = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
        float inv = byte == 0 ? 0.0f : __frcp_rn(b);
        if (a.static_qs) {
            const uint64_t qs2 = pk2(qs, qs);
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
                upk2(mul2(pk2(v[e], v[e + 1]), qs2), v[e], v[e + 1]);
                v[e] = fminf(fmaxf(v[e], -kMaxF32), kMaxF32);
                v[e + 1] = fminf(fmaxf(v[e + 1], -kMaxF32), kMaxF32);
            }
        } else {
            // qs is a power of two: u / b is v / (b / qs), with the same bits
            inv = __fmul_rn(inv, qs);
            b = __fmul_rn(b, __uint_as_float(0x7f000000u - __float_as_uint(qs)));
        }
        w = make_uint2(codes8(v, b, inv), codes8(v + 8, b, inv));
        if (!finite) w = make_uint2(0, 0);
    } else {
        // a block of 32 is two neighbouring lanes' units (K is a multiple of 32)
        bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
        const bool finite = bits < kInfBits;
        byte = (uint32_t)max((int)(bits >> 23) - 2, 0);
        const float up = __uint_as_float((254u - byte) << 23);  // 1 / b, exact, as every product with it
        const uint64_t up2 = pk2(up, up);
#pragma unroll
        for (int e = 0; e < 16; e += 2) upk2(mul2(pk2(v[e], v[e + 1]), up2), v[e], v[e + 1]);
        w = finite ? make_uint2(e2m1x8(v), e2m1x8(v + 8)) : make_uint2(0, 0);
        if (!finite) byte = 0xFFu;
    }
    if (!valid) byte = 0;
    else *reinterpret_cast<uint2*>(codes + (uint32_t)unit * 8u) = w;
    // four blocks' scales are one word of the tile
    constexpr int G = FMT == SQ_NVFP4 ? 4 : 8;  // lanes per word
    const int lane = threadIdx.x & 31;
    uint32_t word;
    if constexpr (FMT == SQ_NVFP4) {
        word = byte << (8 * (lane & 3));
    } else {
        word = (lane & 1) ? 0u : byte << (8 * ((lane >> 1) & 3));
        word |= __shfl_xor_sync(0xffffffffu, word, 4);
    }
    word |= __shfl_xor_sync(0xffffffffu, word, 1);
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    if (valid && (lane & (G - 1)) == 0)
        *reinterpret_cast<uint32_t*>(scales + (uint32_t)(unit / G) * (uint32_t)kFp4TileBytes) = word;
}

// Row maximum over the 2^tl threads (32 to 512) of this row.
__device__ __forceinline__ uint32_t row_max(uint32_t m, int tl, uint32_t* sh) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (tl > 5) {
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, per = 1 << (tl - 5);
        if (lane == 0) sh[warp] = m;
        __syncthreads();
        m = __reduce_max_sync(0xffffffffu, sh[(warp & ~(per - 1)) + (lane & (per - 1))]);
    }
    return m;
}

// UPT units per thread held in registers; UPT = 0: any width, read twice. Blocks
// of BT threads, one round of rows each. (Blocks that go over many rows and fetch
// the next row ahead measured slower, 33 against 30 us at 4096 x 12288: the
// second row's registers cost warps, and it is the warps that hide the chain
// from a block's maximum to its codes.)
template <typename T, int FMT, int SM, int UPT, int BT>
__global__ void __launch_bounds__(BT, (Unit<T, SM>::RAW && UPT <= 4 ? 1024 : 512) / BT)
quantize_fp4_kernel(const QuantArgs a, int tl) {
    __shared__ uint32_t sh[16];
    pdl_wait();
    pdl_trigger();
    const int tpr = 1 << tl;  // threads per row
    const int64_t row = (int64_t)blockIdx.x * (BT >> tl) + (threadIdx.x >> tl);
    const int t = threadIdx.x & (tpr - 1);
    const bool live = row < a.rows;  // the same for a whole warp
    uint8_t* const codes = a.codes + row * (a.K >> 1);
    uint8_t* const scales = a.scales + fp4_scale_offset(row, 0, a.tiles_k);
    if (row >= a.rows && row < a.pad_rows)
        // rows that fill up the last tile: zero scales
        for (int64_t k = t; k < a.tiles_k; k += tpr)
            *reinterpret_cast<uint32_t*>(scales + k * kFp4TileBytes) = 0u;
    const T* x = static_cast<const T*>(a.X) + (live ? row : 0) * a.ld;
    float qs = 1.0f;
    if constexpr (UPT > 0) {
        Unit<T, SM> v[UPT];
        uint32_t bits[UPT];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int u = t + i * tpr;
            if (live && u < a.units) v[i].load(x, a.s, (int64_t)u * 16, a.wide);
            else v[i].clear();
        }
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            bits[i] = v[i].absmax_bits();
            m = max(m, bits[i]);
        }
        if (FMT == SQ_NVFP4 && m >= kInfBits) {
            m = 0;
#pragma unroll 1
            for (int i = 0; i < UPT; ++i) {
                // (not held, but read again: a value that is not finite is rare)
                const int u = t + i * tpr;
                Unit<T, SM> z;
                z.load(x, a.s, (int64_t)(u < a.units ? u : 0) * 16, a.wide);
                if (u < a.units) m = max(m, z.finite_bits());
            }
        }
        if constexpr (FMT == SQ_NVFP4) {
            if (a.static_qs) qs = *a.static_qs;
            else qs = row_scale(row_max(m, tl, sh));
        }
        if (!live) return;
#pragma unroll
        for (int i = 0; i < UPT; ++i)
            if (i * tpr < a.units) {
                float f[16];
                v[i].values(f);
                emit_unit<FMT>(a, codes, scales, t + i * tpr, t + i * tpr < a.units, f, bits[i], qs);
            }
    } else {
        Unit<T, SM> v;
        if constexpr (FMT == SQ_NVFP4) {
            uint32_t m = 0;
            if (!a.static_qs && live)
                for (int u = t; u < a.units; u += tpr) {
                    v.load(x, a.s, (int64_t)u * 16, a.wide);
                    m = max(m, v.finite_bits());
                }
            if (a.static_qs) qs = *a.static_qs;
            else qs = row_scale(row_max(m, tl, sh));
        }
        if (!live) return;
        for (int u0 = 0; u0 < a.units; u0 += tpr) {
            const int u = u0 + t;
            if (u < a.units) v.load(x, a.s, (int64_t)u * 16, a.wide);
            else v.clear();
            float f[16];
            v.values(f);
            emit_unit<FMT>(a, codes, scales, u, u < a.units, f, v.absmax_bits(), qs);
        }
    }
    if (FMT == SQ_NVFP4 && a.qs && t == 0) a.qs[a.static_qs ? 0 : row] = qs;
}

// value = fl(fl(code b) fl(1 / qs)), the first product exact; one rounding to T.
template <typename T, int FMT>
__global__ void __launch_bounds__(256)
dequantize_fp4_kernel(const uint8_t* codes, const uint8_t* scales, const float* qs, int per_row, int64_t rows, int64_t K,
                      int64_t tiles_k, int tl, T* Y, int64_t ldy, bool wide) {
    pdl_wait();
    pdl_trigger();
    const int64_t row = (int64_t)blockIdx.x * (256 >> tl) + (threadIdx.x >> tl);
    const int u = ((int)blockIdx.y << tl) + (threadIdx.x & ((1 << tl) - 1));
    if (row >= rows || u >= (int)(K >> 4)) return;
    const uint2 w = __ldcs(reinterpret_cast<const uint2*>(codes + row * (K >> 1) + (int64_t)u * 8));
    constexpr int G = FMT == SQ_NVFP4 ? 4 : 8;
    const uint8_t byte = scales[fp4_scale_offset(row, u / G, tiles_k) + (FMT == SQ_NVFP4 ? (u & 3) : ((u >> 1) & 3))];
    const float rq = qs ? __frcp_rn(qs[per_row ? row : 0]) : 1.0f;
    float b;
    if constexpr (FMT == SQ_NVFP4) {
        b = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
    } else {
        b = byte == 0xFFu ? __uint_as_float(0x7fffffffu)
                          : byte == 0 ? __uint_as_float(0x00400000u) : __uint_as_float((uint32_t)byte << 23);
    }
    // As fp16 the values of E2M1 differ in their upper bytes only: four codes'
    // bytes come from a table of eight by one byte permute (the conversion
    // instruction runs at an eighth of that rate), the signs from a second one,
    // which repeats the top bit of 0x80 where a selector's own top bit is set.
    float y[16];
    const uint64_t b2 = pk2(b, b), rq2 = pk2(rq, rq);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint32_t c = e & 1 ? (e < 2 ? w.x : w.y) >> 16 : (e < 2 ? w.x : w.y);  // four codes
        const uint32_t mag = __byte_perm(0x3e3c3800u, 0x46444240u, c & 0x7777u);
        uint32_t sign;
        asm("prmt.b32 %0, %1, %1, %2;" : "=r"(sign) : "r"(0x80808080u), "r"(c));
        sign <<= 1;
        const uint32_t hi = mag | (sign & 0x80808080u);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
            const uint32_t h2 = __byte_perm(hi, 0u, q ? 0x3424 : 0x1404);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h2));
            upk2(mul2(mul2(pk2(f.x, f.y), b2), rq2), y[4 * e + 2 * q], y[4 * e + 2 * q + 1]);
        }
    }
    T* out = Y + row * ldy + (int64_t)u * 16;
    if constexpr (sizeof(T) == 4) {
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) p[e] = __float_as_uint(y[e]);
        store32(out, wide, p);
        store32(out + 8, wide, p + 8);
    } else {
        uint32_t p[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) p[e] = (uint32_t)to16<T>(y[2 * e]) | ((uint32_t)to16<T>(y[2 * e + 1]) << 16);
        store32(out, wide, p);
    }
}

// Threads per row (log2): the fewest that hold the row in at most four units of
// 16 each, 32 to 512.
int threads_per_row_log2(int64_t units) {
    int tl = 5;
    while (tl < 9 && units > (4ll << tl)) ++tl;
    return tl;
}

template <typename T, int FMT, int SM, int UPT, int BT>
void launch_quant_upt(const QuantArgs& a, int tl, cudaStream_t stream) {
    const int64_t per = BT >> tl;
    launch_pdl(quantize_fp4_kernel<T, FMT, SM, UPT, BT>, dim3((unsigned)((a.pad_rows + per - 1) / per)), dim3(BT), 0,
               stream, a, tl);
}

template <typename T, int FMT, int SM>
void launch_quant(const QuantArgs& a, cudaStream_t stream) {
    const int tl = threads_per_row_log2(a.units);
    const int64_t upt = (a.units + (1ll << tl) - 1) >> tl;
    if (tl <= 8) {
        if (upt == 1) launch_quant_upt<T, FMT, SM, 1, 256>(a, tl, stream);
        else if (upt == 2) launch_quant_upt<T, FMT, SM, 2, 256>(a, tl, stream);
        else if (upt == 3) launch_quant_upt<T, FMT, SM, 3, 256>(a, tl, stream);
        else launch_quant_upt<T, FMT, SM, 4, 256>(a, tl, stream);
        return;
    }
    if (upt <= 3) return launch_quant_upt<T, FMT, SM, 3, 512>(a, tl, stream);
    if (upt == 4) return launch_quant_upt<T, FMT, SM, 4, 512>(a, tl, stream);
    if constexpr (Unit<T, SM>::RAW)  // (others do not fit a thread's registers)
        if (upt <= 6) return launch_quant_upt<T, FMT, SM, 6, 512>(a, tl, stream);
    launch_quant_upt<T, FMT, SM, 0, 512>(a, tl, stream);
}

template <typename T, int FMT>
void launch_quant_s(const QuantArgs& a, int smooth, cudaStream_t stream) {
    if (smooth == kMul) launch_quant<T, FMT, kMul>(a, stream);
    else if (smooth == kDiv) launch_quant<T, FMT, kDiv>(a, stream);
    else launch_quant<T, FMT, kNone>(a, stream);
}

sq_status_t quantize(const char* name, const void* X, sq_dtype_t dt, int64_t M, int64_t K, int64_t ld, const float* s,
                     int smooth, sq_fp4_t fmt, const float* static_qs, uint8_t* codes, uint8_t* scales, float* qs,
                     cudaStream_t stream) {
    SQ_REQUIRE(dt == SQ_F16 || dt == SQ_BF16 || dt == SQ_F32, SQ_ERR_INVALID_ARG, "%s: dtype must be F16, BF16 or F32",
               name);
    SQ_REQUIRE(fmt == SQ_NVFP4 || fmt == SQ_MXFP4, SQ_ERR_INVALID_ARG, "%s: bad format", name);
    SQ_REQUIRE(M >= 0 && K > 0 && ld >= K, SQ_ERR_UNSUPPORTED_SHAPE, "%s: need K > 0, row stride >= K", name);
    SQ_REQUIRE(K % 32 == 0, SQ_ERR_UNSUPPORTED_SHAPE, "%s: K must be a multiple of 32", name);
    SQ_REQUIRE(M < (1ll << 31) - 128 && K < (1ll << 27), SQ_ERR_UNSUPPORTED_SHAPE, "%s: need rows < 2^31, K < 2^27", name);
    if (M == 0) return SQ_OK;
    SQ_REQUIRE(X && codes && scales, SQ_ERR_INVALID_ARG, "%s: null input, codes or block scales", name);
    SQ_REQUIRE(fmt == SQ_MXFP4 || qs, SQ_ERR_INVALID_ARG, "%s: NVFP4 needs the row scales' output", name);
    SQ_REQUIRE(fmt == SQ_NVFP4 || (!qs && !static_qs), SQ_ERR_INVALID_ARG, "%s: MXFP4 has no row scales", name);
    const int eb = dtype_bytes(dt);
    SQ_REQUIRE(aligned16(X) && (ld * eb) % 16 == 0 && aligned16(codes) && aligned16(scales) && (!s || aligned16(s)),
               SQ_ERR_ALIGNMENT, "%s: pointers and row strides must be 16-byte aligned", name);
    QuantArgs a;
    a.X = X;
    a.s = s;
    a.static_qs = static_qs;
    a.codes = codes;
    a.scales = scales;
    a.qs = qs;
    a.rows = M;
    a.K = K;
    a.ld = ld;
    a.tiles_k = fp4_tiles_k(fmt, K);
    a.pad_rows = fp4_tiles_m(M) * kFp4TileRows;
    a.units = (int)(K >> 4);
    a.wide = (reinterpret_cast<uintptr_t>(X) & 31u) == 0 && (ld * eb) % 32 == 0;
    if (!s) smooth = kNone;
    if (fmt == SQ_NVFP4) {
        if (dt == SQ_F16) launch_quant_s<__half, SQ_NVFP4>(a, smooth, stream);
        else if (dt == SQ_BF16) launch_quant_s<__nv_bfloat16, SQ_NVFP4>(a, smooth, stream);
        else launch_quant_s<float, SQ_NVFP4>(a, smooth, stream);
    } else {
        if (dt == SQ_F16) launch_quant_s<__half, SQ_MXFP4>(a, smooth, stream);
        else if (dt == SQ_BF16) launch_quant_s<__nv_bfloat16, SQ_MXFP4>(a, smooth, stream);
        else launch_quant_s<float, SQ_MXFP4>(a, smooth, stream);
    }
    return check_launch(name);
}

template <typename T>
void launch_dequant(sq_fp4_t fmt, const uint8_t* codes, const uint8_t* scales, const float* qs, int per_row, int64_t M,
                    int64_t K, void* Y, int64_t ldy, cudaStream_t stream) {
    const int64_t units = K >> 4;
    int tl = 0;  // threads per row (log2)
    while (tl < 8 && (1 << tl) < units) ++tl;
    const int64_t per = 256 >> tl;
    const dim3 grid((unsigned)((M + per - 1) / per), (unsigned)((units + (1 << tl) - 1) >> tl));
    const int64_t tk = fp4_tiles_k(fmt, K);
    const bool wide = (reinterpret_cast<uintptr_t>(Y) & 31u) == 0 && (ldy * sizeof(T)) % 32 == 0;
    if (fmt == SQ_NVFP4)
        launch_pdl(dequantize_fp4_kernel<T, SQ_NVFP4>, grid, dim3(256), 0, stream, codes, scales, qs, per_row, M, K, tk,
                   tl, static_cast<T*>(Y), ldy, wide);
    else
        launch_pdl(dequantize_fp4_kernel<T, SQ_MXFP4>, grid, dim3(256), 0, stream, codes, scales, qs, per_row, M, K, tk,
                   tl, static_cast<T*>(Y), ldy, wide);
}

}  // namespace
}  // namespace sq

extern "C" {

size_t sq_fp4_scale_bytes(sq_fp4_t fmt, int64_t rows, int64_t K) {
    if ((fmt != SQ_NVFP4 && fmt != SQ_MXFP4) || rows <= 0 || K <= 0) return 0;
    return (size_t)(sq::fp4_tiles_m(rows) * sq::fp4_tiles_k(fmt, K)) * sq::kFp4TileBytes;
}

sq_status_t sq_quantize_weight_fp4(const void* W, sq_dtype_t dt, int64_t N, int64_t K, const float* s, sq_fp4_t fmt,
                                   uint8_t* Wq, uint8_t* Ws, float* qs_w, sq_stream_t stream) {
    return sq::quantize("sq_quantize_weight_fp4", W, dt, N, K, K, s, sq::kMul, fmt, nullptr, Wq, Ws, qs_w,
                        sq::as_cuda(stream));
}

sq_status_t sq_quantize_act_fp4(const void* X, sq_dtype_t dt, int64_t M, int64_t K, int64_t ldx, const float* s,
                                sq_fp4_t fmt, int per_token, const float* static_qs, uint8_t* Xq, uint8_t* Xs,
                                float* qs_x, sq_stream_t stream) {
    const char* name = "sq_quantize_act_fp4";
    SQ_REQUIRE(per_token || static_qs || fmt != SQ_NVFP4, SQ_ERR_INVALID_ARG,
               "%s: per_token = 0 needs static_qs", name);
    return sq::quantize(name, X, dt, M, K, ldx, s, sq::kDiv, fmt, per_token ? nullptr : static_qs, Xq, Xs, qs_x,
                        sq::as_cuda(stream));
}

sq_status_t sq_dequantize_fp4(const uint8_t* Xq, const uint8_t* Xs, sq_fp4_t fmt, int64_t M, int64_t K,
                              const float* qs, int per_row, sq_dtype_t out_dt, void* Y, int64_t ldy,
                              sq_stream_t stream) {
    const char* name = "sq_dequantize_fp4";
    SQ_REQUIRE(out_dt == SQ_F16 || out_dt == SQ_BF16 || out_dt == SQ_F32, SQ_ERR_INVALID_ARG,
               "%s: out dtype must be F16, BF16 or F32", name);
    SQ_REQUIRE(fmt == SQ_NVFP4 || fmt == SQ_MXFP4, SQ_ERR_INVALID_ARG, "%s: bad format", name);
    SQ_REQUIRE(M >= 0 && K > 0 && ldy >= K, SQ_ERR_UNSUPPORTED_SHAPE, "%s: need K > 0, ldy >= K", name);
    SQ_REQUIRE(K % 32 == 0, SQ_ERR_UNSUPPORTED_SHAPE, "%s: K must be a multiple of 32", name);
    SQ_REQUIRE(M < (1ll << 31) - 256 && K < (1ll << 27), SQ_ERR_UNSUPPORTED_SHAPE, "%s: need M < 2^31, K < 2^27", name);
    if (M == 0) return SQ_OK;
    SQ_REQUIRE(Xq && Xs && Y, SQ_ERR_INVALID_ARG, "%s: null codes, block scales or Y", name);
    SQ_REQUIRE(sq::aligned16(Xq) && sq::aligned16(Xs) && sq::aligned16(Y) &&
                   (ldy * sq::dtype_bytes(out_dt)) % 16 == 0,
               SQ_ERR_ALIGNMENT, "%s: pointers and row strides must be 16-byte aligned", name);
    cudaStream_t st = sq::as_cuda(stream);
    if (out_dt == SQ_F16) sq::launch_dequant<__half>(fmt, Xq, Xs, qs, per_row, M, K, Y, ldy, st);
    else if (out_dt == SQ_BF16) sq::launch_dequant<__nv_bfloat16>(fmt, Xq, Xs, qs, per_row, M, K, Y, ldy, st);
    else sq::launch_dequant<float>(fmt, Xq, Xs, qs, per_row, M, K, Y, ldy, st);
    return sq::check_launch(name);
}

}  // extern "C"
