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
// of 16 elements in registers between the row maximum and the codes. Rows too
// wide for that (over 32768 elements) are read twice, the second time from L2.
// What bounds it: the bytes (2 in and 0.56 out per 16-bit element).
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "sq_common.cuh"
#include "sq_fp4.cuh"

namespace sq {
namespace {

enum Smooth { kNone = 0, kMul = 1, kDiv = 2 };
constexpr uint32_t kInfBits = 0x7f800000u;

// 16 consecutive elements as fp32, smoothed.
template <typename T, int SM>
__device__ __forceinline__ void load16(const T* row, const float* s, int64_t k, float* v) {
    constexpr int VN = Vec<T>::N;
#pragma unroll
    for (int i = 0; i < 16 / VN; ++i) unpack<T>(ldg_nc_v4(row + k + i * VN), v + i * VN);
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
}

// Largest |v| as bits: above kInfBits - 1 if a value is not finite (bit
// patterns of non-negative floats order as the floats do, infinities and NaN
// above every finite value).
__device__ __forceinline__ uint32_t absmax_bits(const float* v) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 16; ++e) m = max(m, __float_as_uint(v[e]) & 0x7fffffffu);
    return m;
}
__device__ __noinline__ uint32_t finite_absmax_bits(const float* v) {
    uint32_t m = 0;
    for (int e = 0; e < 16; ++e) {
        const uint32_t b = __float_as_uint(v[e]) & 0x7fffffffu;
        if (b < kInfBits) m = max(m, b);
    }
    return m;
}

// 2^(10 - floor(log2 m)); m below 2^-100 counts as 2^-100, so the scale and its
// reciprocal stay normal.
__device__ __forceinline__ float row_scale(uint32_t amax_bits) {
    const int field = max((int)(amax_bits >> 23), 27);
    return __uint_as_float((uint32_t)(264 - field) << 23);
}

// Eight codes of fl(u / b), inv = fl(1 / b). The quotient is rounded correctly
// by one residual step (Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990: with inv the correctly rounded
// reciprocal, q = fl(u inv), r = u - q b exactly, fl(q + r inv) is the rounded
// quotient), because a quotient that lies on the border between two codes is
// common (u and b have few bits) and must go to the even code.
__device__ __forceinline__ uint32_t codes8(const float* u, float b, float inv) {
    uint32_t w = 0;
    const uint64_t nb2 = pk2(-b, -b), inv2 = pk2(inv, inv);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t u2 = pk2(u[2 * e], u[2 * e + 1]);
        const uint64_t q2 = mul2(u2, inv2);
        const uint64_t r2 = fma2(q2, nb2, u2);
        float2 t;
        upk2(fma2(r2, inv2, q2), t.x, t.y);
        w |= (uint32_t)__nv_cvt_float2_to_fp4x2(t, __NV_E2M1, cudaRoundNearest) << (8 * e);
    }
    return w;
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
};

// Codes and scale of one unit. bits: |v| maximum of the unit. Every lane of the
// warp calls this (valid = 0 past the row's end).
template <int FMT>
__device__ __forceinline__ void emit_unit(const QuantArgs& a, int64_t row, int unit, bool valid, float* v, uint32_t bits,
                                          float qs) {
    uint32_t byte;
    uint2 w;
    if constexpr (FMT == SQ_NVFP4) {
        const uint64_t qs2 = pk2(qs, qs);
        const float top = __fmul_rn(__uint_as_float(bits), qs);
#pragma unroll
        for (int e = 0; e < 16; e += 2) upk2(mul2(pk2(v[e], v[e + 1]), qs2), v[e], v[e + 1]);
        byte = __nv_cvt_float_to_fp8(__fdiv_rn(top, 6.0f), __NV_SATFINITE, __NV_E4M3);
        const bool finite = bits < kInfBits;
        if (!finite) byte = 0x7Fu;
        const float b = __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3)));
        const float inv = byte == 0 ? 0.0f : __frcp_rn(b);
        w = make_uint2(codes8(v, b, inv), codes8(v + 8, b, inv));
        if (!finite) w = make_uint2(0, 0);
    } else {
        // a block of 32 is two neighbouring lanes' units (K is a multiple of 32)
        bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, 1));
        const bool finite = bits < kInfBits;
        byte = (uint32_t)max((int)(bits >> 23) - 2, 0);
        const float up = __uint_as_float((254u - byte) << 23);  // 1 / b, exact, as every product with it
        const uint64_t up2 = pk2(up, up);
        uint32_t h[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            float2 t;
            upk2(mul2(pk2(v[2 * e], v[2 * e + 1]), up2), t.x, t.y);
            h[e >> 2] |= (uint32_t)__nv_cvt_float2_to_fp4x2(t, __NV_E2M1, cudaRoundNearest) << (8 * (e & 3));
        }
        w = finite ? make_uint2(h[0], h[1]) : make_uint2(0, 0);
        if (!finite) byte = 0xFFu;
    }
    if (!valid) byte = 0;
    else *reinterpret_cast<uint2*>(a.codes + row * (a.K >> 1) + (int64_t)unit * 8) = w;
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
        *reinterpret_cast<uint32_t*>(a.scales + fp4_scale_offset(row, unit / G, a.tiles_k)) = word;
}

// Row maximum over the TPR threads (a power of two, 32 to 512) of this row.
__device__ __forceinline__ uint32_t row_max(uint32_t m, int tpr, uint32_t* sh) {
    m = __reduce_max_sync(0xffffffffu, m);
    if (tpr > 32) {
        const int warp = threadIdx.x >> 5, per = tpr >> 5, first = warp / per * per;
        if ((threadIdx.x & 31) == 0) sh[warp] = m;
        __syncthreads();
        for (int w = 0; w < per; ++w) m = max(m, sh[first + w]);
    }
    return m;
}

// UPT units per thread held in registers; UPT = 0: any width, read twice.
template <typename T, int FMT, int SM, int UPT>
__global__ void __launch_bounds__(512) quantize_fp4_kernel(const QuantArgs a, int tpr) {
    __shared__ uint32_t sh[16];
    pdl_wait();
    pdl_trigger();
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const int t = threadIdx.x & (tpr - 1);
    const bool live = row < a.rows;  // the same for a whole warp
    if (row >= a.rows && row < a.pad_rows)
        // rows that fill up the last tile: zero scales
        for (int64_t k = t; k < a.tiles_k; k += tpr)
            *reinterpret_cast<uint32_t*>(a.scales + fp4_scale_offset(row, k, a.tiles_k)) = 0u;
    const T* x = static_cast<const T*>(a.X) + (live ? row : 0) * a.ld;
    float qs = 1.0f;
    if constexpr (UPT > 0) {
        float v[UPT][16];
        uint32_t bits[UPT];
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            const int u = t + i * tpr;
            bits[i] = 0;
            if (live && u < a.units) {
                load16<T, SM>(x, a.s, (int64_t)u * 16, v[i]);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[i][e] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < UPT; ++i) {
            bits[i] = absmax_bits(v[i]);
            m = max(m, bits[i] < kInfBits ? bits[i] : finite_absmax_bits(v[i]));
        }
        if constexpr (FMT == SQ_NVFP4) {
            if (a.static_qs) qs = *a.static_qs;
            else qs = row_scale(row_max(m, tpr, sh));
        }
        if (!live) return;
#pragma unroll
        for (int i = 0; i < UPT; ++i)
            if (i * tpr < a.units) emit_unit<FMT>(a, row, t + i * tpr, t + i * tpr < a.units, v[i], bits[i], qs);
    } else {
        float v[16];
        if constexpr (FMT == SQ_NVFP4) {
            uint32_t m = 0;
            if (!a.static_qs && live)
                for (int u = t; u < a.units; u += tpr) {
                    load16<T, SM>(x, a.s, (int64_t)u * 16, v);
                    const uint32_t b = absmax_bits(v);
                    m = max(m, b < kInfBits ? b : finite_absmax_bits(v));
                }
            if (a.static_qs) qs = *a.static_qs;
            else qs = row_scale(row_max(m, tpr, sh));
        }
        if (!live) return;
        for (int u0 = 0; u0 < a.units; u0 += tpr) {
            const int u = u0 + t;
            if (u < a.units) {
                load16<T, SM>(x, a.s, (int64_t)u * 16, v);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e) v[e] = 0.0f;
            }
            emit_unit<FMT>(a, row, u, u < a.units, v, absmax_bits(v), qs);
        }
    }
    if (FMT == SQ_NVFP4 && a.qs && t == 0) a.qs[a.static_qs ? 0 : row] = qs;
}

// value = fl(fl(code b) fl(1 / qs)), the first product exact; one rounding to T.
template <typename T, int FMT>
__global__ void __launch_bounds__(256)
dequantize_fp4_kernel(const uint8_t* codes, const uint8_t* scales, const float* qs, int per_row, int64_t rows, int64_t K,
                      int64_t tiles_k, int tpr, T* Y, int64_t ldy) {
    pdl_wait();
    pdl_trigger();
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    const int u = blockIdx.y * tpr + (threadIdx.x & (tpr - 1));
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
    float y[16];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const uint32_t by = ((e < 4 ? w.x : w.y) >> (8 * (e & 3))) & 0xffu;
        const float2 f = __half22float2(__half2(__nv_cvt_fp4x2_to_halfraw2((__nv_fp4x2_storage_t)by, __NV_E2M1)));
        y[2 * e] = __fmul_rn(__fmul_rn(f.x, b), rq);
        y[2 * e + 1] = __fmul_rn(__fmul_rn(f.y, b), rq);
    }
    T* out = Y + row * ldy + (int64_t)u * 16;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            __stcs(reinterpret_cast<float4*>(out) + i, make_float4(y[4 * i], y[4 * i + 1], y[4 * i + 2], y[4 * i + 3]));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
                p[e] = (uint32_t)to16<T>(y[8 * i + 2 * e]) | ((uint32_t)to16<T>(y[8 * i + 2 * e + 1]) << 16);
            __stcs(reinterpret_cast<uint4*>(out) + i, make_uint4(p[0], p[1], p[2], p[3]));
        }
    }
}

// Threads per row: the fewest (a power of two) that hold the row in at most
// four units of 16 each, up to 512.
int threads_per_row(int64_t units) {
    int tpr = 32;
    while (tpr < 512 && units > 4ll * tpr) tpr *= 2;
    return tpr;
}

template <typename T, int FMT, int SM>
void launch_quant(const QuantArgs& a, cudaStream_t stream) {
    const int tpr = threads_per_row(a.units);
    const int threads = tpr > 256 ? tpr : 256;
    const int64_t grid = (a.pad_rows + threads / tpr - 1) / (threads / tpr);
    const int64_t upt = (a.units + tpr - 1) / tpr;
    const dim3 g((unsigned)grid), b(threads);
    if (upt == 1) launch_pdl(quantize_fp4_kernel<T, FMT, SM, 1>, g, b, 0, stream, a, tpr);
    else if (upt == 2) launch_pdl(quantize_fp4_kernel<T, FMT, SM, 2>, g, b, 0, stream, a, tpr);
    else if (upt == 3) launch_pdl(quantize_fp4_kernel<T, FMT, SM, 3>, g, b, 0, stream, a, tpr);
    else if (upt == 4) launch_pdl(quantize_fp4_kernel<T, FMT, SM, 4>, g, b, 0, stream, a, tpr);
    else launch_pdl(quantize_fp4_kernel<T, FMT, SM, 0>, g, b, 0, stream, a, tpr);
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
    SQ_REQUIRE(M < (1ll << 31) - 128 && K < (1ll << 31), SQ_ERR_UNSUPPORTED_SHAPE, "%s: rows and K must be < 2^31", name);
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
    int tpr = 1;
    while (tpr < 256 && tpr < units) tpr *= 2;
    const dim3 grid((unsigned)((M + 256 / tpr - 1) / (256 / tpr)), (unsigned)((units + tpr - 1) / tpr));
    const int64_t tk = fp4_tiles_k(fmt, K);
    if (fmt == SQ_NVFP4)
        launch_pdl(dequantize_fp4_kernel<T, SQ_NVFP4>, grid, dim3(256), 0, stream, codes, scales, qs, per_row, M, K, tk,
                   tpr, static_cast<T*>(Y), ldy);
    else
        launch_pdl(dequantize_fp4_kernel<T, SQ_MXFP4>, grid, dim3(256), 0, stream, codes, scales, qs, per_row, M, K, tk,
                   tpr, static_cast<T*>(Y), ldy);
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
