// The paged int8 K/V cache: K and V codes [num_blocks, Hkv, block, D], one
// scale per block and head in kqs, vqs [num_blocks, Hkv] (value = code / qs),
// and for each sequence a row of block numbers, its length, and its range of
// the flattened new tokens (cu_q).
#pragma once

#include <stdint.h>

#include "sq_tc.cuh"

namespace sq {

// The sequence that holds flattened token t: the last b < B with cu[b] <= t.
// All 32 lanes search together (32 probes a round).
__device__ __forceinline__ int kv8_sequence_of(const int32_t* cu, int B, int64_t t, int lane) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) >> 5;
        const int i = lo + lane * step;
        const unsigned at = __ballot_sync(0xffffffffu, i < hi && (lane == 0 || (int64_t)__ldg(cu + i) <= t));
        lo += (31 - __clz(at)) * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Sizes and pointers that appending to the cache and reading it share.
sq_status_t check_kv8(const char* name, int64_t T, int64_t B, int64_t Hkv, int64_t D, int64_t block, int64_t num_blocks,
                      int64_t max_blocks, int64_t ldb);

// ---------------------------------------------------------------- attention
constexpr float kLog2e = 1.4426950408889634f;
// The running maximum follows a score only when that is this far (in log2) above it,
// and is kept this far below the score that it then follows: the weights stay below
// 2^(kSlack + kLift), inside fp16, and those down to 2^-21 of the largest are normal
// fp16 numbers, smaller ones off by 2^-32 of the largest at most.
constexpr float kSlack = 8.0f, kLift = 7.0f;

struct AttnArgs {
    const void* Q;
    void* Y;
    int64_t ldq, ldy, T, ldb, num_blocks;
    const int32_t* cu;
    const int32_t* lens;
    const int32_t* table;
    const float* kqs;
    const float* vqs;
    int B, Hkv, G, block, block_log2, box, max_blocks, causal;
    int64_t row_limit;  // sequences of more rows (new tokens x G) than this are the prompt kernel's
    float scale;
    int* status;
    int cnt_bytes;  // of the counters
    int* cnt;     // what was counted in of a row tile that several blocks share (zero between launches)
    float* part;  // their parts: O, m and l of the rows
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Bytes of u (code + 128) as fp16 integers: 0x6400 + u is 1024 + u in fp16, so
// subtracting 1152 leaves the code, exactly.
__device__ __forceinline__ uint32_t half2_of(uint32_t u, uint32_t sel) {
    const uint32_t h = __byte_perm(u, 0x64646464u, sel);
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x64806480u));
    return r;
}
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// One sequence's share of the work.
struct Seq {
    int64_t lo;  // first new token
    int n, len, rt, tiles;
    __device__ int64_t work(int Hkv) const { return (int64_t)Hkv * rt * tiles; }
};
template <int ROWS, int KEYS>
__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b) {
    Seq s;
    const int64_t lo = min(max((int64_t)__ldg(a.cu + b), (int64_t)0), a.T);
    const int64_t hi = min((int64_t)__ldg(a.cu + b + 1), a.T);
    s.lo = lo;
    s.n = (int)max(hi - lo, (int64_t)0);
    s.len = min(max(__ldg(a.lens + b), 0), a.max_blocks * a.block);
    s.rt = (int)(((int64_t)s.n * a.G + ROWS - 1) / ROWS);
    s.tiles = max((s.len + KEYS - 1) / KEYS, 1);  // a sequence without keys still has rows to write
    return s;
}

// Keys that row `row` of a sequence sees (rows past the last see what it sees).
__device__ __forceinline__ int seen_by(const AttnArgs& a, const Seq& s, int row) {
    const int i = min(row / a.G, s.n - 1);
    return a.causal ? max(min(s.len - s.n + i + 1, s.len), 0) : s.len;
}

// The cache as [num_blocks, Hkv * block, D] bytes, box D x box x 1, rows
// swizzled over their own width or as they are.
inline bool make_map_kv(CUtensorMap* m, const int8_t* base, int64_t num_blocks, int64_t rows, int64_t D, int box,
                        bool swizzle) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)num_blocks};
    cuuint64_t strides[2] = {(cuuint64_t)D, (cuuint64_t)(rows * D)};
    cuuint32_t bx[3] = {(cuuint32_t)D, (cuuint32_t)box, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<int8_t*>(base), dims, strides, bx, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE,
              !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : D == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Prompts: sequences of more rows than row_limit (kv8_prefill.cu), and the
// bytes of its parts.
size_t kv8_prefill_part_bytes(int64_t D);
sq_status_t launch_kv8_prefill(const char* name, sq_dtype_t dt, int64_t D, const int8_t* Kc, const int8_t* Vc,
                               const AttnArgs& a, cudaStream_t stream);

}  // namespace sq
