// The 8-bit paged cache and the rotary positions: arguments and device helpers shared by
// rope.cu, cache_q8.cu, decode_q8.cu and api_q8.cu.
//
// Cache format: e4m3 codes [NB][Hkv][B][128] for K and for V, and one int8 exponent per
// (block, kv head) for each; the value of a code c is c * 2^e, -60 <= e <= 60.  The scale is a
// power of two: e4m3 keeps four significant bits at any scale, so against amax / 448 it only gives
// up part of one binade at the small end; moving a block to a larger exponent is then exact for
// every code that stays normal, and every kernel applies the scale by adding an exponent.
#pragma once

#include <utility>

#include "pa_internal.cuh"

namespace pa {

constexpr int kExpMin = -60, kExpMax = 60;   // sums of two exponents and the softmax's own stay in fp32
constexpr int kRopeMaxHead = 1024;            // head size of a rotation
constexpr int kQ8MaxRows = 32;               // query rows per (sequence, kv head) of one attention call

struct RopeArgs {
    const void* q;             // [T][Hq][D], rows of tokens q_stride elements apart
    const void* k;             // [T][Hkv][D] (num_kv_heads == 0: none)
    void* out_q;
    void* out_k;
    long long q_stride, k_stride, out_q_stride, out_k_stride;
    const void* positions;     // [T], int32 or int64
    const double* inv_freq;    // [R / 2], radians per position
    float magnitude;
    int wide_positions;        // positions are int64
    int num_tokens;
    int num_q_heads;
    int num_kv_heads;
    int head_dim;
    int rotary_dim;
    int interleaved;
    int in_place_q, in_place_k;   // the unrotated part of a head is already where it belongs
};

struct AppendQ8Args {
    const void* k;             // [T][Hkv][128], tokens k_stride elements apart
    const void* v;
    long long k_stride, v_stride;
    uint8_t* k_cache;          // [NB][Hkv][B][128] e4m3
    uint8_t* v_cache;
    int8_t* k_exp;             // [NB][Hkv]
    int8_t* v_exp;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* q_start;    // null: row s is sequence s's newest token
    unsigned int* status;
    int num_seqs;
    int rows;                  // T
    int max_q;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    int max_blocks_per_seq;
};

struct ReadQ8Args {
    const uint4* k_cache;      // codes, 16 per vector
    const uint4* v_cache;
    const int8_t* k_exp;
    const int8_t* v_exp;
    uint4* dst_k;              // 16-bit pool, 8 elements per vector
    uint4* dst_v;
    const int32_t* src_ids;
    const int32_t* dst_ids;
    unsigned int* status;
    int num_pairs;
    int src_blocks;
    int dst_blocks;
    int num_kv_heads;
    int vecs_per_head;         // B * 128 / 16
};

struct DecodeQ8Args {
    void* out;                 // [T][Hq][128]
    const void* q;
    const uint8_t* k_cache;
    const uint8_t* v_cache;
    const int8_t* k_exp;
    const int8_t* v_exp;
    const int32_t* block_tables;
    const int32_t* context_lens;
    const int32_t* q_start;    // null: one query row per sequence
    unsigned int* status;
    float scale_log2;          // scale * log2(e)
    int num_seqs;
    int q_rows;
    int max_q;
    int num_q_heads;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    int max_blocks_per_seq;
};

// ---- e4m3 conversions (two at a time; the low half of the register comes from the low byte) ----
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t c) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

// Round to nearest even, beyond +-448 (and +-inf) to +-448, NaN to NaN.
__device__ __forceinline__ uint16_t f32_to_e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float2 e4m3x2_to_float2(uint16_t c) {
    const uint32_t h = e4m3x2_to_f16x2(c);
    return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// |x| where x is finite, else 0
__device__ __forceinline__ float finite_abs(float x) {
    const float f = fabsf(x);
    return f <= 3.402823466e38f ? f : 0.f;
}

__device__ __forceinline__ int clamp_exp(int e) { return max(kExpMin, min(kExpMax, e)); }

// 2^e, -126 <= e <= 127
__device__ __forceinline__ float exp2_int(int e) { return __int_as_float((e + 127) << 23); }

// The least e with amax <= 448 * 2^e (448 = 1.75 * 2^8), kept in the exponents' range.
__device__ __forceinline__ int exponent_for(float amax) {
    const int bits = __float_as_int(amax);   // amax >= 0, finite
    const int e = (bits >> 23) - 127 - 8 + ((bits & 0x7fffff) > 0x600000 ? 1 : 0);
    return clamp_exp(e);
}

// The new rows of sequence s with L cached tokens, as pa_multi_query clamps them: row0 .. row0+n-1
// of the new rows hold positions L-n .. L-1.  `bad`: a count or a span had to be clamped.
struct NewRows {
    int row0;
    int n;
    bool bad;
};

__device__ __forceinline__ NewRows new_rows(const int32_t* q_start, int rows, int max_q, int s, int L) {
    const int b = q_start[s], e = q_start[s + 1];
    const int r0 = max(0, min(b, rows));
    const long long want = (long long)e - b;
    const int n = (int)max(0LL, min(min(want, (long long)(rows - r0)), (long long)min(L, max_q)));
    return NewRows{r0, n, b != r0 || want != n};
}

// context_lens[s] kept inside the table.
__device__ __forceinline__ int clamped_len(const int32_t* lens, int s, int max_blocks, int block_size, bool* bad) {
    const int L = lens[s], cap = max_blocks * block_size;
    const int c = max(0, min(L, cap));
    *bad = c != L;
    return c;
}

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t stream);
cudaError_t launch_append_q8(const AppendQ8Args& a, int dtype, cudaStream_t stream);
cudaError_t launch_read_q8(const ReadQ8Args& a, int dtype, cudaStream_t stream);
size_t q8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int max_q, int block_size,
                          int max_blocks_per_seq);
bool q8_line_fits(int num_seqs, int num_kv_heads, int block_size, int max_blocks_per_seq);
cudaError_t launch_decode_q8(const DecodeQ8Args& a, int dtype, void* workspace, cudaStream_t stream);

// Launch with programmatic serialisation: the kernel may start its prologue while the preceding
// one drains, and waits (grid_dependency_wait) before it touches memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    if (e == cudaSuccess) note_launches(1);
    return e;
}

}  // namespace pa
