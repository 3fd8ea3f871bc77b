// The 8-bit cache's write and read-back.
//
// append_q8: each sequence's new rows go to the slots of their positions ("显存虚拟化革命：PagedAttention
// 内存池管理与显存碎片终结", §三 sequence diagram; the address rule of "端侧 SLM 显存保活术：在 4GB
// 内存板卡上实现轻量 PagedAttention 与 KV 缓存分块"), quantised with one exponent per (block, kv head):
//   e_need = least e with amax <= 448 * 2^e, amax over the finite |x| of the call's rows in the block
//   e      = e_need                  when the call writes the block's offset 0 (the block starts afresh)
//          = max(e_old, e_need)      otherwise; rows before the new ones are rounded again if e grew
//   code   = e4m3(x * 2^-e)          to nearest even; beyond 448 (inf, or amax > 448 * 2^60) to +-448
// The products by a power of two are exact, so a code is off by its own rounding alone.
//
// Design: one warp (2 or 4 for large blocks of long chunks) per (touched block, kv head, K or V): it alone
// decides the block's exponent, so there are no atomics and the result has one value.  It holds 16 or 32 rows in
// registers and reads those before them again, from L2, once the exponent is known.  The host does not know how
// many blocks a ragged batch touches; unit v of a sequence is found by a search in the monotone bounds
// query_start[s] / B + 2 s, which leave every sequence at least the blocks it touches.  One row per sequence, the
// decode step's form, has a kernel of its own.
//
// read_q8: code * 2^e rounded to the pool's 16-bit type (bf16 exactly), beyond its range to its
// largest value; one thread per 16 codes of K and of V.
//
// Both are bound by HBM: 512 rows x 16 sequences x 32 heads appended in 33 us (32-token blocks; 0.89 of a copy's
// rate), 2048 blocks of 32 rows x 32 heads read back in 241 us (0.98).  One row a sequence (64 x 2 heads) takes
// 2.2 us: the launch, and length, table and exponent one after another.
#include <type_traits>

#include "q8.cuh"

namespace pa {

namespace {

constexpr int kAppendWarps = 8;

// Largest s in [0, S) with q_start[s] / B + 2 s <= v, by the lanes of a warp together.
__device__ __forceinline__ int find_seq(const AppendQ8Args& a, int v, int lane) {
    int lo = 0, hi = a.num_seqs;   // the answer lies in [lo, hi)
    while (hi - lo > 1) {
        const int step = (hi - lo + 31) / 32;
        const int s = lo + lane * step;
        const bool le = s < hi && max(0, min(a.q_start[s], a.rows)) / a.block_size + 2LL * s <= v;
        const unsigned m = __ballot_sync(0xffffffffu, le);
        const int k = m ? 31 - __clz(m) : 0;
        lo = lo + k * step;
        hi = min(hi, lo + step);
    }
    return lo;
}

// Finite bits of a 16-bit type's magnitude are below this, in both halves of a register.
template <typename T>
constexpr uint32_t kInf2 = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;

// Eight elements times a power of two to e4m3.
template <typename T>
__device__ __forceinline__ uint2 quantise8(const uint4& x, float mul) {
    float f[8];
    unpack8<T>(x, f);
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        w[k] = (uint32_t)f32_to_e4m3x2(f[4 * k] * mul, f[4 * k + 1] * mul) |
               ((uint32_t)f32_to_e4m3x2(f[4 * k + 2] * mul, f[4 * k + 3] * mul) << 16);
    return make_uint2(w[0], w[1]);
}

// Eight codes under a grown exponent.
__device__ __forceinline__ uint2 rescale8(uint2 codes, float down) {
    const uint32_t w[2] = {codes.x, codes.y};
    uint32_t n[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float2 p = e4m3x2_to_float2((uint16_t)(w[k] & 0xffffu)), q = e4m3x2_to_float2((uint16_t)(w[k] >> 16));
        n[k] = (uint32_t)f32_to_e4m3x2(p.x * down, p.y * down) | ((uint32_t)f32_to_e4m3x2(q.x * down, q.y * down) << 16);
    }
    return make_uint2(n[0], n[1]);
}

// The rows r, r + step, .. below `end` (8 codes of each, rows kHeadDim apart from `dst` on) under a grown exponent,
// eight loads in flight (128 ragged sequences of 128-token blocks whose exponents all grow: 14 us beyond the fill that
// lowers them, 25 one row after another; 64 decode steps of 16-token blocks 4.2 and 6.8).
__device__ __forceinline__ void rescale_rows(uint8_t* dst, int r, int end, int step, float down) {
    constexpr int kBatch = 8;
    for (; r < end; r += kBatch * step) {
        uint2 c[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (r + i * step < end) c[i] = *reinterpret_cast<const uint2*>(dst + (r + i * step) * kHeadDim);
#pragma unroll
        for (int i = 0; i < kBatch; ++i)
            if (r + i * step < end) *reinterpret_cast<uint2*>(dst + (r + i * step) * kHeadDim) = rescale8(c[i], down);
    }
}

// One new row per sequence (query_start == null): a warp takes eight kv heads of a sequence, its lower half
// their K rows and its upper half their V rows, so that the walk from length to table to exponent is made once.
constexpr int kOneHeads = 8;

template <typename T>
__global__ void __launch_bounds__(kAppendWarps * 32) append_one_q8_kernel(const AppendQ8Args a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32, c = lane % 16, is_v = lane / 16;
    const int B = a.block_size, Hkv = a.num_kv_heads, groups = (Hkv + kOneHeads - 1) / kOneHeads;
    const unsigned u = blockIdx.x * kAppendWarps + threadIdx.x / 32;
    const int s = (int)(u / groups), h0 = (int)(u % groups) * kOneHeads;
    if (s >= a.num_seqs) return;
    const T* src = static_cast<const T*>(is_v ? a.v : a.k) + s * (is_v ? a.v_stride : a.k_stride) + h0 * kHeadDim + c * 8;
    uint4 x[kOneHeads];
#pragma unroll
    for (int i = 0; i < kOneHeads; ++i) {
        x[i] = make_uint4(0, 0, 0, 0);
        if (h0 + i < Hkv) x[i] = __ldg(reinterpret_cast<const uint4*>(src + i * kHeadDim));
    }
    bool bad_len;
    const int L = clamped_len(a.context_lens, s, a.max_blocks_per_seq, B, &bad_len);
    if (bad_len && h0 == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
    if (L == 0) return;
    const int blk = __ldg(a.block_tables + (size_t)s * a.max_blocks_per_seq + (L - 1) / B), lo = (L - 1) % B;
    if (blk < 0 || blk >= a.num_blocks) {
        if (h0 == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t tile0 = (size_t)blk * Hkv + h0;
    int8_t* exps = (is_v ? a.v_exp : a.k_exp) + tile0;
    int e_old[kOneHeads];
#pragma unroll
    for (int i = 0; i < kOneHeads; ++i) e_old[i] = h0 + i < Hkv ? clamp_exp(exps[i]) : 0;
#pragma unroll
    for (int i = 0; i < kOneHeads; ++i) {
        if (h0 + i >= Hkv) break;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
        uint32_t top = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t m = w[k] & 0x7fff7fffu;
            top = __vmaxu2(top, m & ~__vcmpgeu2(m, kInf2<T>));   // infinities and NaN do not count
        }
        uint32_t amax = max(top & 0xffffu, top >> 16);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const int need = exponent_for(Elem<T>::to_float((uint16_t)amax));
        const int e = lo == 0 ? need : max(e_old[i], need);
        uint8_t* dst = (is_v ? a.v_cache : a.k_cache) + (tile0 + i) * B * kHeadDim + c * 8;
        *reinterpret_cast<uint2*>(dst + lo * kHeadDim) = quantise8<T>(x[i], exp2_int(-e));
        if (e > e_old[i] && lo > 0) rescale_rows(dst, 0, lo, 1, exp2_int(e_old[i] - e));   // earlier rows
        if (c == 0) exps[i] = (int8_t)e;
    }
}

// kWpu: warps of a unit (0: `warps_per_unit`); kCtas: CTAs that share an SM (their registers: a chunk's append is bound
// by the bytes in flight, 512 rows x 16 sequences x 32 heads: 35.9 us with 3 in 16-token blocks, 32.2 with 4; 36.5 with
// 2 in 32-token blocks, 33.3 with 3; 38.8 with 2 in 64-token blocks, 35.4 with 3; a few rows a sequence by the first
// waits: one to eight rows x 100 sequences, 4.1 us with 3 and 4.8 with 4).
template <typename T, int kRows, int kWpu, int kCtas>
__global__ void __launch_bounds__(kAppendWarps * 32, kCtas) append_q8_kernel(const AppendQ8Args a, int blocks, int warps_per_unit) {
    const int wpu = kWpu ? kWpu : warps_per_unit;
    __shared__ uint32_t amax_of[kAppendWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int B = a.block_size, Hkv = a.num_kv_heads;
    const int part = warp % wpu;                               // of the unit's `wpu` warps
    // where query_start decreases, the search below may miss the sequences around (the grid has a thread for each)
    const unsigned tid = blockIdx.x * blockDim.x + threadIdx.x;
    if (tid < (unsigned)a.num_seqs && a.q_start[tid + 1] < a.q_start[tid]) flag_status(a.status, PA_DEV_BAD_CONTEXT);
    const unsigned u = blockIdx.x * (kAppendWarps / wpu) + warp / wpu;   // (virtual block, head, K or V)
    const int is_v = u % 2, h = (int)(u / 2 % Hkv), v = (int)(u / 2 / Hkv);
    if (v >= blocks) return;
    const int s = find_seq(a, v, lane);
    bool bad_len;
    const int L = clamped_len(a.context_lens, s, a.max_blocks_per_seq, B, &bad_len);
    const NewRows nr = new_rows(a.q_start, a.rows, a.max_q, s, L);
    const int j = (int)(v - (nr.row0 / B + 2LL * s));
    const bool speaks = h == 0 && !is_v && part == 0 && lane == 0;
    if ((bad_len || nr.bad) && j == 0 && speaks) flag_status(a.status, PA_DEV_BAD_CONTEXT);
    const int p0 = L - nr.n;                                   // first new position
    const int blk_i = p0 / B + j;                              // logical block
    if (j < 0 || nr.n == 0 || blk_i > (L - 1) / B) return;     // (as all of the unit's warps)
    const int blk = __ldg(a.block_tables + (size_t)s * a.max_blocks_per_seq + blk_i);
    const int lo = max(0, p0 - blk_i * B), hi = min(B, L - blk_i * B);   // new rows of the block: [lo, hi)
    // a batch of rows from b on: this lane has rows b + lane / 16 + 2 i, eight elements (c) of each; the warp's
    // batches begin at `begin` and lie `stride_rows` apart
    const int begin = lo + part * kRows, stride_rows = wpu * kRows;
    const int c = lane % 16;
    const long long stride = is_v ? a.v_stride : a.k_stride;
    const T* src = static_cast<const T*>(is_v ? a.v : a.k) + (nr.row0 + (long long)(blk_i * B - p0)) * stride +
                   h * kHeadDim + c * 8;
    uint4 x[kRows / 2];
    auto load = [&](int b) {
#pragma unroll
        for (int i = 0; i < kRows / 2; ++i) {
            const int r = b + lane / 16 + 2 * i;
            x[i] = make_uint4(0, 0, 0, 0);
            if (r < hi) x[i] = __ldg(reinterpret_cast<const uint4*>(src + r * stride));
        }
    };
    load(begin);
    if (blk < 0 || blk >= a.num_blocks) {
        if (speaks) flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t tile = (size_t)blk * Hkv + h;
    int8_t* exps = is_v ? a.v_exp : a.k_exp;
    const int e_old = clamp_exp(exps[tile]);
    // the largest magnitude, in the type's bits (their order is the values')
    uint32_t top = 0;
    int b = begin;   // the batch held
    for (;;) {
        uint32_t t = top;
#pragma unroll
        for (int i = 0; i < kRows / 2; ++i) {
            const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
            for (int k = 0; k < 4; ++k) t = __vmaxu2(t, w[k] & 0x7fff7fffu);
        }
        if (__any_sync(0xffffffffu, __vcmpgeu2(t, kInf2<T>) != 0)) {   // infinities and NaN do not count
#pragma unroll
            for (int i = 0; i < kRows / 2; ++i) {
                const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const uint32_t m = w[k] & 0x7fff7fffu;
                    top = __vmaxu2(top, m & ~__vcmpgeu2(m, kInf2<T>));
                }
            }
        } else {
            top = t;
        }
        if (b + stride_rows >= hi) break;
        b += stride_rows;
        load(b);
    }
    uint32_t amax = max(top & 0xffffu, top >> 16);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (wpu > 1) {
        if (lane == 0) amax_of[warp] = amax;
        asm volatile("bar.sync %0, %1;" ::"r"(1 + warp / wpu), "r"(wpu * 32) : "memory");
        for (int i = warp - part; i < warp - part + wpu; ++i) amax = max(amax, amax_of[i]);
    }
    const int need = exponent_for(Elem<T>::to_float((uint16_t)amax));   // (every lane has read the old exponent)
    const int e = lo == 0 ? need : max(e_old, need);
    uint8_t* dst = (is_v ? a.v_cache : a.k_cache) + tile * B * kHeadDim + c * 8;
    const float mul = exp2_int(-e);
    for (;;) {   // the batch held, then the earlier ones read again (from L2)
#pragma unroll
        for (int i = 0; i < kRows / 2; ++i) {
            const int r = b + lane / 16 + 2 * i;
            if (r < hi) *reinterpret_cast<uint2*>(dst + r * kHeadDim) = quantise8<T>(x[i], mul);
        }
        if (b == begin) break;
        b -= stride_rows;
        load(b);
    }
    if (e > e_old && lo > 0) rescale_rows(dst, part * 2 + lane / 16, lo, 2 * wpu, exp2_int(e_old - e));   // earlier rows
    if (part == 0 && lane == 0) exps[tile] = (int8_t)e;
}

// Two fp32 to two 16-bit values, to nearest; beyond the type's range to its largest value, NaN stays.
template <typename T>
__device__ __forceinline__ uint32_t pack2_sat(float lo, float hi);
template <>
__device__ __forceinline__ uint32_t pack2_sat<__half>(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.satfinite.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <>
__device__ __forceinline__ uint32_t pack2_sat<__nv_bfloat16>(float lo, float hi) {
    return Elem<__nv_bfloat16>::pack2(lo, hi);   // 448 * 2^60 is far inside bf16's range
}

template <typename T>
__device__ __forceinline__ void read16(uint4 codes, float mul, uint4* dst) {
    const uint32_t c[4] = {codes.x, codes.y, codes.z, codes.w};
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 p = e4m3x2_to_float2((uint16_t)(c[i] & 0xffffu));
        const float2 q = e4m3x2_to_float2((uint16_t)(c[i] >> 16));
        w[2 * i] = pack2_sat<T>(p.x * mul, p.y * mul);
        w[2 * i + 1] = pack2_sat<T>(q.x * mul, q.y * mul);
    }
    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
}

template <typename T>
__global__ void __launch_bounds__(256) read_q8_kernel(const ReadQ8Args a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const int per_block = a.num_kv_heads * a.vecs_per_head;
    const long long pair = i / per_block;
    if (pair >= a.num_pairs) return;
    const int v = (int)(i - pair * per_block);
    const int src = a.src_ids[pair], dst = a.dst_ids[pair];
    if (src < 0 || src >= a.src_blocks || dst < 0 || dst >= a.dst_blocks) {
        if (v == 0) flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
        return;
    }
    const size_t tile = (size_t)src * a.num_kv_heads + v / a.vecs_per_head;
    const size_t from = (size_t)src * per_block + v, to = ((size_t)dst * per_block + v) * 2;
    read16<T>(a.k_cache[from], exp2_int(clamp_exp(a.k_exp[tile])), a.dst_k + to);
    read16<T>(a.v_cache[from], exp2_int(clamp_exp(a.v_exp[tile])), a.dst_v + to);
}

}  // namespace

template <typename T>
static cudaError_t launch_append(const AppendQ8Args& a, cudaStream_t stream) {
    const dim3 block(kAppendWarps * 32);
    if (!a.q_start) {
        const long long warps = (long long)a.num_seqs * ((a.num_kv_heads + kOneHeads - 1) / kOneHeads);
        return launch_pdl(append_one_q8_kernel<T>, dim3((unsigned)((warps + kAppendWarps - 1) / kAppendWarps)), block, 0,
                          stream, a);
    }
    const int blocks = a.rows / a.block_size + 2 * a.num_seqs;
    // 64- and 128-row blocks of long chunks: 2 or 4 warps hold the rows in registers (one pass); of few rows: one
    // warp, whose idle neighbours would only fill the SMs
    const int wpu = a.block_size > 32 && a.rows / a.num_seqs >= a.block_size / 2 ? a.block_size / 32 : 1;
    const long long units = 2LL * blocks * a.num_kv_heads;
    const int per_cta = kAppendWarps / wpu;
    const dim3 grid((unsigned)((units + per_cta - 1) / per_cta));
    if (wpu > 1) return launch_pdl(append_q8_kernel<T, 32, 0, 3>, grid, block, 0, stream, a, blocks, wpu);
    switch (a.block_size) {
        case 16:
            if (a.rows / a.num_seqs >= a.block_size)
                return launch_pdl(append_q8_kernel<T, 16, 1, 4>, grid, block, 0, stream, a, blocks, 1);
            break;
        case 32: return launch_pdl(append_q8_kernel<T, 32, 1, 3>, grid, block, 0, stream, a, blocks, 1);
    }
    return launch_pdl(append_q8_kernel<T, 16, 1, 3>, grid, block, 0, stream, a, blocks, 1);
}

cudaError_t launch_append_q8(const AppendQ8Args& a, int dtype, cudaStream_t stream) {
    return dtype == PA_BF16 ? launch_append<__nv_bfloat16>(a, stream) : launch_append<__half>(a, stream);
}

cudaError_t launch_read_q8(const ReadQ8Args& a, int dtype, cudaStream_t stream) {
    const long long vecs = (long long)a.num_pairs * a.num_kv_heads * a.vecs_per_head;
    const dim3 grid((unsigned)((vecs + 255) / 256)), block(256);
    return dtype == PA_BF16 ? launch_pdl(read_q8_kernel<__nv_bfloat16>, grid, block, 0, stream, a)
                            : launch_pdl(read_q8_kernel<__half>, grid, block, 0, stream, a);
}

}  // namespace pa
