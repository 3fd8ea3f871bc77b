// Rotary positions: pairs of a head's first R elements turned by the token's position.
//
// Pair i of a token at position p turns by the angle p * f_i:
//   (a, b) -> magnitude * (a cos - b sin, b cos + a sin)
// with (a, b) = elements (i, i + R/2) of the head, or (2i, 2i + 1) interleaved; elements R .. D-1
// are passed on as they are.
//
// The angle of a far position needs more than fp32 (p * f_i = 10^6 rad leaves 0.06 rad of it), and
// fp64 is slow here.  A turn is therefore 2^64: F_i = round(frac(f_i / 2 pi) * 2^64), and the product
// p * F_i modulo 2^64 is the reduced angle, exact by integer wrap-around (negative positions too).
// The phase's error is that of F_i, p * 2^-65 turns beside f_i's own in fp64.  It enters fp32 with 24 bits of its own
// size, so that small angles (slow pairs near position 0) keep them too: 2^-23 of the angle at most.
//
// Design: a CTA takes one to 16 tokens, so that the grid is whole waves.  Its threads first work out the tokens' R/2
// cosines and sines once (shared by all heads), with the first vectors of the heads already on their way, then each
// thread turns 16-byte vectors of one column of the heads, four in flight.  Every element is read and written once, and
// HBM bounds the work: 8192 tokens of 40 heads take 28.7 us, interleaved 30.8 (0.86 and 0.80 of a copy's rate; 4 to 26
// tokens a CTA, 2, 3 or 8 vectors in flight and 4 or 6 CTAs an SM took 31.5 to 36).  A step of 64 tokens takes 2.2 us,
// most of it the launch.
#include "q8.cuh"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;   // 128 where one vector per thread is enough
static_assert(kRopeMaxHead / 8 <= 128, "a CTA has a thread for each column of a head");
// CTAs of 256 threads per SM: 48 registers a thread.  A grid that fits with fewer has an instance of 64, whose loads
// are further ahead (1024 tokens of 40 heads 5.8 us against 7.1; as one for all sizes 8192 tokens 30.1 to 33.1 against
// 28.7 to 30.8).
constexpr int kRopePerSm = 5, kRopePerSmFew = 4;
constexpr int kRopeTokens = 16;     // tokens of a CTA at most; their cosines and sines fit in 48 KB
constexpr int kRopePairs = 48 * 1024 / (int)sizeof(float2);

__device__ __forceinline__ uint64_t turns64(double f) {
    const double t = f * 0.15915494309189533577;   // 1 / (2 pi)
    return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of a phase of 2^64 per turn.
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
    float s, c;
    // half turns in [-1, 1] from the phase's halves, both signed (one 64-bit conversion would take 0.3 us of 31)
    const int low = (int32_t)phase, high = (int32_t)(uint32_t)((phase + 0x80000000u) >> 32);
    sincospif(fmaf((float)low, 0x1p-63f, (float)high * 0x1p-31f), &s, &c);
    return make_float2(c, s);
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    uint4 u;
    u.x = Elem<T>::pack2(f[0], f[1]);
    u.y = Elem<T>::pack2(f[2], f[3]);
    u.z = Elem<T>::pack2(f[4], f[5]);
    u.w = Elem<T>::pack2(f[6], f[7]);
    return u;
}

template <typename T, bool kInterleaved, int kPerSm>
__global__ void __launch_bounds__(kRopeThreads, kPerSm) rope_kernel(const RopeArgs a, int tokens) {
    constexpr int kBatch = kInterleaved ? 4 : 2;   // vectors, or pairs of them, of a thread in flight
    extern __shared__ float4 cs4[];   // [tokens][R / 2] (cos, sin), magnitude included
    float2* cs = reinterpret_cast<float2*>(cs4);
    grid_dependency_wait();
    grid_launch_dependents();
    const int t0 = blockIdx.x * tokens, n = min(tokens, a.num_tokens - t0);
    const int pairs = a.rotary_dim / 2, vecs = a.head_dim / 8, heads = a.num_q_heads + a.num_kv_heads;
    const int rot = a.rotary_dim / 8, half = rot / 2, turned = kInterleaved ? rot : half;
    // A thread keeps to one column of the heads: a turned vector (two, one of each half, in the half layout), or
    // one that is passed on; of the CTA's heads, token after token, it takes every `step`-th.
    const int columns = turned + vecs - rot, step = (int)blockDim.x / columns;   // at most 128 columns
    const int first = threadIdx.x / columns, step_t = step / heads, step_h = step - step_t * heads;
    const int col = threadIdx.x - first * columns;
    const bool turns = col < turned;
    const int at = turns ? col : col + rot - turned;
    struct Cursor {
        int t, h;
    };
    auto next = [&](Cursor& c) {
        c.h += step_h;
        c.t += step_t;
        if (c.h >= heads) {
            c.h -= heads;
            ++c.t;
        }
    };
    auto in_of = [&](const Cursor& c) {
        const long long t = t0 + c.t;
        return (c.h < a.num_q_heads
                    ? reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + t * a.q_stride) + c.h * vecs
                    : reinterpret_cast<const uint4*>(static_cast<const T*>(a.k) + t * a.k_stride) + (c.h - a.num_q_heads) * vecs) + at;
    };
    auto out_of = [&](const Cursor& c) {
        const long long t = t0 + c.t;
        return (c.h < a.num_q_heads
                    ? reinterpret_cast<uint4*>(static_cast<T*>(a.out_q) + t * a.out_q_stride) + c.h * vecs
                    : reinterpret_cast<uint4*>(static_cast<T*>(a.out_k) + t * a.out_k_stride) + (c.h - a.num_q_heads) * vecs) + at;
    };
    Cursor from{first < step ? first / heads : n, first % heads}, to = from;
    uint4 x[kBatch], y[kInterleaved ? 1 : kBatch];
    auto load = [&]() {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (from.t < n) {
                const uint4* src = in_of(from);
                x[k] = src[0];
                if (!kInterleaved && turns) y[kInterleaved ? 0 : k] = src[half];
                next(from);
            }
        }
    };
    load();   // on their way while the angles are worked out
    // a thread keeps to one pair (its frequency costs five fp64 operations) and takes tokens in turn
    const int lanes = min(pairs, (int)blockDim.x), groups = blockDim.x / lanes, group = threadIdx.x / lanes;
    if (group < groups)
        for (int f = threadIdx.x - group * lanes; f < pairs; f += lanes) {
            const uint64_t turn = turns64(a.inv_freq[f]);
            for (int t = group; t < n; t += groups) {
                const long long p = a.wide_positions ? static_cast<const long long*>(a.positions)[t0 + t]
                                                     : (long long)static_cast<const int32_t*>(a.positions)[t0 + t];
                const float2 w = cos_sin((uint64_t)p * turn);
                cs[t * pairs + f] = make_float2(w.x * a.magnitude, w.y * a.magnitude);
            }
        }
    __syncthreads();
    while (to.t < n) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (to.t < n) {
                uint4* dst = out_of(to);
                if (!turns) {
                    if (!(to.h < a.num_q_heads ? a.in_place_q : a.in_place_k)) dst[0] = x[k];
                } else if (kInterleaved) {   // four pairs
                    const float4* w4 = cs4 + (to.t * pairs + col * 4) / 2;
                    float f[8], r[8];
                    unpack8<T>(x[k], f);
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const float4 w = w4[j];
                        r[4 * j] = f[4 * j] * w.x - f[4 * j + 1] * w.y;
                        r[4 * j + 1] = f[4 * j + 1] * w.x + f[4 * j] * w.y;
                        r[4 * j + 2] = f[4 * j + 2] * w.z - f[4 * j + 3] * w.w;
                        r[4 * j + 3] = f[4 * j + 3] * w.z + f[4 * j + 2] * w.w;
                    }
                    dst[0] = pack8<T>(r);
                } else {                     // eight pairs, a vector of each half
                    const float4* w4 = cs4 + (to.t * pairs + col * 8) / 2;
                    float f[8], g[8], rf[8], rg[8];
                    unpack8<T>(x[k], f);
                    unpack8<T>(y[kInterleaved ? 0 : k], g);
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const float4 w = w4[j];
                        rf[2 * j] = f[2 * j] * w.x - g[2 * j] * w.y;
                        rg[2 * j] = g[2 * j] * w.x + f[2 * j] * w.y;
                        rf[2 * j + 1] = f[2 * j + 1] * w.z - g[2 * j + 1] * w.w;
                        rg[2 * j + 1] = g[2 * j + 1] * w.z + f[2 * j + 1] * w.w;
                    }
                    dst[0] = pack8<T>(rf);
                    dst[half] = pack8<T>(rg);
                }
                next(to);
            }
        }
        load();
    }
}

}  // namespace

template <typename T>
static cudaError_t launch_type(const RopeArgs& a, cudaStream_t stream) {
    const int rot = a.rotary_dim / 8, per_head = (a.interleaved ? rot : rot / 2) + a.head_dim / 8 - rot;
    // whole waves of CTAs, each CTA with at most kRopeTokens tokens
    const long long slots = kRopePerSm * sm_count_current();
    const long long most = slots * min(kRopeTokens, kRopePairs / (a.rotary_dim / 2));
    const long long waves = (a.num_tokens + most - 1) / most;
    const int tokens = (int)((a.num_tokens + slots * waves - 1) / (slots * waves));
    const bool small = tokens * (a.num_q_heads + a.num_kv_heads) * per_head <= 128;
    const dim3 grid((unsigned)(((long long)a.num_tokens + tokens - 1) / tokens)), block(small ? 128 : kRopeThreads);
    const size_t smem = (size_t)tokens * (a.rotary_dim / 2) * sizeof(float2);
    if (grid.x <= kRopePerSmFew * (unsigned)sm_count_current())
        return a.interleaved ? launch_pdl(rope_kernel<T, true, kRopePerSmFew>, grid, block, smem, stream, a, tokens)
                             : launch_pdl(rope_kernel<T, false, kRopePerSmFew>, grid, block, smem, stream, a, tokens);
    return a.interleaved ? launch_pdl(rope_kernel<T, true, kRopePerSm>, grid, block, smem, stream, a, tokens)
                         : launch_pdl(rope_kernel<T, false, kRopePerSm>, grid, block, smem, stream, a, tokens);
}

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t stream) {
    return dtype == PA_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<__half>(a, stream);
}

}  // namespace pa
