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
// The error is that of F_i, p * 2^-65 turns beside f_i's own in fp64.
//
// Design: a CTA takes one to eight tokens.  Its threads first work out the tokens' R/2 cosines and sines once
// (shared by all heads), with the first vectors of the heads already on their way, then each thread turns
// 16-byte vectors, four in flight.  The work is bound by HBM: every element is read and written once.
#include "q8.cuh"

namespace pa {

namespace {

constexpr int kRopeThreads = 256;   // 128 where one vector per thread is enough
constexpr int kRopeBatch = 4;       // vectors (pairs of vectors) of a thread in flight
constexpr int kRopeTokens = 8;      // tokens of a CTA at most

__device__ __forceinline__ uint64_t turns64(double f) {
    const double t = f * 0.15915494309189533577;   // 1 / (2 pi)
    return __double2ull_rn((t - floor(t)) * 18446744073709551616.0);
}

// cos and sin of a phase of 2^64 per turn.
__device__ __forceinline__ float2 cos_sin(uint64_t phase) {
    float s, c;
    sincospif((float)(int32_t)(phase >> 32) * (1.f / 2147483648.f), &s, &c);   // half turns in [-1, 1)
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

// Vector `i` of a CTA's work: its token, its head's first vectors, and its index in the head: the turned
// vectors first (pairs of vectors in the half layout), then those passed on.
struct Item {
    const uint4* in;
    uint4* out;
    int t, v;
    bool keep;   // passed on in place: nothing to do
};

template <typename T>
__device__ __forceinline__ Item item_at(const RopeArgs& a, unsigned t0, unsigned i, unsigned per_head, unsigned turned) {
    const unsigned heads = a.num_q_heads + a.num_kv_heads;
    const unsigned th = i / per_head, t = th / heads, h = th - t * heads, v = i - th * per_head;
    const bool is_q = h < (unsigned)a.num_q_heads;
    const unsigned at = (is_q ? h : h - a.num_q_heads) * (a.head_dim / 8);
    const long long tok = t0 + t;
    return Item{reinterpret_cast<const uint4*>(static_cast<const T*>(is_q ? a.q : a.k) + tok * (is_q ? a.q_stride : a.k_stride)) + at,
                reinterpret_cast<uint4*>(static_cast<T*>(is_q ? a.out_q : a.out_k) + tok * (is_q ? a.out_q_stride : a.out_k_stride)) + at,
                (int)t, (int)v, v >= turned && (is_q ? a.in_place_q : a.in_place_k)};
}

template <typename T, bool kInterleaved>
__global__ void __launch_bounds__(kRopeThreads, 4) rope_kernel(const RopeArgs a, int tokens) {
    extern __shared__ float2 cs[];   // [tokens][R / 2] cos, sin (magnitude included)
    grid_dependency_wait();
    grid_launch_dependents();
    const int t0 = blockIdx.x * tokens, n = min(tokens, a.num_tokens - t0);
    const int pairs = a.rotary_dim / 2;
    const int rot = a.rotary_dim / 8, half = rot / 2, turned = kInterleaved ? rot : half;
    const int rest = rot - turned;   // where the vectors passed on begin, less `turned`
    const int per_head = turned + a.head_dim / 8 - rot;
    const int items = n * (a.num_q_heads + a.num_kv_heads) * per_head;
    uint4 x[kRopeBatch], y[kInterleaved ? 1 : kRopeBatch];
    auto load = [&](int i0) {
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            const int i = i0 + k * blockDim.x;
            if (i < items) {
                const Item it = item_at<T>(a, t0, i, per_head, turned);
                x[k] = it.in[it.v >= turned ? it.v + rest : it.v];
                if (!kInterleaved && it.v < turned) y[kInterleaved ? 0 : k] = it.in[it.v + half];
            }
        }
    };
    load(threadIdx.x);   // on their way while the angles are worked out
    for (int i = threadIdx.x; i < n * pairs; i += blockDim.x) {
        const int t = i / pairs, f = i - t * pairs;
        const long long p = a.wide_positions ? static_cast<const long long*>(a.positions)[t0 + t]
                                             : (long long)static_cast<const int32_t*>(a.positions)[t0 + t];
        const float2 w = cos_sin((uint64_t)p * turns64(a.inv_freq[f]));
        cs[i] = make_float2(w.x * a.magnitude, w.y * a.magnitude);
    }
    __syncthreads();
    for (int i0 = threadIdx.x;;) {
#pragma unroll
        for (int k = 0; k < kRopeBatch; ++k) {
            const int i = i0 + k * blockDim.x;
            if (i >= items) break;
            const Item it = item_at<T>(a, t0, i, per_head, turned);
            if (it.v >= turned) {
                if (!it.keep) it.out[it.v + rest] = x[k];
            } else if (kInterleaved) {   // four pairs
                float f[8], r[8];
                unpack8<T>(x[k], f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 w = cs[it.t * pairs + it.v * 4 + j];
                    r[2 * j] = f[2 * j] * w.x - f[2 * j + 1] * w.y;
                    r[2 * j + 1] = f[2 * j + 1] * w.x + f[2 * j] * w.y;
                }
                it.out[it.v] = pack8<T>(r);
            } else {                     // eight pairs, a vector of each half
                float f[8], g[8], rf[8], rg[8];
                unpack8<T>(x[k], f);
                unpack8<T>(y[kInterleaved ? 0 : k], g);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const float2 w = cs[it.t * pairs + it.v * 8 + j];
                    rf[j] = f[j] * w.x - g[j] * w.y;
                    rg[j] = g[j] * w.x + f[j] * w.y;
                }
                it.out[it.v] = pack8<T>(rf);
                it.out[it.v + half] = pack8<T>(rg);
            }
        }
        i0 += kRopeBatch * blockDim.x;
        if (i0 >= items) break;
        load(i0);
    }
}

}  // namespace

template <typename T>
static cudaError_t launch_type(const RopeArgs& a, cudaStream_t stream) {
    const int rot = a.rotary_dim / 8, per_head = (a.interleaved ? rot : rot / 2) + a.head_dim / 8 - rot;
    // as many tokens to a CTA as leave four CTAs to every SM, eight at most
    const int tokens = max(1, min(kRopeTokens, a.num_tokens / (4 * sm_count_current())));
    const bool small = tokens * (a.num_q_heads + a.num_kv_heads) * per_head <= 128;
    const dim3 grid((unsigned)((a.num_tokens + tokens - 1) / tokens)), block(small ? 128 : kRopeThreads);
    const size_t smem = (size_t)tokens * (a.rotary_dim / 2) * sizeof(float2);
    return a.interleaved ? launch_pdl(rope_kernel<T, true>, grid, block, smem, stream, a, tokens)
                         : launch_pdl(rope_kernel<T, false>, grid, block, smem, stream, a, tokens);
}

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t stream) {
    return dtype == PA_BF16 ? launch_type<__nv_bfloat16>(a, stream) : launch_type<__half>(a, stream);
}

}  // namespace pa
