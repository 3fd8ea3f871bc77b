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
// Design: one CTA per token.  Its threads first work out the R/2 cosines and sines once (shared by
// all heads), then each thread turns 16-byte vectors of the heads.  The work is bound by HBM: every
// element is read and written once.
#include "q8.cuh"

namespace pa {

namespace {

constexpr int kRopeThreads = 128;

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

template <typename T>
__device__ __forceinline__ void turn_head(const uint4* in, uint4* out, const float2* cs, int item, int half_vecs,
                                          bool interleaved) {
    if (interleaved) {   // item = vector of four pairs
        float x[8], y[8];
        unpack8<T>(in[item], x);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 w = cs[item * 4 + i];
            y[2 * i] = x[2 * i] * w.x - x[2 * i + 1] * w.y;
            y[2 * i + 1] = x[2 * i + 1] * w.x + x[2 * i] * w.y;
        }
        out[item] = pack8<T>(y);
    } else {             // item = eight pairs, a vector of each half
        float a[8], b[8], ya[8], yb[8];
        unpack8<T>(in[item], a);
        unpack8<T>(in[item + half_vecs], b);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 w = cs[item * 8 + i];
            ya[i] = a[i] * w.x - b[i] * w.y;
            yb[i] = b[i] * w.x + a[i] * w.y;
        }
        out[item] = pack8<T>(ya);
        out[item + half_vecs] = pack8<T>(yb);
    }
}

template <typename T>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const RopeArgs a) {
    extern __shared__ float2 cs[];   // [R / 2] cos, sin (magnitude included)
    grid_dependency_wait();
    grid_launch_dependents();
    const int t = blockIdx.x;
    const long long p = a.wide_positions ? static_cast<const long long*>(a.positions)[t]
                                         : (long long)static_cast<const int32_t*>(a.positions)[t];
    for (int i = threadIdx.x; i < a.rotary_dim / 2; i += blockDim.x) {
        const float2 w = cos_sin((uint64_t)p * turns64(a.inv_freq[i]));
        cs[i] = make_float2(w.x * a.magnitude, w.y * a.magnitude);
    }
    __syncthreads();
    const int vecs = a.head_dim / 8, rot_vecs = a.rotary_dim / 8, half_vecs = rot_vecs / 2;
    const int items = a.interleaved ? rot_vecs : half_vecs;      // turned vectors (pairs of vectors) per head
    const int rest = vecs - rot_vecs;
    const int heads = a.num_q_heads + a.num_kv_heads;
    const int per_head = items + rest;
    for (int i = threadIdx.x; i < heads * per_head; i += blockDim.x) {
        const int h = i / per_head, item = i - h * per_head;
        const bool is_q = h < a.num_q_heads;
        const int hh = is_q ? h : h - a.num_q_heads;
        const uint4* in = reinterpret_cast<const uint4*>(static_cast<const T*>(is_q ? a.q : a.k) +
                                                         (long long)t * (is_q ? a.q_stride : a.k_stride)) + hh * vecs;
        uint4* out = reinterpret_cast<uint4*>(static_cast<T*>(is_q ? a.out_q : a.out_k) +
                                              (long long)t * (is_q ? a.out_q_stride : a.out_k_stride)) + hh * vecs;
        if (item < items)
            turn_head<T>(in, out, cs, item, half_vecs, a.interleaved != 0);
        else if (!(is_q ? a.in_place_q : a.in_place_k))
            out[rot_vecs + item - items] = in[rot_vecs + item - items];
    }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int dtype, cudaStream_t stream) {
    const dim3 grid((unsigned)a.num_tokens), block(kRopeThreads);
    const size_t smem = (size_t)a.rotary_dim / 2 * sizeof(float2);
    return dtype == PA_BF16 ? launch_pdl(rope_kernel<__nv_bfloat16>, grid, block, smem, stream, a)
                            : launch_pdl(rope_kernel<__half>, grid, block, smem, stream, a);
}

}  // namespace pa
