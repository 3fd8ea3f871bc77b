// Attention over the 8-bit paged cache: one query token per sequence, or several attending causally.
//
// What it computes ("显存虚拟化革命：PagedAttention 内存池管理与显存碎片终结", §五.1, over codes and
// exponents): for query row i of sequence s at position p = L - n + i and query head h,
//   out = sum_{t <= p} softmax_t(scale * q . (2^ke K_t)) * 2^ve V_t
// with K_t, V_t the codes of token t and ke, ve its block's exponents.  Tokens of a block whose table
// entry lies outside the pool are left out.
//
// Design: one warp per (query row, query head); a lane holds four elements of the head.  A running
// maximum and sum of the softmax in fp32, one pass over the tokens.
#include "q8.cuh"

namespace pa {

namespace {

template <typename T>
__global__ void __launch_bounds__(128) decode_q8_kernel(const DecodeQ8Args a) {
    grid_dependency_wait();
    grid_launch_dependents();
    const int lane = threadIdx.x % 32;
    const long long w = (long long)blockIdx.x * 4 + threadIdx.x / 32;
    const int h = (int)(w % a.num_q_heads);
    const long long si = w / a.num_q_heads;
    const int s = (int)(si / a.max_q), i = (int)(si % a.max_q);
    if (s >= a.num_seqs) return;
    bool bad_len;
    const int L = clamped_len(a.context_lens, s, a.max_blocks_per_seq, a.block_size, &bad_len);
    const NewRows nr = new_rows(a.q_start, a.q_rows, a.max_q, s, L);
    if ((bad_len || nr.bad) && i == 0 && h == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
    const int rows = a.q_start ? nr.n : 1;
    if (i >= rows) return;
    const size_t at = ((size_t)(nr.row0 + i) * a.num_q_heads + h) * kHeadDim + lane * 4;
    const int hk = h / (a.num_q_heads / a.num_kv_heads), B = a.block_size;
    const uint2 qu = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(a.q) + at);
    const float2 q0 = Elem<T>::to_float2(qu.x), q1 = Elem<T>::to_float2(qu.y);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    const int end = a.q_start ? L - nr.n + i + 1 : L;
    for (int t = 0; t < end; ++t) {
        const int blk = a.block_tables[(size_t)s * a.max_blocks_per_seq + t / B];
        if (blk < 0 || blk >= a.num_blocks) {
            if (h == 0 && lane == 0) flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
            continue;
        }
        const size_t tile = (size_t)blk * a.num_kv_heads + hk;
        const size_t row = (tile * B + t % B) * kHeadDim + lane * 4;
        const uint32_t kc = *reinterpret_cast<const uint32_t*>(a.k_cache + row);
        const uint32_t vc = *reinterpret_cast<const uint32_t*>(a.v_cache + row);
        const float2 k0 = e4m3x2_to_float2((uint16_t)kc), k1 = e4m3x2_to_float2((uint16_t)(kc >> 16));
        const float2 v0 = e4m3x2_to_float2((uint16_t)vc), v1 = e4m3x2_to_float2((uint16_t)(vc >> 16));
        const float ks = exp2_int(clamp_exp(a.k_exp[tile])), vs = exp2_int(clamp_exp(a.v_exp[tile]));
        const float x = warp_sum(q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y) * ks * a.scale_log2;
        const float m2 = fmaxf(m, x);
        const float keep = m == -INFINITY ? 0.f : exp2f(m - m2), p = exp2f(x - m2);
        l = l * keep + p;
        const float pv = p * vs;
        o[0] = o[0] * keep + pv * v0.x;
        o[1] = o[1] * keep + pv * v0.y;
        o[2] = o[2] * keep + pv * v1.x;
        o[3] = o[3] * keep + pv * v1.y;
        m = m2;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2 r;
    r.x = Elem<T>::pack2(o[0] * inv, o[1] * inv);
    r.y = Elem<T>::pack2(o[2] * inv, o[3] * inv);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + at) = r;
}

}  // namespace

size_t q8_workspace_bytes(int, int, int, int, int, int) { return 0; }

cudaError_t launch_decode_q8(const DecodeQ8Args& a, int dtype, void*, cudaStream_t stream) {
    const long long warps = (long long)a.num_seqs * a.max_q * a.num_q_heads;
    const dim3 grid((unsigned)((warps + 3) / 4)), block(128);
    return dtype == PA_BF16 ? launch_pdl(decode_q8_kernel<__nv_bfloat16>, grid, block, 0, stream, a)
                            : launch_pdl(decode_q8_kernel<__half>, grid, block, 0, stream, a);
}

}  // namespace pa
