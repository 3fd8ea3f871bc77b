// libpa C ABI of the rotary positions and the 8-bit cache: argument checks and dispatch.
#include "q8.cuh"

namespace pa {

namespace {

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

int finish(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    cudaGetLastError();
    return PA_ERR_CUDA;
}

bool bad_dtype(int dtype) { return dtype != PA_F16 && dtype != PA_BF16; }

// Shape of an 8-bit cache and its tables.
int check_q8_shape(int num_seqs, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                   int max_blocks_per_seq) {
    if (num_seqs < 0 || num_kv_heads <= 0 || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq < 0)
        return PA_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128))
        return PA_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || num_kv_heads > 65535) return PA_ERR_UNSUPPORTED;
    if ((long long)max_blocks_per_seq * block_size > (1LL << 30)) return PA_ERR_UNSUPPORTED;
    if ((long long)num_blocks * num_kv_heads * block_size > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

bool bad_cache(const void* k_cache, const void* v_cache, const void* k_exp, const void* v_exp) {
    return !k_cache || !v_cache || !k_exp || !v_exp || !aligned(k_cache, 16) || !aligned(v_cache, 16);
}

// Rows of `width` elements, `stride` apart: an operand of pa_rope in memory.
struct Rows {
    const char* p;
    long long width, stride;   // bytes
    int n;
    long long span() const { return (n - 1) * stride + width; }
};

// May the two share a byte?  (Rows of one stride that interleave, as the parts of one projection's
// output do, share none.)
bool overlap(const Rows& a, const Rows& b) {
    if (a.n == 0 || b.n == 0 || a.width == 0 || b.width == 0) return false;
    if (a.p + a.span() <= b.p || b.p + b.span() <= a.p) return false;
    if (a.stride != b.stride || a.stride == 0 || a.n == 1) return true;
    long long d = (b.p - a.p) % a.stride;
    if (d < 0) d += a.stride;
    return d < a.width || d + b.width > a.stride;
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

int pa_rope(void* out_q, void* out_k, const void* q, const void* k, long long out_q_stride, long long out_k_stride,
            long long q_stride, long long k_stride, const void* positions, int position_bytes, const double* inv_freq,
            float magnitude, int num_tokens, int num_q_heads, int num_kv_heads, int head_dim, int rotary_dim,
            int interleaved, int dtype, void* stream) {
    if (bad_dtype(dtype) || (position_bytes != 4 && position_bytes != 8)) return PA_ERR_INVALID_ARG;
    if (num_tokens < 0 || num_q_heads <= 0 || num_kv_heads < 0 || head_dim <= 0 || rotary_dim <= 0 ||
        rotary_dim > head_dim)
        return PA_ERR_INVALID_ARG;
    if (head_dim % 8 || rotary_dim % 16 || head_dim > kRopeMaxHead || num_q_heads > 65535 || num_kv_heads > 65535)
        return PA_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PA_OK;
    const bool has_k = num_kv_heads > 0;
    if (!out_q || !q || !positions || !inv_freq || (has_k && (!out_k || !k))) return PA_ERR_INVALID_ARG;
    if (!aligned(out_q, 16) || !aligned(q, 16) || (has_k && (!aligned(out_k, 16) || !aligned(k, 16))) ||
        !aligned(positions, position_bytes) || !aligned(inv_freq, 8))
        return PA_ERR_INVALID_ARG;
    const long long qw = (long long)num_q_heads * head_dim, kw = (long long)num_kv_heads * head_dim;
    // inputs may repeat a row (stride 0); outputs may not share elements
    if (q_stride < 0 || k_stride < 0 || q_stride % 8 || out_q_stride % 8 || (num_tokens > 1 && out_q_stride < qw))
        return PA_ERR_INVALID_ARG;
    if (has_k && (k_stride % 8 || out_k_stride % 8 || (num_tokens > 1 && out_k_stride < kw))) return PA_ERR_INVALID_ARG;
    const Rows in_q{static_cast<const char*>(q), 2 * qw, 2 * q_stride, num_tokens};
    const Rows in_k{static_cast<const char*>(k), 2 * kw, 2 * k_stride, has_k ? num_tokens : 0};
    const Rows to_q{static_cast<const char*>(out_q), 2 * qw, 2 * out_q_stride, num_tokens};
    const Rows to_k{static_cast<const char*>(out_k), 2 * kw, 2 * out_k_stride, has_k ? num_tokens : 0};
    const bool same_q = out_q == q && (out_q_stride == q_stride || num_tokens == 1);
    const bool same_k = has_k && out_k == k && (out_k_stride == k_stride || num_tokens == 1);
    if ((!same_q && overlap(to_q, in_q)) || (!same_k && overlap(to_k, in_k)) || overlap(to_q, in_k) ||
        overlap(to_k, in_q) || overlap(to_q, to_k))
        return PA_ERR_INVALID_ARG;
    RopeArgs a;
    a.q = q;
    a.k = k;
    a.out_q = out_q;
    a.out_k = out_k;
    a.q_stride = q_stride;
    a.k_stride = k_stride;
    a.out_q_stride = out_q_stride;
    a.out_k_stride = out_k_stride;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.magnitude = magnitude;
    a.wide_positions = position_bytes == 8;
    a.num_tokens = num_tokens;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved != 0;
    a.in_place_q = same_q;
    a.in_place_k = same_k;
    return finish(launch_rope(a, dtype, static_cast<cudaStream_t>(stream)));
}

int pa_cache_append_q8(const void* k, const void* v, long long k_stride, long long v_stride, void* k_cache,
                       void* v_cache, int8_t* k_exp, int8_t* v_exp, const int32_t* block_tables,
                       const int32_t* context_lens, const int32_t* query_start, int num_seqs, int num_tokens,
                       int max_q_per_seq, int num_kv_heads, int head_dim, int block_size, int num_blocks,
                       int max_blocks_per_seq, int dtype, void* stream) {
    if (bad_dtype(dtype) || num_tokens < 0 || max_q_per_seq < 1) return PA_ERR_INVALID_ARG;
    const int rc = check_q8_shape(num_seqs, num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq);
    if (rc != PA_OK) return rc;
    if (!query_start && num_tokens != num_seqs) return PA_ERR_INVALID_ARG;
    if (num_seqs == 0 || num_tokens == 0) return PA_OK;
    if (!k || !v || !block_tables || !context_lens || bad_cache(k_cache, v_cache, k_exp, v_exp))
        return PA_ERR_INVALID_ARG;
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(query_start, 4))
        return PA_ERR_INVALID_ARG;
    if (k_stride < 0 || v_stride < 0 || k_stride % 8 || v_stride % 8) return PA_ERR_INVALID_ARG;
    // one launch: its units must fit the grid
    if (2LL * (num_tokens / block_size + 2LL * num_seqs) * num_kv_heads > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    AppendQ8Args a;
    a.k = k;
    a.v = v;
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.k_cache = static_cast<uint8_t*>(k_cache);
    a.v_cache = static_cast<uint8_t*>(v_cache);
    a.k_exp = k_exp;
    a.v_exp = v_exp;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.q_start = query_start;
    a.status = device_status_ptr();
    a.num_seqs = num_seqs;
    a.rows = num_tokens;
    a.max_q = max_q_per_seq;
    a.num_kv_heads = num_kv_heads;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    a.max_blocks_per_seq = max_blocks_per_seq;
    return finish(launch_append_q8(a, dtype, static_cast<cudaStream_t>(stream)));
}

int pa_read_blocks_q8(const void* k_cache, const void* v_cache, const int8_t* k_exp, const int8_t* v_exp,
                      int src_blocks, void* dst_k, void* dst_v, int dst_blocks, const int32_t* src_ids,
                      const int32_t* dst_ids, int num_pairs, int num_kv_heads, int head_dim, int block_size, int dtype,
                      void* stream) {
    if (bad_dtype(dtype) || num_pairs < 0 || dst_blocks < 0) return PA_ERR_INVALID_ARG;
    if (num_pairs == 0) return PA_OK;
    const int rc = check_q8_shape(0, num_kv_heads, head_dim, block_size, src_blocks, 0);
    if (rc != PA_OK) return rc;
    if (!dst_k || !dst_v || !src_ids || !dst_ids || bad_cache(k_cache, v_cache, k_exp, v_exp))
        return PA_ERR_INVALID_ARG;
    if (!aligned(dst_k, 16) || !aligned(dst_v, 16) || !aligned(src_ids, 4) || !aligned(dst_ids, 4))
        return PA_ERR_INVALID_ARG;
    ReadQ8Args a;
    a.k_cache = static_cast<const uint4*>(k_cache);
    a.v_cache = static_cast<const uint4*>(v_cache);
    a.k_exp = k_exp;
    a.v_exp = v_exp;
    a.dst_k = static_cast<uint4*>(dst_k);
    a.dst_v = static_cast<uint4*>(dst_v);
    a.src_ids = src_ids;
    a.dst_ids = dst_ids;
    a.status = device_status_ptr();
    a.num_pairs = num_pairs;
    a.src_blocks = src_blocks;
    a.dst_blocks = dst_blocks;
    a.num_kv_heads = num_kv_heads;
    a.vecs_per_head = block_size * kHeadDim / 16;
    if (((long long)num_pairs * num_kv_heads * a.vecs_per_head + 255) / 256 > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    return finish(launch_read_q8(a, dtype, static_cast<cudaStream_t>(stream)));
}

static int q8_attention_shape(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                              int num_blocks, int max_blocks_per_seq, int max_q) {
    const int rc = check_q8_shape(num_seqs, num_kv_heads, head_dim, block_size, num_blocks, max_blocks_per_seq);
    if (rc != PA_OK) return rc;
    if (num_q_heads <= 0 || num_q_heads % num_kv_heads || max_q < 1) return PA_ERR_INVALID_ARG;
    if (num_q_heads > 65535 || (long long)(num_q_heads / num_kv_heads) * max_q > kQ8MaxRows) return PA_ERR_UNSUPPORTED;
    if (!q8_line_fits(num_seqs, num_kv_heads, block_size, max_blocks_per_seq)) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

size_t pa_decode_q8_workspace_size(int num_seqs, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
                                   int max_blocks_per_seq, int max_q_per_seq) {
    if (q8_attention_shape(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, 1, max_blocks_per_seq,
                           max_q_per_seq) != PA_OK)
        return 0;
    return q8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, max_q_per_seq, block_size, max_blocks_per_seq);
}

static int decode_q8_impl(void* out, const void* q, const void* k_cache, const void* v_cache, const int8_t* k_exp,
                          const int8_t* v_exp, const int32_t* block_tables, const int32_t* context_lens,
                          const int32_t* query_start, float scale, int num_kv_heads, int num_seqs, int num_q_tokens,
                          int max_q, int num_q_heads, int head_dim, int block_size, int num_blocks,
                          int max_blocks_per_seq, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (bad_dtype(dtype) || num_q_tokens < 0) return PA_ERR_INVALID_ARG;
    const int rc = q8_attention_shape(num_seqs, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                                      max_blocks_per_seq, max_q);
    if (rc != PA_OK) return rc;
    if (num_seqs == 0 || num_q_tokens == 0) return PA_OK;
    if (!out || !q || !block_tables || !context_lens || bad_cache(k_cache, v_cache, k_exp, v_exp))
        return PA_ERR_INVALID_ARG;
    if (!aligned(out, 16) || !aligned(q, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
        !aligned(query_start, 4))
        return PA_ERR_INVALID_ARG;
    const size_t need =
        q8_workspace_bytes(num_seqs, num_q_heads, num_kv_heads, max_q, block_size, max_blocks_per_seq);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16))) return PA_ERR_WORKSPACE;
    DecodeQ8Args a;
    a.out = out;
    a.q = q;
    a.k_cache = static_cast<const uint8_t*>(k_cache);
    a.v_cache = static_cast<const uint8_t*>(v_cache);
    a.k_exp = k_exp;
    a.v_exp = v_exp;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.q_start = query_start;
    a.status = device_status_ptr();
    a.scale_log2 = scale * 1.4426950408889634f;
    a.num_seqs = num_seqs;
    a.q_rows = num_q_tokens;
    a.max_q = max_q;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    a.max_blocks_per_seq = max_blocks_per_seq;
    return finish(launch_decode_q8(a, dtype, workspace, static_cast<cudaStream_t>(stream)));
}

int pa_decode_q8(void* out, const void* q, const void* k_cache, const void* v_cache, const int8_t* k_exp,
                 const int8_t* v_exp, const int32_t* block_tables, const int32_t* context_lens, float scale,
                 int num_kv_heads, int num_seqs, int num_q_heads, int head_dim, int block_size, int num_blocks,
                 int max_blocks_per_seq, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    return decode_q8_impl(out, q, k_cache, v_cache, k_exp, v_exp, block_tables, context_lens, nullptr, scale,
                          num_kv_heads, num_seqs, num_seqs, 1, num_q_heads, head_dim, block_size, num_blocks,
                          max_blocks_per_seq, dtype, workspace, workspace_bytes, stream);
}

int pa_multi_query_q8(void* out, const void* q, const void* k_cache, const void* v_cache, const int8_t* k_exp,
                      const int8_t* v_exp, const int32_t* block_tables, const int32_t* context_lens,
                      const int32_t* query_start, float scale, int num_kv_heads, int num_seqs, int num_q_tokens,
                      int max_q_per_seq, int num_q_heads, int head_dim, int block_size, int num_blocks,
                      int max_blocks_per_seq, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!query_start) return PA_ERR_INVALID_ARG;
    return decode_q8_impl(out, q, k_cache, v_cache, k_exp, v_exp, block_tables, context_lens, query_start, scale,
                          num_kv_heads, num_seqs, num_q_tokens, max_q_per_seq, num_q_heads, head_dim, block_size,
                          num_blocks, max_blocks_per_seq, dtype, workspace, workspace_bytes, stream);
}

}  // extern "C"
