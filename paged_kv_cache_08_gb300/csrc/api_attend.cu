// libpa C ABI of attention with capped, biased and masked scores and of attention over shared prefixes: argument checks,
// workspaces and dispatch.
#include <cmath>

#include "attend.cuh"

namespace pa {

namespace {

inline bool aligned(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

int finish(cudaError_t e) {
    if (e == cudaSuccess) return PA_OK;
    cudaGetLastError();
    return PA_ERR_CUDA;
}

int check_shape(int num_seqs, int num_q_tokens, int max_q, int num_q_heads, int num_kv_heads, int head_dim,
                int block_size, int num_blocks, int max_blocks_per_seq) {
    if (num_seqs < 0 || num_q_tokens < 0 || max_q < 1 || num_kv_heads <= 0 || num_q_heads <= 0 ||
        num_q_heads % num_kv_heads || block_size <= 0 || num_blocks <= 0 || max_blocks_per_seq < 0)
        return PA_ERR_INVALID_ARG;
    if (head_dim != kHeadDim || (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128))
        return PA_ERR_UNSUPPORTED;
    if (num_seqs > 65535 || num_q_heads > 65535 || num_kv_heads > 32767 || (long long)num_q_tokens * num_q_heads > 0x7fffffffLL)
        return PA_ERR_UNSUPPORTED;
    if ((long long)max_blocks_per_seq * block_size > (1LL << 30)) return PA_ERR_UNSUPPORTED;
    if ((long long)num_blocks * num_kv_heads * block_size > 0x7fffffffLL) return PA_ERR_UNSUPPORTED;
    if (!stream_line_fits(num_seqs, num_kv_heads, block_size, max_blocks_per_seq)) return PA_ERR_UNSUPPORTED;
    return PA_OK;
}

// How a call runs, and where its partial results lie in the workspace.
struct Dispatch {
    bool stream;          // every sequence's own keys by attend_stream.cu, else by attend_tc.cu
    int stream_ctas;
    TcSplits own;         // of the latter
    TcSplits prefix;      // the shared prefixes' keys (splits 0: none)
    int own_slots;        // partial results of a row
    bool partial;
    size_t o, ml, stream_ws, bytes;
};

Dispatch dispatch(int num_seqs, int num_q_tokens, int max_q, int num_q_heads, int num_kv_heads, int block_size,
                  int max_blocks_per_seq, int num_groups, int max_prefix_blocks) {
    Dispatch d;
    const int group = num_q_heads / num_kv_heads, sms = sm_count_current();
    // Query rows of all sequences, whose counts the kernels clamp, and of all groups, whose tiles lie over all rows from the
    // first sequence's to the last one's, those that a clamped count leaves out among them.
    const long long rows = min((long long)num_q_tokens, (long long)num_seqs * max_q) * group;
    const long long group_rows = (long long)num_q_tokens * group;
    const long long keys = (long long)max_blocks_per_seq * block_size, prefix = (long long)max_prefix_blocks * block_size;
    d.stream = (long long)group * max_q <= kStreamRows;
    // Where the tables bound all contexts together to 16 MB, reading the prefix for every sequence costs less than the
    // launches that join the parts (4 sequences of 260 to 320 tokens 10 us against 14.5; the two meet near 20 MB).
    const bool small = d.stream && keys * num_seqs * num_kv_heads <= (16LL << 20) / (2 * kHeadDim * 2);
    const bool shared = num_groups > 0 && max_prefix_blocks > 0 && !small;
    d.prefix = TcSplits{0, 0};
    d.own = TcSplits{0, 1};
    int most = 0;   // CTAs of the streaming kernel
    if (shared) {
        int tc_sms = sms;
        if (d.stream) {
            // Both parts run side by side, each on SMs of its own: the split that the model of their times finds best.  A
            // stage takes a CTA with two tiles 1.1 us, a streaming CTA reads 60 KB in 1 us with up to 8 rows a segment and
            // half of that with more, all together 6 TB/s (6000 KB a microsecond); half the rest of the tables is taken for the
            // tails' length, which is not known here.
            const TcSplits one = tc_splits(group_rows, num_groups, num_kv_heads, prefix, 1, sms);
            const double stages = (double)one.items * num_kv_heads * (double)(prefix / 64 + 1);
            const bool few = group * max_q <= 8;
            const double kb = (group * max_q > kSegmentRows ? 1.0 : 0.5) * num_kv_heads * num_seqs *
                              (0.5 * (double)max(0LL, keys - prefix) + block_size);
            double best = 1e30;
            for (int n = 8; n <= sms - 8; n += 8) {
                const double t = max(6.0 + 1.1 * stages / (sms - n), 4.0 + kb / min((few ? 60.0 : 30.0) * n, 6000.0));
                if (t < best) {
                    best = t;
                    most = n;
                }
            }
            tc_sms = sms - most;
        }
        d.prefix = tc_splits(group_rows, num_groups, num_kv_heads, prefix, kMostPrefix, tc_sms);
    }
    if (!d.stream) d.own = tc_splits(rows, num_seqs, num_kv_heads, keys, kMostOwn, sms);
    d.stream_ctas = d.stream ? stream_ctas(num_seqs, num_kv_heads, group * max_q, block_size, max_blocks_per_seq, most) : 0;
    d.own_slots = d.own.splits;
    d.partial = shared || d.own.splits > 1;
    const size_t all = (size_t)num_q_tokens * num_q_heads, slots = d.partial ? d.own_slots + d.prefix.splits : 0;
    d.o = 0;
    d.ml = align256(slots * all * kHeadDim * sizeof(float));
    d.stream_ws = d.ml + align256(slots * all * sizeof(float2));
    d.bytes = d.stream_ws;
    if (d.stream) d.bytes += stream_workspace_bytes(num_seqs, d.stream_ctas, group * max_q);
    return d;
}

// Caps so far from the scores that the kernels' fp32 would leave its range are put within it.  A cap of 2^-64 or less leaves
// every score within 2^-64 of zero, whose weights are all one; under one of 2^80 |scale| and more no product below 2^68 is
// changed by as much as its own rounding.
void normalise_cap(AttendArgs* a) {
    if (a->cap == 0.f) return;
    if (a->cap <= 0x1p-64f) {
        a->cap = a->scale = 0.f;
    } else if (a->cap >= 0x1p80 * std::fabs((double)a->scale)) {
        a->cap = 0.f;
    } else {
        a->cap = std::fmin(a->cap, 0x1p120f);
        const double most = 0x1p90 * a->cap;   // (scores of other than zero are +-cap)
        if (std::fabs(a->scale) > most) a->scale = std::copysign((float)most, a->scale);
    }
}

int run(AttendArgs a, int head_dim, int dtype, void* workspace, size_t workspace_bytes, void* stream_ptr) {
    if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_INVALID_ARG;
    const int rc = check_shape(a.num_seqs, a.q_rows, a.max_q, a.num_q_heads, a.num_kv_heads, head_dim, a.block_size,
                               a.num_blocks, a.max_blocks_per_seq);
    if (rc != PA_OK) return rc;
    if (!(a.cap >= 0.f) || !std::isfinite(a.cap)) return PA_ERR_INVALID_ARG;
    if (a.num_seqs == 0 || a.q_rows == 0) return PA_OK;
    if (!a.out || !a.q || !a.k_cache || !a.v_cache || !a.block_tables || !a.context_lens) return PA_ERR_INVALID_ARG;
    if (!aligned(a.out, 16) || !aligned(a.q, 16) || !aligned(a.k_cache, 16) || !aligned(a.v_cache, 16) ||
        !aligned(a.block_tables, 4) || !aligned(a.context_lens, 4) || !aligned(a.q_start, 4) || !aligned(a.slopes, 4) ||
        !aligned(a.first_key, 4) || !aligned(a.bidirectional, 4))
        return PA_ERR_INVALID_ARG;
    const Dispatch d = dispatch(a.num_seqs, a.q_rows, a.max_q, a.num_q_heads, a.num_kv_heads, a.block_size,
                                a.max_blocks_per_seq, a.num_groups, a.max_prefix_blocks);
    if (d.bytes && (!workspace || workspace_bytes < d.bytes || !aligned(workspace, 16))) return PA_ERR_WORKSPACE;
    const cudaStream_t stream = static_cast<cudaStream_t>(stream_ptr);
    char* ws = static_cast<char*>(workspace);
    a.status = device_status_ptr();
    normalise_cap(&a);
    if (d.partial) {
        a.part_o = reinterpret_cast<float*>(ws + d.o);
        a.part_ml = reinterpret_cast<float2*>(ws + d.ml);
    }
    if (!d.prefix.splits) a.prefix_lens = nullptr;
    cudaError_t e = cudaSuccess;
    if (d.prefix.splits) e = launch_attend_tc(a, dtype, kPrefixKeys, d.prefix, d.own_slots, stream);
    if (e == cudaSuccess)
        e = d.stream ? launch_attend_stream(a, dtype, d.stream_ctas, d.prefix.splits > 0, ws + d.stream_ws, stream)
                     : launch_attend_tc(a, dtype, d.prefix.splits ? kTailKeys : kAllKeys, d.own, 0, stream);
    if (e == cudaSuccess && d.partial) e = launch_attend_combine(a, dtype, d.own_slots, d.prefix.splits, stream);
    return finish(e);
}

AttendArgs args_of(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                   const int32_t* context_lens, const int32_t* query_start, float scale, int num_kv_heads, int num_seqs,
                   int num_q_tokens, int max_q, int num_q_heads, int block_size, int num_blocks, int max_blocks_per_seq) {
    AttendArgs a = {};
    a.out = out;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.q_start = query_start;
    a.scale = scale;
    a.num_seqs = num_seqs;
    a.q_rows = num_q_tokens;
    a.max_q = max_q;
    a.num_q_heads = num_q_heads;
    a.num_kv_heads = num_kv_heads;
    a.block_size = block_size;
    a.num_blocks = num_blocks;
    a.max_blocks_per_seq = max_blocks_per_seq;
    return a;
}

// The prefix of a shared call; PA_OK, or what is wrong with it.
int add_prefix(AttendArgs& a, const int32_t* prefix_tables, const int32_t* prefix_lens, const int32_t* group_start,
               int num_groups, int max_prefix_blocks) {
    if (num_groups < 0 || max_prefix_blocks < 0) return PA_ERR_INVALID_ARG;
    if (num_groups > 65535 || (long long)max_prefix_blocks * a.block_size > (1LL << 30)) return PA_ERR_UNSUPPORTED;
    if (num_groups == 0 || max_prefix_blocks == 0) return PA_OK;
    if (a.num_seqs > 0 && a.q_rows > 0 &&
        (!prefix_tables || !prefix_lens || !group_start || !aligned(prefix_tables, 4) || !aligned(prefix_lens, 4) ||
         !aligned(group_start, 4)))
        return PA_ERR_INVALID_ARG;
    a.prefix_tables = prefix_tables;
    a.prefix_lens = prefix_lens;
    a.group_start = group_start;
    a.num_groups = num_groups;
    a.max_prefix_blocks = max_prefix_blocks;
    return PA_OK;
}

}  // namespace

}  // namespace pa

using namespace pa;

extern "C" {

int pa_decode_scored(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                     const int32_t* context_lens, float scale, float cap, const float* slopes, const int32_t* first_key,
                     int num_kv_heads, int num_seqs, int num_q_heads, int head_dim, int block_size, int num_blocks,
                     int max_blocks_per_seq, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    AttendArgs a = args_of(out, q, k_cache, v_cache, block_tables, context_lens, nullptr, scale, num_kv_heads, num_seqs,
                           num_seqs, 1, num_q_heads, block_size, num_blocks, max_blocks_per_seq);
    a.cap = cap;
    a.slopes = slopes;
    a.first_key = first_key;
    return run(a, head_dim, dtype, workspace, workspace_bytes, stream);
}

int pa_multi_query_scored(void* out, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                          float scale, float cap, const float* slopes, const int32_t* first_key,
                          const int32_t* bidirectional, int num_kv_heads, int num_seqs, int num_q_tokens,
                          int max_q_per_seq, int num_q_heads, int head_dim, int block_size, int num_blocks,
                          int max_blocks_per_seq, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    if (!query_start) return PA_ERR_INVALID_ARG;
    AttendArgs a = args_of(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, num_kv_heads,
                           num_seqs, num_q_tokens, max_q_per_seq, num_q_heads, block_size, num_blocks,
                           max_blocks_per_seq);
    a.cap = cap;
    a.slopes = slopes;
    a.first_key = first_key;
    a.bidirectional = bidirectional;
    return run(a, head_dim, dtype, workspace, workspace_bytes, stream);
}

int pa_decode_shared(void* out, const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                     const int32_t* context_lens, const int32_t* prefix_tables, const int32_t* prefix_lens,
                     const int32_t* group_start, int num_groups, int max_prefix_blocks, float scale, int num_kv_heads,
                     int num_seqs, int num_q_heads, int head_dim, int block_size, int num_blocks,
                     int max_blocks_per_seq, int dtype, void* workspace, size_t workspace_bytes, void* stream) {
    AttendArgs a = args_of(out, q, k_cache, v_cache, block_tables, context_lens, nullptr, scale, num_kv_heads, num_seqs,
                           num_seqs, 1, num_q_heads, block_size, num_blocks, max_blocks_per_seq);
    const int rc = add_prefix(a, prefix_tables, prefix_lens, group_start, num_groups, max_prefix_blocks);
    return rc != PA_OK ? rc : run(a, head_dim, dtype, workspace, workspace_bytes, stream);
}

int pa_multi_query_shared(void* out, const void* q, const void* k_cache, const void* v_cache,
                          const int32_t* block_tables, const int32_t* context_lens, const int32_t* query_start,
                          const int32_t* prefix_tables, const int32_t* prefix_lens, const int32_t* group_start,
                          int num_groups, int max_prefix_blocks, float scale, int num_kv_heads, int num_seqs,
                          int num_q_tokens, int max_q_per_seq, int num_q_heads, int head_dim, int block_size,
                          int num_blocks, int max_blocks_per_seq, int dtype, void* workspace, size_t workspace_bytes,
                          void* stream) {
    if (!query_start) return PA_ERR_INVALID_ARG;
    AttendArgs a = args_of(out, q, k_cache, v_cache, block_tables, context_lens, query_start, scale, num_kv_heads,
                           num_seqs, num_q_tokens, max_q_per_seq, num_q_heads, block_size, num_blocks,
                           max_blocks_per_seq);
    const int rc = add_prefix(a, prefix_tables, prefix_lens, group_start, num_groups, max_prefix_blocks);
    return rc != PA_OK ? rc : run(a, head_dim, dtype, workspace, workspace_bytes, stream);
}

size_t pa_attend_workspace_size(int num_seqs, int num_q_tokens, int max_q_per_seq, int num_q_heads, int num_kv_heads,
                                int head_dim, int block_size, int max_blocks_per_seq, int num_groups,
                                int max_prefix_blocks) {
    if (check_shape(num_seqs, num_q_tokens, max_q_per_seq, num_q_heads, num_kv_heads, head_dim, block_size, 1,
                    max_blocks_per_seq) != PA_OK ||
        num_groups < 0 || max_prefix_blocks < 0 || num_groups > 65535 ||
        (long long)max_prefix_blocks * block_size > (1LL << 30) || num_seqs == 0 || num_q_tokens == 0)
        return 0;
    return dispatch(num_seqs, num_q_tokens, max_q_per_seq, num_q_heads, num_kv_heads, block_size, max_blocks_per_seq,
                    num_groups, max_prefix_blocks).bytes;
}

}  // extern "C"
