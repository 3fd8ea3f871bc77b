// Attention over the 16-bit paged cache with capped, biased and masked scores, or over a prefix that sequences share:
// arguments and device helpers of attend_stream.cu, attend_tc.cu and api_attend.cu.
//
// Scores: z = scale q.K_t; with a cap c > 0, z = c tanh(z / c); with slopes, z -= slope_h |p - t|.  The row at position p
// of sequence s sees the tokens t < L with first_key[row] <= t and (t <= p or t < bidirectional[s]).
#pragma once

#include "q8.cuh"

namespace pa {

// Query rows per (sequence, kv head) that attend_stream.cu takes, and of one of its segments.
constexpr int kStreamRows = 32, kSegmentRows = 16;
// Pieces of a row's keys in attend_tc.cu: of its own ones, and of the shared prefix's.
constexpr int kMostOwn = 64, kMostPrefix = 128;
constexpr int kMostSlots = kMostOwn + kMostPrefix;

struct AttendArgs {
    void* out;                   // [T][Hq][128]
    const void* q;
    const void* k_cache;         // [NB][Hkv][B][128]
    const void* v_cache;
    const int32_t* block_tables; // [S][max_blocks]
    const int32_t* context_lens; // [S]
    const int32_t* q_start;      // null: one query row per sequence
    unsigned int* status;
    float scale;
    float cap;                   // 0: none
    const float* slopes;         // [Hq], or null
    const int32_t* first_key;    // [T], or null
    const int32_t* bidirectional;// [S], or null
    int num_seqs;
    int q_rows;                  // T
    int max_q;
    int num_q_heads;
    int num_kv_heads;
    int block_size;
    int num_blocks;
    int max_blocks_per_seq;
    // a shared prefix: sequences group_start[g] .. group_start[g+1]-1 read tokens below prefix_lens[g] through
    // prefix_tables[g] (null: none)
    const int32_t* group_start;
    const int32_t* prefix_tables;
    const int32_t* prefix_lens;
    int num_groups;
    int max_prefix_blocks;
    // partial results, [slot][T * Hq]: unnormalised output rows, and (base in log2 units, sum); null: `out` is written
    float* part_o;
    float2* part_ml;
};

// Rows of one softmax joined with another's: base -inf where nothing was seen.
__device__ __forceinline__ float join_factor(float m, float to) { return m == -INFINITY ? 0.f : exp2f(m - to); }

// The group of sequence s, or -1.
__device__ __forceinline__ int group_of(const AttendArgs& a, int s) {
    int lo = 0, hi = a.num_groups;   // the last g with group_start[g] <= s
    while (lo < hi) {
        const int mid = (lo + hi + 1) / 2;
        if (mid < a.num_groups && a.group_start[mid] <= s) lo = mid;
        else hi = mid - 1;
    }
    return a.num_groups > 0 && a.group_start[lo] <= s && s < a.group_start[lo + 1] ? lo : -1;
}

// The last i of 0 .. n-1 with values[i] <= x (0: none), by a converged warp: each round of loads narrows it 32-fold.
__device__ __forceinline__ int last_not_above(const int32_t* values, int n, int x) {
    int from = 0;
    const int lane = threadIdx.x % 32;
    for (int len = n; len > 1;) {
        const int step = (len + 31) / 32, i = from + lane * step;
        const unsigned m = __ballot_sync(0xffffffffu, i < n && lane * step < len && values[i] <= x);
        const int at = m ? 31 - __clz(m) : 0;
        from += at * step;
        len = min(step, len - at * step);
    }
    return from;
}

// prefix_lens[g], kept inside the prefix's table.
__device__ __forceinline__ int prefix_len(const AttendArgs& a, int g) {
    return max(0, min(a.prefix_lens[g], a.max_prefix_blocks * a.block_size));
}

// Tokens of sequence s that its group reads together (0: none).
__device__ __forceinline__ int prefix_of(const AttendArgs& a, int s) {
    if (!a.prefix_lens) return 0;
    const int g = group_of(a, s);
    return g < 0 ? 0 : prefix_len(a, g);
}

// The new rows of sequence s with L cached tokens.
__device__ __forceinline__ NewRows rows_of(const AttendArgs& a, int s, int L) {
    return a.q_start ? new_rows(a.q_start, a.q_rows, a.max_q, s, L) : NewRows{s, 1, false};
}

// tanh(y) / y for |y| <= 3/4 as a polynomial in y^2, to 6.5e-7 (least squares weighted towards the largest error).
constexpr float kTanhReach = 0.75f;
constexpr float kTanh1 = -0.333296676f, kTanh2 = 0.132682369f, kTanh3 = -0.0502779472f, kTanh4 = 0.0131058294f;

// Weights as a high and a low bf16 part, 16 bits together.  The high part is rounded towards zero and the low one is at least
// 2^-22 of the weight, so that both are positive and a value of infinity stays one.
__device__ __forceinline__ uint32_t high_part2(float a, float b) {
    uint32_t w;
    asm("cvt.rz.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
constexpr float kLowPart = 1.f + 0x1p-22f;   // low = kLowPart * weight - high

// Which keys a launch of attend_tc.cu reads.
enum AttendKeys { kAllKeys = 0, kTailKeys = 1, kPrefixKeys = 2 };

struct TcSplits {
    int items;    // row tiles of a kv head at most
    int splits;   // pieces of an item's keys
};
// sms: the CTAs that are to run at once.
TcSplits tc_splits(long long rows_bound, int units, int num_kv_heads, long long max_keys, int most, int sms);
// slot0: where the pieces go among the partial results (splits of them); ignored when a.part_o is null.
cudaError_t launch_attend_tc(const AttendArgs& a, int dtype, AttendKeys keys, TcSplits grid, int slot0,
                             cudaStream_t stream);
// Joins partial results: slots 0 .. own-1 of every row, and for rows of sequences in a group own .. own+shared-1 too.
cudaError_t launch_attend_combine(const AttendArgs& a, int dtype, int own, int shared, cudaStream_t stream);

// Rows up to kStreamRows.  With a.part_o the results go to slot 0 of the partial results.  ctas: 0, or how many at most.
// early: the launch before this one is attend_tc.cu's of the same call, which it need not wait for.
int stream_ctas(int num_seqs, int num_kv_heads, int rows, int block_size, int max_blocks_per_seq, int most);
size_t stream_workspace_bytes(int num_seqs, int ctas, int rows);
bool stream_line_fits(int num_seqs, int num_kv_heads, int block_size, int max_blocks_per_seq);
cudaError_t launch_attend_stream(const AttendArgs& a, int dtype, int ctas, bool early, void* workspace,
                                 cudaStream_t stream);

}  // namespace pa
