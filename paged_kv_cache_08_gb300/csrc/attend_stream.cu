// Attention of few query rows (up to 32 a kv head) over the 16-bit paged cache, with capped, biased and masked scores, or
// over what follows a shared prefix.
//
// What it computes: attend.cuh, by the running-maximum softmax of "显存虚拟化革命：PagedAttention 内存池管理与显存碎片终结",
// §五.1, in log2 units: x = log2(e) z, O = sum 2^(x_t - b) V_t, l = sum 2^(x_t - b), out = O / l.  P = 2^(x - b) is
// rounded for the PV product: for fp16 values to fp16, with the base so far below the largest x that weights keep 11 bits
// down to 2^-23 of the largest, for bf16 values as a high and a low bf16 part (two products).
//
// Work split, as decode_q8.cu's: a segment is a (sequence, kv head), with more than 16 rows one for each 16 of them (their
// registers hold no more; the second reads K and V from L2); the 16-token tiles that any of its rows sees, and two
// units for its start and end, lie on a line, segment after segment, and every warp of the grid takes an equal share of
// the line.  A warp streams its tiles through a ring of its own, filled by TMA (4 KB of K, 4 KB of V, 128-byte swizzle).  A
// segment inside one share goes straight to the output; pieces of a cut one meet at the CTA's end, and where it is cut
// between CTAs in the workspace, which a second launch joins.  No atomics, no initial contents.
//
// Tile math (one warp, mma.sync m16n8k16, rows = tokens for QK and dims for PV, columns = query rows):
//   S = K Q^T: lane (g, t) = (lane / 4, lane % 4) holds dims 16 t .. 16 t + 15 of each half of tokens g and g + 8; the
//       product's k index is a permutation of the head's dims, the same one for Q.
//   O += V^T P^T: V by transposing matrix loads, P^T from S by movmatrix; the lane holds dims 8 c + g.
//
// What bounds it: HBM in long contexts and large batches (256 short chats of 32 heads 113 us, 0.87 of a copy's rate; 16
// windows of 4096 tokens, 8 kv heads of 4 rows 49 us, 0.81), and in small ones the chain before the first tile (lengths,
// line, table, copy: 4 us), the joins at the CTA's end and the joining launch (2.5 us): 64 sequences of 16 to 2048 tokens
// 14.8 us, four short contexts 8.7 us.
#include <atomic>
#include <type_traits>

#include "attend.cuh"
#include "decode_common.cuh"
#include "q8_join.h"

namespace pa {

namespace {

constexpr int kFewWarps = 8, kManyWarps = 12;       // warps of a CTA
constexpr int kTile = 16;                           // tokens per tile
constexpr uint32_t kHalf = kTile * 128;             // 64 dims of a tile's tokens
constexpr uint32_t kKBytes = 2 * kHalf;
constexpr uint32_t kTileBytes = 2 * kKBytes;
constexpr int kStartUnits = 2;                      // what a segment's start and end cost, in tiles
constexpr int kMaxSeqs = 1024;                      // sequences of one launch (their lengths stay on chip)
// log2 of P: a new base puts the largest at 2^kTopNew, and moves when one would exceed 2^kTopMost (fp16's range)
constexpr float kTopNew = 9.f, kTopMost = 15.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xffffffffu;

// Floats of a piece of `rows` rows: O, then (base, sum) of each row; a multiple of 16 bytes.
__host__ __device__ constexpr int piece_floats(int rows) { return rows * kHeadDim + (2 * rows + 3) / 4 * 4; }

// Partial results of one CTA for the joining launch.
struct CtaPieces {
    int first;      // slot 0: 0 none, 1 ends here, 2 the whole CTA is inside one segment, 3 no work
    int last;       // slot 1 holds the head of a segment that goes on in later CTAs
    int end;        // the CTA in which it ends
    int row0, rows; // its query rows
    int head;       // its kv head
    int pad[2];
};

struct StreamLaunch {
    AttendArgs a;
    float* parts;         // [grid][2] pieces of `rows` rows
    float* firsts;        // [grid * warps] pieces
    CtaPieces* pieces;    // [grid]
    int rows;             // query rows of a segment at most
    int row_parts;        // 1, or more than kSegmentRows rows: a kv head's segments of as many each (below)
    bool early;           // the grid before this one is waited for at the end
    int block_log2;
    int group;            // query heads per kv head
    unsigned group_inv;   // ceil(2^16 / group)
    int seq0;             // the batch's sequence that is this launch's first
};

template <int NT, int kW>
struct Smem {
    static constexpr int kRows = NT * 8, kWarps = kW, kThreads = kWarps * 32;
    static constexpr int kStages = kW > kFewWarps ? 2 : 3;   // tiles of a warp's ring
    static constexpr uint32_t kRing = kStages * kTileBytes;
    static constexpr uint32_t kOffLastMl = kWarps * kRing;
    static constexpr uint32_t kOffDesc = kOffLastMl + kWarps * kRows * 8;
    static constexpr uint32_t kOffBar = kOffDesc + kWarps * 16;
    static constexpr uint32_t kOffP = kOffBar + kWarps * kStages * 8;
    static constexpr uint32_t kOffLen = kOffP + (kMaxSeqs + 2) * 8;
    static constexpr uint32_t kOffTile0 = kOffLen + kMaxSeqs * 4;
    static constexpr uint32_t kOffRow0 = kOffTile0 + kMaxSeqs * 4;
    static constexpr uint32_t kOffN = kOffRow0 + kMaxSeqs * 4;
    static constexpr uint32_t kBytes = kOffN + kMaxSeqs;
    static_assert(kRing >= kRows * kHeadDim * 4, "a warp's last piece is kept in its ring");
    static constexpr uint32_t kStatic = kWarps * 8;   // declared in the kernel
    static_assert(1024 + kBytes + kStatic <= 227 * 1024, "shared memory of one CTA");
};

// What a warp leaves for the end of its CTA (flags as in q8_join.h, then segments as s << 16 | h).
struct WarpPieces {
    int flags, first_seg, last_seg, pad;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ uint16_t lds16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr));
    return v;
}

// Halves of w whose exponent is all ones, as 0x8000 each.
template <typename T>
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
    constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    return ((w & kExp) + kOne) & 0x80008000u;
}

// (m, l, acc) of one row joined with a piece.
__device__ __forceinline__ void add_piece(float& m, float& l, float4& acc, float2 ml, float4 v) {
    const float m2 = fmaxf(m, ml.x);
    const float f0 = join_factor(m, m2), f1 = join_factor(ml.x, m2);
    m = m2;
    l = l * f0 + ml.y * f1;
    acc.x = acc.x * f0 + v.x * f1;
    acc.y = acc.y * f0 + v.y * f1;
    acc.z = acc.z * f0 + v.z * f1;
    acc.w = acc.w * f0 + v.w * f1;
}

// Four elements of row `row` of [T * Hq]: finished, or among the partial results.  A row that saw no token is zero.
template <typename T>
__device__ __forceinline__ void emit4(const AttendArgs& a, size_t row, int lane, float m, float l, const float4& acc) {
    if (a.part_o) {
        *reinterpret_cast<float4*>(a.part_o + row * kHeadDim + lane * 4) = acc;
        if (lane == 0) a.part_ml[row] = make_float2(m, l);
        return;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2 w;
    w.x = Elem<T>::pack2(acc.x * inv, acc.y * inv);
    w.y = Elem<T>::pack2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.out) + row * kHeadDim + lane * 4) = w;
}

// Query token of row r of a kv head's, r / group for r < 32, by the multiplier that p.group_inv holds.
__device__ __forceinline__ int token_of(const StreamLaunch& p, int r) { return (int)((unsigned)r * p.group_inv >> 16); }

// The segments of a sequence with n query tokens: every kv head with the first kSegmentRows rows, then (more than 16 rows)
// every kv head with the next.  Segment h's kv head, first row and number of rows:
__device__ __forceinline__ int segments(const StreamLaunch& p, int n) {
    return p.row_parts == 1 ? p.a.num_kv_heads : p.a.num_kv_heads * ((n * p.group + kSegmentRows - 1) / kSegmentRows);
}
__device__ __forceinline__ int head_of(const StreamLaunch& p, int h) {
    return p.row_parts == 1 ? h : h % p.a.num_kv_heads;
}
__device__ __forceinline__ int first_row(const StreamLaunch& p, int h) {
    return p.row_parts == 1 ? 0 : h / p.a.num_kv_heads * kSegmentRows;
}
__device__ __forceinline__ int num_rows(const StreamLaunch& p, int h, int n) {
    return min(kSegmentRows, n * p.group - first_row(p, h));
}

// Query row r of segment h (token r / group, group member r % group of its kv head's rows) as a row of [T * Hq].
__device__ __forceinline__ size_t row_at(const StreamLaunch& p, int row0, int h, int r) {
    r += first_row(p, h);
    const int i = token_of(p, r);
    return (size_t)(row0 + i) * p.a.num_q_heads + (size_t)head_of(p, h) * p.group + r - i * p.group;
}

// In a piece, the dims of row r lie at d ^ 8 (r / 2 % 4): the lanes that store a fragment (four row pairs at once) then
// meet no bank conflict.  `at` for one dim, `chunk_at` for 16-byte chunk c.
__device__ __forceinline__ int at(int r, int d) { return r * kHeadDim + (d ^ (r >> 1 & 3) * 8); }
__device__ __forceinline__ int chunk_at(int r, int c) { return r * (kHeadDim / 4) + (c ^ (r >> 1 & 3) * 2); }

template <typename T, int NT, int kW, bool kMulti, bool kScored>
__global__ void __launch_bounds__(Smem<NT, kW>::kThreads, 1)
    stream_kernel(const StreamLaunch p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using M = Smem<NT, kW>;
    constexpr int kWarps = M::kWarps, kThreads = M::kThreads, kStages = M::kStages;
    constexpr uint32_t kRing = M::kRing;
    constexpr bool kSplitP = std::is_same<T, __nv_bfloat16>::value;
    const AttendArgs& a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, t = lane % 4;
    long long* P = reinterpret_cast<long long*>(smem + M::kOffP);
    int* lens = reinterpret_cast<int*>(smem + M::kOffLen);
    int* tile0_of = reinterpret_cast<int*>(smem + M::kOffTile0);
    int* row0_of = reinterpret_cast<int*>(smem + M::kOffRow0);
    uint8_t* n_of = smem + M::kOffN;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kOffBar) + warp * kStages;
    WarpPieces* wp = reinterpret_cast<WarpPieces*>(smem + M::kOffDesc);
    const uint32_t ring = smem_u32(smem) + warp * kRing;

    if (lane < kStages) {
        mbar_init(&bars[lane], 1);
        fence_mbar_init();
    }
    if (tid == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    if (!p.early) grid_dependency_wait();
    grid_launch_dependents();

    // ---- lengths, the first tile that a row sees, and the units before each sequence (P) ----
    const int S = a.num_seqs, group = p.group;
    auto units_of = [&](int s) { return (lens[s] + kTile - 1) / kTile - tile0_of[s] + kStartUnits; };   // of one segment
    auto segs_of = [&](int s) { return segments(p, n_of[s]); };
    {
        __shared__ long long warp_sum_of[kWarps];
        static_assert(sizeof(warp_sum_of) == M::kStatic, "as Smem counts it");
        long long carry = 0;
        for (int s0 = 0; s0 < S; s0 += kThreads) {
            const int s = s0 + tid;
            long long w = 0;
            if (s < S) {
                // (loads that do not wait for one another: the first key's, with one query token, is a row's own)
                int lo = !kMulti && a.first_key ? a.first_key[s] : a.prefix_lens ? prefix_of(a, p.seq0 + s) : 0;
                bool bad;
                const int L = clamped_len(a.context_lens, s, a.max_blocks_per_seq, a.block_size, &bad);
                int n = 1, row0 = s;
                if (kMulti) {
                    const NewRows nr = new_rows(a.q_start, a.q_rows, a.max_q, s, L);
                    n = nr.n;
                    row0 = nr.row0;
                    bad |= nr.bad;
                    if (a.first_key && n > 0) {
                        lo = a.first_key[row0];
                        for (int i = 1; i < n; ++i) lo = min(lo, a.first_key[row0 + i]);
                    }
                }
                if (bad && blockIdx.x == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
                lo = max(0, lo);
                lens[s] = L;
                row0_of[s] = row0;
                n_of[s] = (uint8_t)n;
                tile0_of[s] = lo / kTile;
                if (lo < L && n > 0) w = (long long)((L + kTile - 1) / kTile - lo / kTile + kStartUnits) * segments(p, n);
            }
            long long incl = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long v = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += v;
            }
            if (s0 > 0) __syncthreads();   // warp_sum_of of the round before has been read
            if (lane == 31) warp_sum_of[warp] = incl;
            __syncthreads();
            long long before = carry + incl - w;
#pragma unroll
            for (int i = 0; i < kWarps; ++i) {
                const long long x = warp_sum_of[i];
                if (i < warp) before += x;
                carry += x;
            }
            if (s < S) P[s] = before;
        }
        if (tid == 0) P[S] = carry;
        __syncthreads();
    }

    const long long total = P[S];
    // share i of the line begins at unit floor(total * i / shares) (32-bit divisions: 64-bit ones take 0.3 us each)
    const unsigned shares = gridDim.x * kWarps, me = blockIdx.x * kWarps + warp;
    const long long each = total >> 32 ? total / shares : (long long)((unsigned)total / shares);
    const unsigned odd = (unsigned)(total - each * shares);
    auto share_at = [&](unsigned i) { return each * i + (odd * i) / shares; };
    // A cut among a segment's start units goes before them; in a short segment one next to its first or last tile goes to
    // the begin or the end, too, since the piece costs more than the tile.
    auto near_of = [&](int w) { return (NT > 1 || gridDim.x == 1) && w <= kStartUnits + 8 ? 1 : 0; };
    // The share's first unit (r of segment (s, h)) and, by the upper half of the warp, the next share's.
    int s, h, r, units;
    long long u0;
    {
        const int half = lane & 16, of_half = lane & 15;
        long long u = share_at(me + (half >> 4));
        s = 0;   // the last s with P[s] <= u
        for (int n = S; n > 1;) {
            n = (n + 15) / 16;
            const int i = s + of_half * n;
            const unsigned m = __ballot_sync(kAll, i < S && P[min(i, S)] <= u) >> half & 0xffff;
            s += (31 - __clz(m)) * n;
        }
        const int w = max(1, units_of(s));
        const unsigned long long rem = u - P[s];
        h = rem <= 0xffffffffu ? (uint32_t)rem / w : (int)(rem / w);
        r = (int)(rem - (unsigned long long)h * w);
        if (u < total) {
            const int near = near_of(w);
            if (r <= kStartUnits + near) {
                u -= r;
                r = 0;
            } else if (w - r <= near) {
                u += w - r;
                r = 0;
                if (++h == segs_of(s)) {
                    h = 0;
                    do ++s;
                    while (s < S && P[s + 1] == P[s]);
                }
            }
        }
        u0 = __shfl_sync(kAll, u, 0);
        units = (int)(__shfl_sync(kAll, u, 16) - u0);
        s = __shfl_sync(kAll, s, 0);
        h = __shfl_sync(kAll, h, 0);
        r = __shfl_sync(kAll, r, 0);
    }

    // ---- per-lane fragment addresses inside a tile (128-byte swizzle: 16-byte unit ^ (row & 7)) ----
    const uint32_t k_off0 = g * 128 + ((uint32_t)((2 * t) ^ g) << 4);
    const uint32_t k_off1 = g * 128 + ((uint32_t)((2 * t + 1) ^ g) << 4);
    const uint32_t v_tok = (lane & 7) + (lane >> 4) * 8;   // matrices: tokens 0-7 of two chunks, then tokens 8-15
    const uint32_t v_row = kKBytes + v_tok * 128, v_chunk = lane >> 3 & 1;

    float o[NT][8][4];
    float base[NT][2], sum[NT][2];
    // of this lane's score columns (rows 2 t and 2 t + 1 of each 8): the positions the row sees, its own, its slope
    int lim_lo[NT][2], lim_hi[NT][2];
    float slope[NT][2];
    int pos[NT][2];
    uint32_t qreg[NT][16];
    uint4 qn[NT][4];                     // Q rows of the segment that comes next
    int L = 0, row0 = 0, nrows = 0;
    int all_lo = 0, all_hi = 0;          // positions that every row sees: all_lo .. all_hi
    uint32_t phases = 0;
    const float xs = kScored && a.cap > 0.f ? a.cap * kLog2e : a.scale * kLog2e;
    const float ks = kScored && a.cap > 0.f ? a.scale / a.cap : 0.f;

    // Loads of Q row 8 nt + g, dims 16 t .. 16 t + 15 of each half, of segment (s, h), ahead of its begin.
    auto fetch_q = [&](int s, int h) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int rows = num_rows(p, h, n_of[s]), r = nt * 8 + g;
            const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                              row_at(p, row0_of[s], h, r < rows ? r : 0) * kHeadDim);
#pragma unroll
            for (int i = 0; i < 4; ++i)
                qn[nt][i] = r < rows ? __ldg(src + (i >> 1) * 8 + 2 * t + (i & 1)) : make_uint4(0, 0, 0, 0);
        }
    };

    auto begin_segment = [&]() {
        L = lens[s];
        row0 = row0_of[s];
        const int n = n_of[s];
        nrows = num_rows(p, h, n);
        all_lo = 0;
        all_hi = L - 1;
        const int until = a.bidirectional ? min(a.bidirectional[s], L) : 0;
        const int from = a.prefix_lens ? prefix_of(a, p.seq0 + s) : 0;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                qreg[nt][4 * i] = qn[nt][i].x;
                qreg[nt][4 * i + 1] = qn[nt][i].y;
                qreg[nt][4 * i + 2] = qn[nt][i].z;
                qreg[nt][4 * i + 3] = qn[nt][i].w;
            }
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = nt * 8 + 2 * t + c;
                lim_lo[nt][c] = 0;
                lim_hi[nt][c] = L - 1;
                pos[nt][c] = 0;
                slope[nt][c] = 0.f;
                if (col < nrows) {
                    const int row = first_row(p, h) + col, i = token_of(p, row), at = L - n + i;
                    lim_lo[nt][c] = a.first_key ? max(0, a.first_key[row0 + i]) : from;
                    lim_hi[nt][c] = max(at, until - 1);
                    pos[nt][c] = at;
                    if (kScored && a.slopes) slope[nt][c] = a.slopes[head_of(p, h) * group + row - i * group] * kLog2e;
                    all_lo = max(all_lo, lim_lo[nt][c]);
                    all_hi = min(all_hi, lim_hi[nt][c]);
                }
                base[nt][c] = -INFINITY;
                sum[nt][c] = 0.f;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
        }
#pragma unroll
        for (int k = 1; k < 4; k <<= 1) {
            all_lo = max(all_lo, __shfl_xor_sync(kAll, all_lo, k));
            all_hi = min(all_hi, __shfl_xor_sync(kAll, all_hi, k));
        }
    };
    auto sees = [&](int nt, int c, int tok) { return tok >= lim_lo[nt][c] && tok <= lim_hi[nt][c]; };

    // One tile of tokens t0 .. t0 + 15.
    auto run_tile = [&](uint32_t tile, int t0) {
        // S = K Q^T
        float x[NT][4], y[4] = {0.f, 0.f, 0.f, 0.f};   // one tile of rows: odd steps on their own, for two short chains
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[nt][c] = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {   // (half, chunk)
            const uint32_t off = tile + (i >> 1) * kHalf + (i & 1 ? k_off1 : k_off0);
            const uint4 ka = lds128(off), kb = lds128(off + 1024);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                mma16816<T>(x[nt], ka.x, kb.x, ka.y, kb.y, qreg[nt][4 * i], qreg[nt][4 * i + 1]);
                mma16816<T>(NT == 1 ? y : x[nt], ka.z, kb.z, ka.w, kb.w, qreg[nt][4 * i + 2], qreg[nt][4 * i + 3]);
            }
        }
        if (NT == 1) {
#pragma unroll
            for (int c = 0; c < 4; ++c) x[0][c] += y[c];
        }
        // V^T: of dims 16 i .. 16 i + 15, tokens 2t, 2t+1 (0, 1) and 2t+8, 2t+9 (2, 3)
        uint32_t v[8][4];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t chunk = (2 * i + v_chunk) & 7;
            ldsm_x4_t(tile + v_row + (i >> 2) * kHalf + ((chunk ^ (v_tok & 7)) << 4), v[i][0], v[i][1], v[i][2], v[i][3]);
        }

        // scores in log2 units
        if (kScored && a.cap > 0.f) {
            bool far = false;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    x[nt][c] *= ks;
                    far |= !(fabsf(x[nt][c]) <= kTanhReach);
                }
            far = __any_sync(kAll, far);
            // (a score's own size chooses its form; the vote spares the exponentials where no lane wants one)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const float z = x[nt][c], z2 = z * z;
                    x[nt][c] = fmaf(fmaf(fmaf(fmaf(kTanh4, z2, kTanh3), z2, kTanh2), z2, kTanh1), z2 * z, z);
                    if (far && !(fabsf(z) <= kTanhReach)) x[nt][c] = 1.f - __fdividef(2.f, 1.f + ex2(z * (2.f * kLog2e)));
                }
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[nt][c] *= xs;
                if (kScored && a.slopes)
                    x[nt][c] = fmaf(-slope[nt][c & 1], fabsf((float)(t0 + g + (c >> 1) * 8 - pos[nt][c & 1])), x[nt][c]);
            }
        const bool masked = t0 < all_lo || t0 + kTile - 1 > all_hi;
        bool wrong = false;
        if (masked) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (!sees(nt, c & 1, t0 + g + (c >> 1) * 8)) x[nt][c] = -INFINITY;
            // a weight of zero meets no value that is not finite: rows behind the last token hold anything, and with one
            // query token a row that is masked is masked for all
            const int first = kMulti ? 0 : all_lo, last = kMulti ? L - 1 : all_hi;
            auto keep = [&](int tok) { return tok >= first && tok <= last ? 0xffffu : 0u; };
            const uint32_t k01 = keep(t0 + 2 * t) | keep(t0 + 2 * t + 1) << 16,
                           k23 = keep(t0 + 2 * t + 8) | keep(t0 + 2 * t + 9) << 16;
            uint32_t bad = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[i][e] &= e < 2 ? k01 : k23;
                    if (kMulti) bad |= non_finite<T>(v[i][e]);
                }
            if (kMulti) {
                wrong = __any_sync(kAll, bad != 0);
                if (wrong) {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
#pragma unroll
                        for (int e = 0; e < 4; ++e) v[i][e] &= ~((non_finite<T>(v[i][e]) >> 15) * 0xffffu);
                }
            }
        }
        bool move = false;   // a column without a base yet (-inf) takes one as soon as it sees a token
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) move |= fmaxf(x[nt][c], x[nt][c + 2]) - base[nt][c] > kTopMost;
        if (__any_sync(kAll, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float m = fmaxf(x[nt][c], x[nt][c + 2]);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, k));
                    // (a column's own scores alone decide: another row may see tokens that this one does not)
                    m = m - base[nt][c] > kTopMost ? __fadd_ru(m, -kTopNew) : base[nt][c];
                    const float f = join_factor(base[nt][c], m);
                    base[nt][c] = m;
                    sum[nt][c] *= f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        o[nt][k][c] *= f;
                        o[nt][k][c + 2] *= f;
                    }
                }
        }
        uint32_t b0[NT], b1[NT], l0[kSplitP ? NT : 1], l1[kSplitP ? NT : 1];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float pr[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)   // (0 for what a row without a base yet has: masked scores and ones below fp32's range)
                pr[c] = ex2(x[nt][c] - (base[nt][c & 1] == -INFINITY ? 0.f : base[nt][c & 1]));
            sum[nt][0] += pr[0] + pr[2];
            sum[nt][1] += pr[1] + pr[3];
            const uint32_t h0 = kSplitP ? high_part2(pr[0], pr[1]) : Elem<T>::pack2(pr[0], pr[1]),
                           h1 = kSplitP ? high_part2(pr[2], pr[3]) : Elem<T>::pack2(pr[2], pr[3]);
            b0[nt] = movmatrix_trans(h0);
            b1[nt] = movmatrix_trans(h1);
            if (kSplitP) {
                const float2 f0 = Elem<T>::to_float2(h0), f1 = Elem<T>::to_float2(h1);
                l0[kSplitP ? nt : 0] = movmatrix_trans(Elem<T>::pack2(fmaf(pr[0], kLowPart, -f0.x), fmaf(pr[1], kLowPart, -f0.y)));
                l1[kSplitP ? nt : 0] = movmatrix_trans(Elem<T>::pack2(fmaf(pr[2], kLowPart, -f1.x), fmaf(pr[3], kLowPart, -f1.y)));
            }
        }
        // O += V^T P^T
#pragma unroll
        for (int i = 0; i < 8; ++i)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<T>(o[nt][i], v[i][0], v[i][1], v[i][2], v[i][3], b0[nt], b1[nt]);
        if (kSplitP) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    mma16816<T>(o[nt][i], v[i][0], v[i][1], v[i][2], v[i][3], l0[kSplitP ? nt : 0], l1[kSplitP ? nt : 0]);
        }
        if (kMulti && wrong) {
            // rare: what is not finite into the dims and rows that see such a token
            for (int j = 0; j < min(kTile, L - t0); ++j) {
#pragma unroll
                for (int c = 0; c < 16; ++c) {   // dim 8 c + g
                    const uint16_t w = lds16(tile + kKBytes + (c >> 3) * kHalf + j * 128 + ((uint32_t)((c & 7) ^ (j & 7)) << 4) + g * 2);
                    if (non_finite<T>(w)) {
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                            for (int e = 0; e < 2; ++e)
                                if (sees(nt, e, t0 + j)) o[nt][c >> 1][(c & 1) * 2 + e] += Elem<T>::to_float(w);
                    }
                }
            }
        }
    };

    // Sum over the lanes that share a column.
    auto finish_sums = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int m = 4; m < 32; m <<= 1) sum[nt][c] += __shfl_xor_sync(kAll, sum[nt][c], m);
            }
    };

    auto store_piece = [&](float* slot, float2* ml) {
        finish_sums();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = nt * 8 + 2 * t + c;
                if (r < nrows) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        slot[at(r, 16 * i + g)] = o[nt][i][c];
                        slot[at(r, 16 * i + 8 + g)] = o[nt][i][c + 2];
                    }
                    if (g == 0) ml[r] = make_float2(base[nt][c], sum[nt][c]);
                }
            }
    };

    auto store_out = [&](int h) {
        finish_sums();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if (a.part_o) {
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    const int r = nt * 8 + 2 * t + c;
                    if (r < nrows) {
                        const size_t row = row_at(p, row0, h, r);
                        float* to = a.part_o + row * kHeadDim + g;
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            to[16 * i] = o[nt][i][c];
                            to[16 * i + 8] = o[nt][i][c + 2];
                        }
                        if (g == 0) a.part_ml[row] = make_float2(base[nt][c], sum[nt][c]);
                    }
                }
            } else {
                // a chunk's 8 dims x 8 rows transposed: the lane then has dims 8 c + 2 t, + 1 of row g
                const float i0 = sum[nt][0] == 0.f ? 0.f : 1.f / sum[nt][0], i1 = sum[nt][1] == 0.f ? 0.f : 1.f / sum[nt][1];
                const int r = nt * 8 + g;
                uint32_t* to = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(a.out) +
                                                           row_at(p, row0, h, r < nrows ? r : 0) * kHeadDim) + t;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t w0 = movmatrix_trans(Elem<T>::pack2(o[nt][i][0] * i0, o[nt][i][1] * i1));
                    const uint32_t w1 = movmatrix_trans(Elem<T>::pack2(o[nt][i][2] * i0, o[nt][i][3] * i1));
                    if (r < nrows) {
                        to[8 * i] = w0;
                        to[8 * i + 4] = w1;
                    }
                }
            }
        }
    };

    // pieces of warp w: the first in memory, the last in its ring (every copy has landed)
    auto first_of = [&](int w) { return p.firsts + ((size_t)blockIdx.x * kWarps + w) * piece_floats(p.rows); };
    auto last_of = [&](int w) { return reinterpret_cast<float*>(smem + w * kRing); };
    auto first_ml_of = [&](int w) { return reinterpret_cast<float2*>(first_of(w) + p.rows * kHeadDim); };
    auto last_ml_of = [&](int w) { return reinterpret_cast<float2*>(smem + M::kOffLastMl) + w * M::kRows; };

    // ---- the stream ----
    WarpPieces mine{units == 0 ? kNoUnits : 0, 0, 0, 0};
    if (units > 0) {
        // of the unit this lane owns in a window of 32: the pool row of its tile's first token (-1: a start
        // unit or none, -2: a block outside the pool)
        int A_y = -1, B_y = -1, lane_s = s;
        auto look = [&](int i, int& y) {   // unit u0 + i; i grows from call to call
            y = -1;
            if (i >= units) return;
            const long long u = u0 + i;
            while (P[lane_s + 1] <= u) ++lane_s;
            const uint32_t w = units_of(lane_s);
            const unsigned long long rem = u - P[lane_s];
            const int hh = rem <= 0xffffffffu ? (uint32_t)rem / w : (int)(rem / w);
            const int r = (int)(rem - (unsigned long long)hh * w);
            if (r < kStartUnits) return;
            const int t0 = (tile0_of[lane_s] + r - kStartUnits) * kTile;
            const int id = __ldg(a.block_tables + (size_t)lane_s * a.max_blocks_per_seq + (t0 >> p.block_log2));
            if (id < 0 || id >= a.num_blocks) {
                flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
                y = -2;
                return;
            }
            y = ((id * a.num_kv_heads + head_of(p, hh)) << p.block_log2) + (t0 & (a.block_size - 1));   // fits: num_blocks * num_kv_heads * B < 2^31
        };
        fetch_q(s, h);
        look(lane, A_y);
        auto issue = [&](int j, int y) {   // by the lane that owns unit j
            const int st = j % kStages;
            const uint32_t dst = ring + st * kTileBytes;
            mbar_arrive_expect_tx(&bars[st], kTileBytes);
            tma_load_2d(dst, &kmap, 0, y, &bars[st]);
            tma_load_2d(dst + kHalf, &kmap, 64, y, &bars[st]);
            tma_load_2d(dst + kKBytes, &vmap, 0, y, &bars[st]);
            tma_load_2d(dst + kKBytes + kHalf, &vmap, 64, y, &bars[st]);
        };
        if (lane < kStages && A_y >= 0) issue(lane, A_y);
        bool dead = false;
        int i = 0;
        while (i < units) {
            // segment (s, h) from its unit r on
            const int left = units_of(s) - r, stop = min(units, i + left);
            const bool from_before = r > 0, ends = i + left <= units;
            begin_segment();
            const int this_s = s, this_h = h, tile0 = tile0_of[s];
            int next_s = s, next_h = h + 1;
            if (i + left < units) {
                if (next_h == segs_of(s)) {
                    next_h = 0;
                    do ++next_s;
                    while (P[next_s + 1] == P[next_s]);
                }
                fetch_q(next_s, next_h);
            }
            for (; i < stop; ++i, ++r) {
                const int w = i & 31;
                if (w == 0) {
                    if (i > 0) A_y = B_y;
                    if (i + 32 < units) look(i + 32 + lane, B_y);
                }
                const int y = __shfl_sync(kAll, A_y, w);
                if (y >= 0) {
                    const int st = i % kStages;
                    if (!mbar_wait_bounded(&bars[st], (phases >> st) & 1)) {
                        flag_status(a.status, PA_DEV_TIMEOUT);
                        dead = true;
                    }
                    dead = __any_sync(kAll, dead);
                    if (dead) break;
                    phases ^= 1u << st;
                    run_tile(ring + st * kTileBytes, (tile0 + r - kStartUnits) * kTile);
                }
                // every lane has the tile in registers: its stage takes the unit kStages further on
                __syncwarp();
                const int j = i + kStages;
                if (j < units && lane == (j & 31)) {
                    const int yj = (j >> 5) == (i >> 5) ? A_y : B_y;
                    if (yj >= 0) issue(j, yj);
                }
            }
            if (dead) break;
            if (!ends) {
                store_piece(last_of(warp), last_ml_of(warp));
                mine.flags |= kHasLast | (from_before ? kThrough : 0);
                mine.last_seg = this_s << 16 | this_h;
            } else if (from_before) {
                store_piece(first_of(warp), first_ml_of(warp));
                mine.flags |= kHasFirst;
                mine.first_seg = this_s << 16 | this_h;
            } else {
                store_out(this_h);
            }
            s = next_s;
            h = next_h;
            r = 0;
        }
        if (dead) {   // let the copies in flight land (again with a limit) before the CTA's memory is given up
            mine.flags = kGaveUp;
            for (int j = i; j < min(units, i + kStages); ++j) {
                const int yj = __shfl_sync(kAll, (j >> 5) == (i >> 5) ? A_y : B_y, j & 31);
                if (yj >= 0) mbar_wait_bounded(&bars[j % kStages], (phases >> (j % kStages)) & 1);
            }
        }
    }
    if (lane == 0) wp[warp] = mine;
    __syncthreads();

    // ---- join the pieces of cut segments ----
    // Of a chain of pieces (q8_join.h) ws .. we, warp we gives its first piece if the chain ends there, every other
    // warp its last.  The rows of all chains are dealt to the warps, four at a time.
    int left_first, left_last, left_seg = 0;
    {
        constexpr int kGroup = kWarps <= 8 ? 8 : 16, kTake = 32 / kGroup;   // lanes a row, rows at a time
        const WarpPieces x = lane < kWarps ? wp[lane] : WarpPieces{kNoUnits, 0, 0, 0};
        const CtaJoin join = cta_join(__ballot_sync(kAll, x.flags & kNoUnits), __ballot_sync(kAll, x.flags & kHasFirst),
                                      __ballot_sync(kAll, x.flags & kHasLast), __ballot_sync(kAll, x.flags & kThrough),
                                      __ballot_sync(kAll, x.flags & kGaveUp), kWarps);
        const unsigned some = join.some, events = join.events;
        const int last_warp = join.last_warp;
        left_first = join.left_first;
        left_last = join.left_last;
        if (left_last) left_seg = __shfl_sync(kAll, x.last_seg, last_warp);
        const int batches = (p.rows + kTake - 1) / kTake, items = __popc(events) * batches;
        for (int item = warp; item < items; item += kWarps) {
            unsigned ev = events;
            int k = item;
            for (; k >= batches; k -= batches) ev &= ev - 1;
            const JoinChain chain = join.chain(ev);
            const int ws = chain.from, we = chain.to;
            const bool closed = we < kWarps, before = chain.before;
            const unsigned pieces = some & ~((1u << ws) - 1) & ((2u << we) - 1);
            const int seg = __shfl_sync(kAll, closed ? x.first_seg : x.last_seg, closed ? we : last_warp);
            const int sg = seg >> 16, hh = seg & 0xffff, r0 = k * kTake;
            const int first = row0_of[sg], rows = num_rows(p, hh, n_of[sg]);
            if (r0 >= rows) continue;
            float* to = p.parts + ((size_t)blockIdx.x * 2 + (before ? 0 : 1)) * piece_floats(p.rows);
            // kTake rows at a time: lane kGroup i + w weighs warp w's piece of row i, then every lane has four elements of
            // each row
            const int w = lane % kGroup, rw = r0 + lane / kGroup;
            float4 vf[kTake];   // the piece that ends the chain, on its way early
#pragma unroll
            for (int i = 0; i < kTake; ++i)
                if (closed && r0 + i < rows) vf[i] = reinterpret_cast<const float4*>(first_of(we))[chunk_at(r0 + i, lane)];
            float2 ml = make_float2(-INFINITY, 0.f);
            if ((pieces >> w & 1) && rw < rows) ml = (closed && w == we ? first_ml_of(w) : last_ml_of(w))[rw];
            float m = ml.x;
#pragma unroll
            for (int k = 1; k < kGroup; k <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, k));
            const float f = join_factor(ml.x, m);
            float l = f * ml.y;
#pragma unroll
            for (int k = 1; k < kGroup; k <<= 1) l += __shfl_xor_sync(kAll, l, k);
            float4 acc[kTake];
#pragma unroll
            for (int i = 0; i < kTake; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int last_end = closed ? we : last_warp + 1;
#pragma unroll 1
            for (int pw = ws; pw < last_end; ++pw) {   // last pieces
                if (!(pieces >> pw & 1)) continue;
#pragma unroll
                for (int i = 0; i < kTake; ++i) {
                    const float fw = __shfl_sync(kAll, f, i * kGroup + pw);
                    if (r0 + i < rows) {
                        const float4 x = reinterpret_cast<const float4*>(last_of(pw))[chunk_at(r0 + i, lane)];
                        acc[i].x = fmaf(fw, x.x, acc[i].x);
                        acc[i].y = fmaf(fw, x.y, acc[i].y);
                        acc[i].z = fmaf(fw, x.z, acc[i].z);
                        acc[i].w = fmaf(fw, x.w, acc[i].w);
                    }
                }
            }
            if (closed)
#pragma unroll
                for (int i = 0; i < kTake; ++i) {
                    const float fw = __shfl_sync(kAll, f, i * kGroup + we);
                    if (r0 + i < rows) {
                        acc[i].x = fmaf(fw, vf[i].x, acc[i].x);
                        acc[i].y = fmaf(fw, vf[i].y, acc[i].y);
                        acc[i].z = fmaf(fw, vf[i].z, acc[i].z);
                        acc[i].w = fmaf(fw, vf[i].w, acc[i].w);
                    }
                }
#pragma unroll
            for (int i = 0; i < kTake; ++i) {
                const float mi = __shfl_sync(kAll, m, i * kGroup), li = __shfl_sync(kAll, l, i * kGroup);
                const int r = r0 + i;
                if (r < rows) {
                    if (closed && !before) {
                        emit4<T>(a, row_at(p, first, hh, r), lane, mi, li, acc[i]);
                    } else {
                        *reinterpret_cast<float4*>(to + r * kHeadDim + lane * 4) = acc[i];
                        if (lane == 0) reinterpret_cast<float2*>(to + p.rows * kHeadDim)[r] = make_float2(mi, li);
                    }
                }
            }
        }
    }
    if (tid == 0 && gridDim.x > 1) {
        CtaPieces left{left_first, left_last, 0, 0, 0, 0, {0, 0}};
        if (left_last) {
            const int sg = left_seg >> 16, hh = left_seg & 0xffff;
            // the share that holds its last unit: a guess good to a share or two, put right
            const int w = units_of(sg);
            const long long last_unit = P[sg] + (long long)(hh + 1) * w - 1;
            int i = max(0, min((int)((float)last_unit * (float)shares / (float)total), (int)shares - 1));
            while (share_at(i) > last_unit) --i;
            while (share_at(i + 1) <= last_unit) ++i;
            const int near = near_of(w);   // (cuts moved to the segment's end)
            while (last_unit + 1 - share_at(i) <= near && w - (last_unit + 1 - share_at(i)) > kStartUnits + near) --i;
            left.end = i / kWarps;
            left.row0 = row0_of[sg];
            left.rows = num_rows(p, hh, n_of[sg]);
            left.head = hh;
        }
        p.pieces[blockIdx.x] = left;
    }
    // rows of sequences of which no token is seen
    for (int e = blockIdx.x; e < S; e += gridDim.x)
        if (P[e + 1] == P[e])
            for (int i = warp; i < n_of[e] * a.num_q_heads; i += kWarps)
                emit4<T>(a, (size_t)row0_of[e] * a.num_q_heads + i, lane, -INFINITY, 0.f, make_float4(0.f, 0.f, 0.f, 0.f));
    if (p.early) grid_dependency_wait();   // so that whatever waits for this grid also waits for the one before
}

// Joins the segments cut between CTAs: CTA (c, .) takes the segment whose head is CTA c's last piece; the
// pieces that follow are the first ones of the next CTAs, up to the one that ends it.  A row goes to `split`
// warps (1, 2, 4 or 8), which share its pieces.
constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32, 5) stream_join_kernel(const StreamLaunch p, int ctas, int split) {
    __shared__ float4 acc_of[kJoinWarps][32];
    __shared__ float2 ml_of[kJoinWarps];
    const int c = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int part = warp & (split - 1), r = (blockIdx.y * kJoinWarps + warp) / split;
    grid_dependency_wait();
    grid_launch_dependents();
    constexpr int kBatch = 4;
    float2 ml[kBatch];
    float4 v[kBatch];
    int some[kBatch];
    auto load = [&](int i0, int end) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = min(i0 + k * split, end);
            const float* piece = p.parts + ((size_t)i * 2 + (i == c ? 1 : 0)) * piece_floats(p.rows);
            some[k] = p.pieces[i].first;
            ml[k] = reinterpret_cast<const float2*>(piece + p.rows * kHeadDim)[r];
            v[k] = *reinterpret_cast<const float4*>(piece + r * kHeadDim + lane * 4);
        }
    };
    // the first pieces are read before it is known whether they are the segment's: one round trip less
    if (r < p.rows) load(c + part, ctas - 1);
    const CtaPieces head = p.pieces[c];
    if (!head.last) return;
    const int end = min(head.end, ctas - 1);
    const bool have = r < head.rows;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    if (have)
        for (int i0 = c + part; i0 <= end; i0 += split * kBatch) {
            if (i0 != c + part) load(i0, end);
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int i = i0 + k * split;
                if (i <= end && (i == c || some[k] != 3)) add_piece(m, l, acc, ml[k], v[k]);
            }
        }
    if (split > 1) {
        acc_of[warp][lane] = acc;
        if (lane == 0) ml_of[warp] = make_float2(m, l);
        __syncthreads();
        if (part > 0) return;
        for (int w = 1; w < split; ++w) add_piece(m, l, acc, ml_of[warp + w], acc_of[warp + w][lane]);
    }
    if (have) emit4<T>(p.a, row_at(p, head.row0, head.head, r), lane, m, l, acc);
}

inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

long long units_bound(int block_size, int max_blocks) {   // of one segment
    return ((long long)max_blocks * block_size + kTile - 1) / kTile + kStartUnits;
}

// Sequences of one launch: their lengths fit on chip.
int slice_of(int num_seqs) { return min(num_seqs, kMaxSeqs); }

// num_kv_heads: times the segments of one.
long long line_bound(int num_seqs, int num_kv_heads, int block_size, int max_blocks) {
    return (long long)slice_of(num_seqs) * num_kv_heads * units_bound(block_size, max_blocks);
}

int parts_of(int rows) { return (rows + kSegmentRows - 1) / kSegmentRows; }

struct Layout {
    size_t firsts, pieces, bytes;
};

Layout layout_of(int ctas, int rows) {
    Layout w;
    const size_t piece = (size_t)piece_floats(rows) * sizeof(float);
    w.firsts = align256(2 * (size_t)ctas * piece);
    w.pieces = w.firsts + align256((size_t)ctas * kManyWarps * piece);
    w.bytes = w.pieces + align256((size_t)ctas * sizeof(CtaPieces));
    return w;
}

template <typename T, int NT, int kW, bool kMulti, bool kScored>
cudaError_t launch_kind(const StreamLaunch& p, int ctas, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    constexpr size_t smem = 1024 + Smem<NT, kW>::kBytes;
    auto kernel = stream_kernel<T, NT, kW, kMulti, kScored>;
    cudaError_t e;
    static std::atomic<unsigned long long> allowed{0};   // devices on which the kernel may have its shared memory
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev > 63 || !(allowed.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(dev > 63 ? 0 : bit);
    }
    e = launch_pdl(kernel, dim3(ctas), dim3(Smem<NT, kW>::kThreads), smem, stream, p, k, v);
    if (e != cudaSuccess || ctas == 1) return e;
    // as many warps to a row as a segment has pieces when all are equally long
    const int pieces = ctas / max(1, min(ctas, p.a.num_seqs * p.a.num_kv_heads * p.row_parts));
    const int split = pieces >= 32 ? 8 : pieces >= 16 ? 4 : pieces >= 8 ? 2 : 1;
    const int grid_y = (p.rows * split + kJoinWarps - 1) / kJoinWarps;
    return launch_pdl(stream_join_kernel<T>, dim3(ctas - 1, grid_y), dim3(kJoinWarps * 32), 0, stream, p, ctas, split);
}

template <typename T, int NT, int kW>
cudaError_t launch_rows(const StreamLaunch& p, int ctas, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    const bool scored = p.a.cap > 0.f || p.a.slopes;
    if (p.a.q_start)
        return scored ? launch_kind<T, NT, kW, true, true>(p, ctas, k, v, stream)
                      : launch_kind<T, NT, kW, true, false>(p, ctas, k, v, stream);
    return scored ? launch_kind<T, NT, kW, false, true>(p, ctas, k, v, stream)
                  : launch_kind<T, NT, kW, false, false>(p, ctas, k, v, stream);
}

// Twelve warps a CTA for up to 8 rows, whose waits fill one another's (256 short chats of 32 heads 116 -> 113 us, 64
// sequences of up to 2048 tokens 15.9 -> 14.8); eight where one CTA takes all (9.3 -> 8.5: fewer pieces), or with more rows,
// whose accumulators need the registers.
bool many_warps(int rows, int ctas) { return rows <= 8 && ctas > 1; }

template <typename T>
cudaError_t launch_type(const StreamLaunch& p, int ctas, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    if (many_warps(p.rows, ctas)) return launch_rows<T, 1, kManyWarps>(p, ctas, k, v, stream);
    return p.rows <= 8 ? launch_rows<T, 1, kFewWarps>(p, ctas, k, v, stream)
                       : launch_rows<T, 2, kFewWarps>(p, ctas, k, v, stream);
}

}  // namespace

// One CTA per SM, fewer for little work: a cut between CTAs costs the joining launch (2.5 us), so at the longest contexts
// the tables allow one CTA takes up to eight units a warp alone, and several take four at least.
int stream_ctas(int num_seqs, int num_kv_heads, int rows, int block_size, int max_blocks, int most) {
    const long long units = line_bound(num_seqs, num_kv_heads * parts_of(rows), block_size, max_blocks);
    if (units <= 8 * kFewWarps) return 1;
    const int sms = sm_count_current();
    return (int)min((units + 4 * kFewWarps - 1) / (4 * kFewWarps), (long long)(most > 0 ? min(most, sms) : sms));
}

size_t stream_workspace_bytes(int num_seqs, int ctas, int rows) {
    return num_seqs == 0 ? 0 : layout_of(ctas, min(rows, kSegmentRows)).bytes;
}

bool stream_line_fits(int num_seqs, int num_kv_heads, int block_size, int max_blocks_per_seq) {
    const int heads = num_kv_heads * parts_of(kStreamRows);
    return line_bound(num_seqs, heads, block_size, max_blocks_per_seq) / kFewWarps < (1LL << 30);   // even one CTA's shares
}

cudaError_t launch_attend_stream(const AttendArgs& a, int dtype, int ctas, bool early, void* workspace,
                                 cudaStream_t stream) {
    CUtensorMap k, v;
    const unsigned long long pool_rows = (unsigned long long)a.num_blocks * a.num_kv_heads * a.block_size;
    if (!encode_pool_map(a.k_cache, pool_rows, kTile, &k)) {
        // a host thread that has made no CUDA call yet has no current context, which the encoding asks for
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess ||
            !encode_pool_map(a.k_cache, pool_rows, kTile, &k))
            return cudaErrorInvalidValue;
    }
    if (!encode_pool_map(a.v_cache, pool_rows, kTile, &v)) return cudaErrorInvalidValue;
    StreamLaunch p;
    p.group = a.num_q_heads / a.num_kv_heads;
    p.group_inv = (65536u + p.group - 1) / p.group;
    p.row_parts = parts_of(p.group * a.max_q);
    p.rows = min(p.group * a.max_q, kSegmentRows);
    const Layout w = layout_of(ctas, p.rows);
    char* ws = static_cast<char*>(workspace);
    p.parts = reinterpret_cast<float*>(ws);
    p.firsts = reinterpret_cast<float*>(ws + w.firsts);
    p.pieces = reinterpret_cast<CtaPieces*>(ws + w.pieces);
    // larger batches go in slices, one after another
    const int slice = slice_of(a.num_seqs);
    for (int s0 = 0; s0 < a.num_seqs; s0 += slice) {
        p.a = a;
        p.seq0 = s0;
        p.block_log2 = __builtin_ctz(a.block_size);
        p.early = early && s0 == 0;   // (later ones write the pieces that the join before them reads)
        p.a.num_seqs = min(slice, a.num_seqs - s0);
        p.a.block_tables += (size_t)s0 * a.max_blocks_per_seq;
        p.a.context_lens += s0;
        if (a.bidirectional) p.a.bidirectional += s0;
        if (a.q_start) {
            p.a.q_start += s0;
        } else {
            const size_t rows = (size_t)s0 * a.num_q_heads;
            p.a.q = static_cast<const uint16_t*>(a.q) + rows * kHeadDim;
            if (a.first_key) p.a.first_key += s0;
            if (a.part_o) {
                p.a.part_o += rows * kHeadDim;
                p.a.part_ml += rows;
            } else {
                p.a.out = static_cast<uint16_t*>(a.out) + rows * kHeadDim;
            }
        }
        const cudaError_t e = dtype == PA_BF16 ? launch_type<__nv_bfloat16>(p, ctas, k, v, stream)
                                               : launch_type<__half>(p, ctas, k, v, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace pa
