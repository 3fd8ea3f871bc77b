// Attention over the 8-bit paged cache: one query token per sequence, or several attending causally.
//
// What it computes ("显存虚拟化革命：PagedAttention 内存池管理与显存碎片终结", §五.1, over codes and
// exponents): for query row i of sequence s at position p = L - n + i and query head h,
//   out = sum_{t <= p} softmax_t(scale * q . (2^ke K_t)) * 2^ve V_t
// with K_t, V_t the codes of token t and ke, ve its block's exponents.  Tokens of a block whose table
// entry lies outside the pool are left out.
//
// The exponents cost a product each: with x_t = scale log2(e) 2^ke (q . K_t) and a base b,
//   p_t = 2^(x_t - b),  P_t = p_t 2^ve,  O = sum P_t V_t (codes),  l = sum p_t,  out = O / l,
// so V is never scaled, P_t stays in fp16's range whatever the blocks' scales (the base follows the maximum
// of x_t + ve, not of the score), and b cancels.  p_t keeps the weights' sum: between blocks of scales 2^-60 and
// 2^60 it spans 2^-51 .. 2^75 where it counts, inside fp32 (factors between bases may be subnormal: exp2f).
// Codes become fp16 exactly; P is rounded to fp16 for the PV product (fp32 sums): 2^-11 of a weight, averaged
// over the tokens.  The base leaves the largest P between 2^9 and 2^15, so that weights keep these bits down to
// 2^-23 of the largest, and steps of 2^-33 of it below: a long context's tail beside one dominant token (a base
// at the largest itself loses 3 % of the output with 131072 tokens and 98 % of the weight on one).  bf16 queries are scaled by a power of two per row into fp16's range (exact down to
// 2^-29 of the row's largest element).
//
// Work split: a segment is a (sequence, kv head); its 16-token tiles and two or three units for its start
// and end (`start_units`) lie on a line, segment after segment, and every warp of the grid takes an equal,
// contiguous share of the line.
// Warps are independent while they stream: each has a ring of tiles filled by its own TMA loads (2 KB of K
// and of V, 128-byte swizzle, so that the 16-byte fragment loads below meet no bank conflict).  A segment
// that lies in one warp's share goes straight to `out`; the pieces of a cut one meet in shared memory at the
// CTA's end and, where it is cut between CTAs, in the workspace, which a second small launch joins.  No
// atomics: every sum has one order, and the workspace needs no initial contents.
//
// Tile math (one warp, mma.sync m16n8k16, rows = tokens for QK and dims for PV, columns = query rows):
//   S = K Q^T: lane (g, t) = (lane / 4, lane % 4) holds bytes 32 t .. 32 t + 31 of tokens g and g + 8; the
//       product's k index is a permutation of the head's dims, the same one for the Q fragments.
//   O += V^T P^T: the lane holds dims 16 g .. 16 g + 15 of tokens 2t, 2t+1, 2t+8, 2t+9; byte permutes pair
//       the tokens of a dim.  P^T comes from S by movmatrix.
// The base moves only when a weight grows to 2^6 of the largest when it was taken (then O and l are rescaled), so
// most tiles need no shuffle.
//
// Bound by HBM (one byte per cached element) with up to 8 rows a segment: 16 contexts of 16384 tokens, 8 kv heads of
// 4 rows 86 us (6.2 TB/s, 0.92 of a copy's rate), 256 short chats of 32 heads 58 us (5.2 TB/s).  With more rows by the
// warps' waits for their own products: a tile of 32 rows fills a warp's registers, so that a scheduler has two warps,
// each in one chain of dependent steps (272 instructions a tile of 8 rows, 348 of 16, 541 of 32, about 0.36 a cycle and
// scheduler; waits of a fixed latency are the largest stall, two warps an issue).  The long contexts take 104 us with 16
// rows, 131 with 24 and 163 with 32.  The smallest calls are a chain of latencies: four short contexts 6.2 us, 64
// sequences of 16 to 2048 tokens 12.7 us.
#include <atomic>
#include <type_traits>

#include "decode_common.cuh"
#include "q8.cuh"
#include "q8_join.h"

namespace pa {

namespace {

// Warps of a CTA.  12 where a warp begins and ends several short segments, whose waits the others fill (256 short
// chats of 32 heads 62 -> 57 us); 8 elsewhere, with deeper rings and fewer streams (16 contexts of 16384 tokens
// 90 -> 85 us).
constexpr int kFewWarps = 8, kManyWarps = 12;
constexpr int kTile = 16;                       // tokens per tile
constexpr uint32_t kTileHalf = kTile * kHeadDim;   // 2 KB of K, 2 KB of V
constexpr uint32_t kTileBytes = 2 * kTileHalf;
// What a segment's start and end cost, in tiles: with more than 16 rows Q is fetched as it begins, not ahead.
__host__ __device__ constexpr int start_units(int rows) { return rows > 16 ? 3 : 2; }
constexpr int kQ8MaxSeqs = 1024;                // sequences of one launch (their lengths stay on chip)
// log2 of P: a new base puts the largest at 2^kTopNew, and moves when one would exceed 2^kTopMost (fp16's largest is
// below 2^16).  9 is the highest that costs nothing: one to five new tokens 22.8 us with 7 and 9, 23.5 with 11, 24.7
// with 13, since the base then moves more often.  (Scores of 2^24 and more leave few bits for such offsets: the distance
// to the base, not the sum with it, is compared, and a new base is rounded up.)
constexpr float kTopNew = 9.f, kTopMost = 15.f;

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

struct Q8Launch {
    DecodeQ8Args a;
    float* parts;         // [grid][2] pieces of `rows` rows
    float* firsts;        // [grid * warps] pieces, when they do not fit in shared memory
    CtaPieces* pieces;    // [grid]
    int rows;             // query rows of a segment at most (max_q * group)
    int group;            // query heads per kv head
    unsigned group_inv;   // ceil(2^16 / group)
};

template <int NT, int kW>
struct Q8Smem {
    static constexpr int kRows = NT * 8, kWarps = kW, kThreads = kWarps * 32;
    static constexpr bool kQInSmem = NT >= 3;              // Q fragments (16 registers per 8 rows) leave the registers
    static constexpr bool kFirstInSmem = NT <= 2;
    static constexpr int kStages = kW > kFewWarps ? 3 : NT == 1 ? 5 : 4;
    static constexpr uint32_t kRing = kStages * kTileBytes;  // per warp
    static constexpr uint32_t kOffFirst = kWarps * kRing;
    static constexpr uint32_t kOffLastMl = kOffFirst + (kFirstInSmem ? kWarps * piece_floats(kRows) * 4 : 0);
    static constexpr uint32_t kOffQ = kOffLastMl + kWarps * kRows * 8;
    static constexpr uint32_t kOffCol = kOffQ + (kQInSmem ? kWarps * NT * 16 * 32 * 4 : 0);
    static constexpr uint32_t kOffDesc = kOffCol + (kQInSmem ? kWarps * kRows * 8 : 0);
    static constexpr uint32_t kOffBar = kOffDesc + kWarps * 16;
    static constexpr uint32_t kOffP = kOffBar + kWarps * kStages * 8;
    static constexpr uint32_t kOffLen = kOffP + (kQ8MaxSeqs + 4) * 4;
    static constexpr uint32_t kOffRow0 = kOffLen + kQ8MaxSeqs * 4;   // several tokens: first row and count
    static constexpr uint32_t kOffN = kOffRow0 + kQ8MaxSeqs * 4;
    static constexpr uint32_t kBytes = kOffN + kQ8MaxSeqs;
    static_assert(kRing >= kRows * kHeadDim * 4, "a warp's last piece is kept in its ring");
    static_assert(1024 + kBytes + 64 <= 227 * 1024, "shared memory of one CTA");
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
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lo_f16x2(uint32_t w) { return e4m3x2_to_f16x2((uint16_t)(w & 0xffffu)); }
__device__ __forceinline__ uint32_t hi_f16x2(uint32_t w) { return e4m3x2_to_f16x2((uint16_t)(w >> 16)); }

// (m, l, acc) of one row joined with a piece; a piece that saw no token has base -inf.
__device__ __forceinline__ void add_piece(float& m, float& l, float4& acc, float2 ml, float4 v) {
    const float m2 = fmaxf(m, ml.x);
    const float f0 = m == -INFINITY ? 0.f : exp2f(m - m2), f1 = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m2);
    m = m2;
    l = l * f0 + ml.y * f1;
    acc.x = acc.x * f0 + v.x * f1;
    acc.y = acc.y * f0 + v.y * f1;
    acc.z = acc.z * f0 + v.z * f1;
    acc.w = acc.w * f0 + v.w * f1;
}

// Four elements of a finished row; a row that saw no token is zero.
template <typename T>
__device__ __forceinline__ void store_row4(void* out, size_t at, float l, const float4& acc) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2 w;
    w.x = Elem<T>::pack2(acc.x * inv, acc.y * inv);
    w.y = Elem<T>::pack2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + at) = w;
}

// Query token of row r of a segment, r / group for r < 32, by the multiplier that p.group_inv holds.
__device__ __forceinline__ int token_of(const Q8Launch& p, int r) { return (int)((unsigned)r * p.group_inv >> 16); }

// Element of query row r (token r / group, group member r % group) of kv head h's segment.
__device__ __forceinline__ size_t row_at(const Q8Launch& p, int row0, int h, int r) {
    const int i = token_of(p, r);
    return ((size_t)(row0 + i) * p.a.num_q_heads + (size_t)h * p.group + r - i * p.group) * kHeadDim;
}

// In a piece in shared memory, 16-byte chunk c of row r lies at c ^ (r / 2 % 4): the lanes that store
// a fragment (four row pairs at once) then meet no bank conflict.
__device__ __forceinline__ int chunk_of(int r, int c) { return r * (kHeadDim / 4) + (c ^ (r >> 1 & 3)); }

template <typename T, int NT, int kW, bool kMulti>
__global__ void __launch_bounds__(Q8Smem<NT, kW>::kThreads, 1)
    q8_attend_kernel(const Q8Launch p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using M = Q8Smem<NT, kW>;
    constexpr int kStages = M::kStages, kStartUnits = start_units(NT * 8);
    constexpr uint32_t kAll = 0xffffffffu;
    const DecodeQ8Args& a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, t = lane % 4;
    int* P = reinterpret_cast<int*>(smem + M::kOffP);
    int* lens = reinterpret_cast<int*>(smem + M::kOffLen);
    int* row0_of = reinterpret_cast<int*>(smem + M::kOffRow0);
    uint8_t* n_of = smem + M::kOffN;
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kOffBar) + warp * kStages;
    WarpPieces* wp = reinterpret_cast<WarpPieces*>(smem + M::kOffDesc);
    const uint32_t ring = smem_u32(smem) + warp * M::kRing;

    if (lane < kStages) {
        mbar_init(&bars[lane], 1);
        fence_mbar_init();
    }
    if (tid == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- lengths, and the units of one kv head before each sequence (P) ----
    const int S = a.num_seqs, Hkv = a.num_kv_heads, group = p.group;
    {
        __shared__ int warp_sum_of[M::kWarps];
        int carry = 0;
        for (int s0 = 0; s0 < S; s0 += M::kThreads) {
            const int s = s0 + tid;
            int w = 0;
            if (s < S) {
                bool bad;
                const int L = clamped_len(a.context_lens, s, a.max_blocks_per_seq, a.block_size, &bad);
                int n = 1;
                if (kMulti) {
                    const NewRows nr = new_rows(a.q_start, a.q_rows, a.max_q, s, L);
                    n = nr.n;
                    bad |= nr.bad;
                    row0_of[s] = nr.row0;
                    n_of[s] = (uint8_t)n;
                }
                if (bad && blockIdx.x == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
                lens[s] = L;
                if (L > 0 && n > 0) w = (L + kTile - 1) / kTile + kStartUnits;
            }
            int incl = w;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(kAll, incl, o);
                if (lane >= o) incl += v;
            }
            if (s0 > 0) __syncthreads();   // warp_sum_of of the round before has been read
            if (lane == 31) warp_sum_of[warp] = incl;
            __syncthreads();
            int before = carry + incl - w;
#pragma unroll
            for (int i = 0; i < M::kWarps; ++i) {
                const int x = warp_sum_of[i];
                if (i < warp) before += x;
                carry += x;
            }
            if (s < S) P[s] = before;
        }
        if (tid == 0) P[S] = carry;
        __syncthreads();
    }

    const long long total = (long long)P[S] * Hkv;
    // share i of the line begins at unit floor(total * i / shares) (32-bit divisions: 64-bit ones take 0.3 us each)
    const unsigned shares = gridDim.x * M::kWarps, me = blockIdx.x * M::kWarps + warp;
    const long long each = total >> 32 ? total / shares : (long long)((unsigned)total / shares);
    const unsigned odd = (unsigned)(total - each * shares);
    auto share_at = [&](unsigned i) { return each * i + (odd * i) / shares; };
    // A cut among a segment's start units goes before them: its first tile begins the segment in any case, and the
    // share before would leave an empty piece.  In a short segment a cut next to its first or last tile goes to the
    // begin or the end, too, since the piece costs more than the tile (four contexts of up to 64 tokens 7.5 us without,
    // 6.2 with; 64 contexts of up to 2048 tokens, 30 rows 25.9 and 25.4; few rows of longer contexts gain nothing:
    // their shares only become unequal).
    auto near_of = [&](int w) {
        return (M::kWarps > kFewWarps || NT > 1 || gridDim.x == 1) && w <= kStartUnits + 8 ? 1 : 0;
    };
    // The share's first unit (r of segment (s, h)) and, by the upper half of the warp, the next share's.
    int s, h, r, units;
    long long u0;
    {
        const int half = lane & 16, of_half = lane & 15;
        long long u = share_at(me + (half >> 4));
        s = 0;   // the last s with P[s] * Hkv <= u
        for (int n = S; n > 1;) {
            n = (n + 15) / 16;
            const int at = s + of_half * n;
            const unsigned m = __ballot_sync(kAll, at < S && (long long)P[min(at, S)] * Hkv <= u) >> half & 0xffff;
            s += (31 - __clz(m)) * n;
        }
        const int w = max(1, P[s + 1] - P[s]);
        const unsigned long long rem = u - (long long)P[s] * Hkv;
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
                if (++h == Hkv) {
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
    const uint32_t v_off0 = kTileHalf + (2 * t) * 128 + ((uint32_t)(g ^ (2 * t)) << 4);
    const uint32_t v_off1 = kTileHalf + (2 * t + 1) * 128 + ((uint32_t)(g ^ (2 * t + 1)) << 4);

    float o[NT][8][4];
    float base[NT][2], sum[NT][2];
    // of this lane's score columns (rows 2 t and 2 t + 1 of each 8): the factor to log2 units and the last
    // position the row sees; with Q in shared memory these are kept there too
    float qf_reg[M::kQInSmem ? 1 : NT][2] = {};
    int lim_reg[M::kQInSmem ? 1 : NT][2] = {};
    float2* qf_sm = reinterpret_cast<float2*>(smem + M::kOffCol) + warp * M::kRows;          // [NT][4] factors,
    int2* lim_sm = reinterpret_cast<int2*>(qf_sm + M::kRows / 2);                            // [NT][4] limits
    auto qf_of = [&](int nt) {
        return M::kQInSmem ? qf_sm[nt * 4 + t] : make_float2(qf_reg[M::kQInSmem ? 0 : nt][0], qf_reg[M::kQInSmem ? 0 : nt][1]);
    };
    auto lim_of = [&](int nt) {
        return M::kQInSmem ? lim_sm[nt * 4 + t] : make_int2(lim_reg[M::kQInSmem ? 0 : nt][0], lim_reg[M::kQInSmem ? 0 : nt][1]);
    };
    uint32_t qreg[M::kQInSmem ? 1 : NT][16];
    uint4* qsm = reinterpret_cast<uint4*>(smem + M::kOffQ) + warp * NT * 4 * 32 + lane;
    uint4 qn[M::kQInSmem ? 1 : NT][4];   // Q rows of the segment that comes next, as they lie in memory
    int L = 0, row0 = 0, nrows = 0, p0 = 0;
    uint32_t phases = 0;

    // Loads of Q row 8 nt + g, dims 32 t .. 32 t + 31 of segment (s, h).
    auto load_q = [&](int s, int h, int nt, uint4 (&to)[4]) {
        const int first = kMulti ? row0_of[s] : s, rows = (kMulti ? n_of[s] : 1) * group, r = nt * 8 + g;
        const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                          row_at(p, first, h, r < rows ? r : 0) + 32 * t);
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = r < rows ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
    };
    // Ahead of a segment's begin, as far as registers hold the rows.
    auto fetch_q = [&](int s, int h) {
        if (!M::kQInSmem) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) load_q(s, h, nt, qn[M::kQInSmem ? 0 : nt]);
        }
    };

    // Q fragments of the segment, their scales, and the positions its rows see.
    auto begin_segment = [&]() {
        L = lens[s];
        row0 = kMulti ? row0_of[s] : s;
        const int n = kMulti ? n_of[s] : 1;
        nrows = n * group;
        p0 = L - n;
        uint4 now[M::kQInSmem ? NT : 1][4];
        if (M::kQInSmem) {   // the accumulators are not live here: room for all rows at once
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) load_q(s, h, nt, now[M::kQInSmem ? nt : 0]);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 w = M::kQInSmem ? now[M::kQInSmem ? nt : 0][i] : qn[M::kQInSmem ? 0 : nt][i];
                x[4 * i] = w.x;
                x[4 * i + 1] = w.y;
                x[4 * i + 2] = w.z;
                x[4 * i + 3] = w.w;
            }
            float2 qf = make_float2(a.scale_log2, a.scale_log2);
            if (std::is_same<T, __nv_bfloat16>::value) {
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = Elem<T>::to_float2(x[i]);
                    amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
                }
                amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(kAll, amax, 2));
                // largest element into [2^14, 2^15)
                const int up = max(-126, min(126, 14 - ((__float_as_int(amax) >> 23) - 127)));
                const float mul = exp2_int(up), scale = exp2_int(-up);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = Elem<T>::to_float2(x[i]);
                    x[i] = Elem<__half>::pack2(f.x * mul, f.y * mul);
                }
                qf.x = __shfl_sync(kAll, scale, (2 * t) * 4) * a.scale_log2;
                qf.y = __shfl_sync(kAll, scale, (2 * t + 1) * 4) * a.scale_log2;
            }
            if (M::kQInSmem) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    qsm[(nt * 4 + i) * 32] = make_uint4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) qreg[M::kQInSmem ? 0 : nt][i] = x[i];
            }
            int lim[2];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = nt * 8 + 2 * t + c;
                lim[c] = kMulti && col < nrows ? p0 + token_of(p, col) : L - 1;
                base[nt][c] = -INFINITY;
                sum[nt][c] = 0.f;
            }
            if (M::kQInSmem) {
                if (g == 0) {
                    qf_sm[nt * 4 + t] = qf;
                    lim_sm[nt * 4 + t] = make_int2(lim[0], lim[1]);
                }
            } else {
                qf_reg[M::kQInSmem ? 0 : nt][0] = qf.x;
                qf_reg[M::kQInSmem ? 0 : nt][1] = qf.y;
                lim_reg[M::kQInSmem ? 0 : nt][0] = lim[0];
                lim_reg[M::kQInSmem ? 0 : nt][1] = lim[1];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
        }
        if (M::kQInSmem) __syncwarp();
    };

    // One tile of tokens t0 .. t0 + 15 against the first K x 8 rows.
    auto run_tile = [&](auto kc, uint32_t tile, int t0, int ke, int ve) {
        constexpr int K = decltype(kc)::value;
        // S = K Q^T
        float x[K][4];
        {
            const uint4 k0 = lds128(tile + k_off0), k1 = lds128(tile + k_off1);
            const uint4 k2 = lds128(tile + k_off0 + 1024), k3 = lds128(tile + k_off1 + 1024);
            const uint32_t ka[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
            const uint32_t kb[8] = {k2.x, k2.y, k2.z, k2.w, k3.x, k3.y, k3.z, k3.w};
            float y[K][4];   // one tile of rows: odd steps on their own, for two short chains
#pragma unroll
            for (int nt = 0; nt < K; ++nt)
#pragma unroll
                for (int c = 0; c < 4; ++c) x[nt][c] = y[nt][c] = 0.f;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                uint4 b[K];
#pragma unroll
                for (int nt = 0; nt < K; ++nt) {
                    if (M::kQInSmem) b[nt] = qsm[(nt * 4 + q) * 32];
                    else
                        b[nt] = make_uint4(qreg[M::kQInSmem ? 0 : nt][4 * q], qreg[M::kQInSmem ? 0 : nt][4 * q + 1],
                                           qreg[M::kQInSmem ? 0 : nt][4 * q + 2], qreg[M::kQInSmem ? 0 : nt][4 * q + 3]);
                }
                {
                    const uint32_t a0 = lo_f16x2(ka[2 * q]), a1 = lo_f16x2(kb[2 * q]), a2 = hi_f16x2(ka[2 * q]),
                                   a3 = hi_f16x2(kb[2 * q]);
#pragma unroll
                    for (int nt = 0; nt < K; ++nt) mma16816<__half>(x[nt], a0, a1, a2, a3, b[nt].x, b[nt].y);
                }
                {
                    const uint32_t a0 = lo_f16x2(ka[2 * q + 1]), a1 = lo_f16x2(kb[2 * q + 1]),
                                   a2 = hi_f16x2(ka[2 * q + 1]), a3 = hi_f16x2(kb[2 * q + 1]);
#pragma unroll
                    for (int nt = 0; nt < K; ++nt)
                        mma16816<__half>(K == 1 ? y[nt] : x[nt], a0, a1, a2, a3, b[nt].z, b[nt].w);
                }
            }
            if (K == 1) {
#pragma unroll
                for (int c = 0; c < 4; ++c) x[0][c] += y[0][c];
            }
        }
        uint4 v0 = lds128(tile + v_off0), v1 = lds128(tile + v_off1);
        uint4 v2 = lds128(tile + v_off0 + 1024), v3 = lds128(tile + v_off1 + 1024);

        // x = score in log2 units; positions a row does not see to -inf
        const float ks = exp2_int(ke), vs = exp2_int(ve), vef = (float)ve, slack = kTopMost - vef;
        const bool masked = t0 + kTile > p0 + 1;
        bool nan_v = false;
#pragma unroll
        for (int nt = 0; nt < K; ++nt) {
            const float2 qf = qf_of(nt);
#pragma unroll
            for (int c = 0; c < 4; ++c) x[nt][c] *= (c & 1 ? qf.y : qf.x) * ks;
        }
        if (masked) {
#pragma unroll
            for (int nt = 0; nt < K; ++nt) {
                const int2 lim = lim_of(nt);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (t0 + g + (c >> 1) * 8 > (c & 1 ? lim.y : lim.x)) x[nt][c] = -INFINITY;
            }
            // rows behind the last token hold anything: zero codes
            const int left = L - t0;
            if (2 * t >= left) v0 = make_uint4(0, 0, 0, 0);
            if (2 * t + 1 >= left) v1 = make_uint4(0, 0, 0, 0);
            if (2 * t + 8 >= left) v2 = make_uint4(0, 0, 0, 0);
            if (2 * t + 9 >= left) v3 = make_uint4(0, 0, 0, 0);
            if (kMulti) {
                // a NaN of a token that some rows do not see must not reach them through 0 * NaN
                auto nans = [](uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); };
                auto any4 = [&](const uint4& v) { return nans(v.x) | nans(v.y) | nans(v.z) | nans(v.w); };
                nan_v = __any_sync(kAll, (any4(v0) | any4(v1) | any4(v2) | any4(v3)) != 0);
                if (nan_v) {
                    auto drop = [&](uint4& v) {
                        v.x &= ~nans(v.x);
                        v.y &= ~nans(v.y);
                        v.z &= ~nans(v.z);
                        v.w &= ~nans(v.w);
                    };
                    drop(v0);
                    drop(v1);
                    drop(v2);
                    drop(v3);
                }
            }
        }
        bool move = false;   // a column without a base yet (-inf) takes one as soon as it sees a token
#pragma unroll
        for (int nt = 0; nt < K; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) move |= fmaxf(x[nt][c], x[nt][c + 2]) - base[nt][c] > slack;
        if (__any_sync(kAll, move)) {
#pragma unroll
            for (int nt = 0; nt < K; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    float m = fmaxf(x[nt][c], x[nt][c + 2]);
#pragma unroll
                    for (int k = 4; k < 32; k <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, k));
                    m = fmaxf(__fadd_ru(m, vef - kTopNew), base[nt][c]);   // never below: P must stay in range
                    const float f = base[nt][c] == -INFINITY ? 0.f : exp2f(base[nt][c] - m);
                    base[nt][c] = m;
                    sum[nt][c] *= f;
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        o[nt][k][c] *= f;
                        o[nt][k][c + 2] *= f;
                    }
                }
        }
        uint32_t b0[K], b1[K];
#pragma unroll
        for (int nt = 0; nt < K; ++nt) {
            float pr[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) pr[c] = ex2(x[nt][c] - base[nt][c & 1]);
            if (masked) {   // a row without a base yet has -inf - -inf here
                const int2 lim = lim_of(nt);
#pragma unroll
                for (int c = 0; c < 4; ++c)
                    if (t0 + g + (c >> 1) * 8 > (c & 1 ? lim.y : lim.x)) pr[c] = 0.f;
            }
            sum[nt][0] += pr[0] + pr[2];
            sum[nt][1] += pr[1] + pr[3];
            b0[nt] = movmatrix_trans(Elem<__half>::pack2(pr[0] * vs, pr[1] * vs));
            b1[nt] = movmatrix_trans(Elem<__half>::pack2(pr[2] * vs, pr[3] * vs));
        }
        // O += V^T P^T
        const uint32_t va[4] = {v0.x, v0.y, v0.z, v0.w}, vb[4] = {v1.x, v1.y, v1.z, v1.w};
        const uint32_t vc[4] = {v2.x, v2.y, v2.z, v2.w}, vd[4] = {v3.x, v3.y, v3.z, v3.w};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint32_t sel = e ? 0x7362 : 0x5140;   // dims 2e, 2e+1 of tokens (first, second)
                const uint32_t ab = __byte_perm(va[q], vb[q], sel), cd = __byte_perm(vc[q], vd[q], sel);
                const uint32_t a0 = lo_f16x2(ab), a1 = hi_f16x2(ab), a2 = lo_f16x2(cd), a3 = hi_f16x2(cd);
#pragma unroll
                for (int nt = 0; nt < K; ++nt) mma16816<__half>(o[nt][2 * q + e], a0, a1, a2, a3, b0[nt], b1[nt]);
            }
        }
        if (kMulti && nan_v) {
            // rare: NaN into the dims and rows that see such a token
            for (int j = 0; j < min(kTile, L - t0); ++j) {
                const uint4 v = lds128(tile + kTileHalf + j * 128 + ((uint32_t)(g ^ (j & 7)) << 4));
                const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int d = 0; d < 16; ++d)
                    if (((vw[d / 4] >> (8 * (d % 4))) & 0x7f) == 0x7f)
#pragma unroll
                        for (int nt = 0; nt < K; ++nt)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
                                if (t0 + j <= (c ? lim_of(nt).y : lim_of(nt).x)) o[nt][d / 2][c + 2 * (d % 2)] = __int_as_float(0x7fffffff);
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

    auto store_piece = [&](float4* slot, float2* ml) {
        finish_sums();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = nt * 8 + 2 * t + c;
                if (r < nrows) {
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        slot[chunk_of(r, g * 4 + i / 2)] =
                            make_float4(o[nt][i][c], o[nt][i][c + 2], o[nt][i + 1][c], o[nt][i + 1][c + 2]);
                    if (g == 0) ml[r] = make_float2(base[nt][c], sum[nt][c]);
                }
            }
    };

    auto store_out = [&]() {
        finish_sums();
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int r = nt * 8 + 2 * t + c;
                if (r < nrows) {
                    const float inv = sum[nt][c] == 0.f ? 0.f : 1.f / sum[nt][c];
                    uint32_t w[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) w[i] = Elem<T>::pack2(o[nt][i][c] * inv, o[nt][i][c + 2] * inv);
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row_at(p, row0, h, r) +
                                                          g * 16);
                    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
    };

    // pieces of warp w: the first in memory of its own, the last in its ring (every copy has landed)
    const int slot_rows = M::kFirstInSmem ? M::kRows : p.rows;
    auto first_of = [&](int w) {
        return reinterpret_cast<float4*>(
            M::kFirstInSmem ? reinterpret_cast<float*>(smem + M::kOffFirst) + w * piece_floats(M::kRows)
                            : p.firsts + ((size_t)blockIdx.x * M::kWarps + w) * piece_floats(p.rows));
    };
    auto last_of = [&](int w) { return reinterpret_cast<float4*>(smem + w * M::kRing); };
    auto first_ml_of = [&](int w) { return reinterpret_cast<float2*>(first_of(w) + slot_rows * kHeadDim / 4); };
    auto last_ml_of = [&](int w) { return reinterpret_cast<float2*>(smem + M::kOffLastMl) + w * M::kRows; };

    // ---- the stream ----
    WarpPieces mine{units == 0 ? kNoUnits : 0, 0, 0, 0};
    if (units > 0) {
        // of the unit this lane owns in a window of 32: the pool row of its tile's first token (-1: a start
        // unit or none, -2: a block outside the pool) and its block's exponents
        int A_y = -1, A_ke = 0, A_ve = 0, B_y = -1, B_ke = 0, B_ve = 0, lane_s = s;
        auto look = [&](int i, int& y, int& ke, int& ve) {   // unit u0 + i; i grows from call to call
            y = -1;
            if (i >= units) return;
            const long long u = u0 + i;
            while ((long long)P[lane_s + 1] * Hkv <= u) ++lane_s;
            const uint32_t w = P[lane_s + 1] - P[lane_s];
            const unsigned long long rem = u - (long long)P[lane_s] * Hkv;
            const int hh = rem <= 0xffffffffu ? (uint32_t)rem / w : (int)(rem / w);
            const int r = (int)(rem - (unsigned long long)hh * w);
            if (r < kStartUnits) return;
            const int t0 = (r - kStartUnits) * kTile, B = a.block_size;
            const int id = __ldg(a.block_tables + (size_t)lane_s * a.max_blocks_per_seq + t0 / B);
            if (id < 0 || id >= a.num_blocks) {
                flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
                y = -2;
                return;
            }
            const int tile = id * Hkv + hh;                // fits: num_blocks * Hkv * B < 2^31
            y = tile * B + t0 % B;
            ke = __ldg(a.k_exp + tile);
            ve = __ldg(a.v_exp + tile);
        };
        fetch_q(s, h);
        look(lane, A_y, A_ke, A_ve);
        auto issue = [&](int j, int y) {   // by the lane that owns unit j
            const int st = j % kStages;
            const uint32_t dst = ring + st * kTileBytes;
            mbar_arrive_expect_tx(&bars[st], kTileBytes);
            tma_load_2d(dst, &kmap, 0, y, &bars[st]);
            tma_load_2d(dst + kTileHalf, &vmap, 0, y, &bars[st]);
        };
        if (lane < kStages && A_y >= 0) issue(lane, A_y);
        bool dead = false;
        int i = 0;
        while (i < units) {
            // segment (s, h) from its unit r on
            const int left = P[s + 1] - P[s] - r, stop = min(units, i + left);
            const bool from_before = r > 0, ends = i + left <= units;
            begin_segment();
            const int this_s = s, this_h = h;
            int next_s = s, next_h = h + 1;
            if (i + left < units) {
                if (next_h == Hkv) {
                    next_h = 0;
                    do ++next_s;
                    while (P[next_s + 1] == P[next_s]);
                }
                fetch_q(next_s, next_h);
            }
            const int tiles_of_8 = (nrows + 7) / 8;
            for (; i < stop; ++i, ++r) {
                const int w = i & 31;
                if (w == 0) {
                    if (i > 0) {
                        A_y = B_y;
                        A_ke = B_ke;
                        A_ve = B_ve;
                    }
                    if (i + 32 < units) look(i + 32 + lane, B_y, B_ke, B_ve);
                }
                const int y = __shfl_sync(kAll, A_y, w);
                if (y >= 0) {
                    const int ke = clamp_exp(__shfl_sync(kAll, A_ke, w)), ve = clamp_exp(__shfl_sync(kAll, A_ve, w));
                    const int st = i % kStages;
                    if (!mbar_wait_bounded(&bars[st], (phases >> st) & 1)) {
                        flag_status(a.status, PA_DEV_TIMEOUT);
                        dead = true;
                    }
                    dead = __any_sync(kAll, dead);
                    if (dead) break;
                    phases ^= 1u << st;
                    const uint32_t tile = ring + st * kTileBytes;
                    const int t0 = (r - kStartUnits) * kTile;
                    if (!kMulti || NT == 1) {
                        run_tile(std::integral_constant<int, NT>{}, tile, t0, ke, ve);
                    } else {
                        switch (tiles_of_8) {
                            case 1: run_tile(std::integral_constant<int, 1>{}, tile, t0, ke, ve); break;
                            case 2: run_tile(std::integral_constant<int, 2>{}, tile, t0, ke, ve); break;
                            case 3: run_tile(std::integral_constant<int, NT < 3 ? NT : 3>{}, tile, t0, ke, ve); break;
                            default: run_tile(std::integral_constant<int, NT>{}, tile, t0, ke, ve); break;
                        }
                    }
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
                store_out();
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
        constexpr int kGroup = M::kWarps <= 8 ? 8 : 16, kTake = 32 / kGroup;   // lanes a row, rows at a time
        const WarpPieces x = lane < M::kWarps ? wp[lane] : WarpPieces{kNoUnits, 0, 0, 0};
        const CtaJoin join = cta_join(__ballot_sync(kAll, x.flags & kNoUnits), __ballot_sync(kAll, x.flags & kHasFirst),
                                      __ballot_sync(kAll, x.flags & kHasLast), __ballot_sync(kAll, x.flags & kThrough),
                                      __ballot_sync(kAll, x.flags & kGaveUp), M::kWarps);
        const unsigned some = join.some, events = join.events;
        const int last_warp = join.last_warp;
        left_first = join.left_first;
        left_last = join.left_last;
        if (left_last) left_seg = __shfl_sync(kAll, x.last_seg, last_warp);
        const int batches = (p.rows + kTake - 1) / kTake, items = __popc(events) * batches;
        for (int item = warp; item < items; item += M::kWarps) {
            unsigned ev = events;
            int k = item;
            for (; k >= batches; k -= batches) ev &= ev - 1;
            const JoinChain chain = join.chain(ev);
            const int ws = chain.from, we = chain.to;
            const bool closed = we < M::kWarps, before = chain.before;
            const unsigned pieces = some & ~((1u << ws) - 1) & ((2u << we) - 1);
            const int seg = __shfl_sync(kAll, closed ? x.first_seg : x.last_seg, closed ? we : last_warp);
            const int sg = seg >> 16, hh = seg & 0xffff, r0 = k * kTake;
            const int first = kMulti ? row0_of[sg] : sg, rows = (kMulti ? n_of[sg] : 1) * group;
            if (r0 >= rows) continue;
            float* to = p.parts + ((size_t)blockIdx.x * 2 + (before ? 0 : 1)) * piece_floats(p.rows);
            // four rows at a time: lane 8 i + w weighs warp w's piece of row i, then every lane has four
            // elements of each row
            const int w = lane % kGroup, rw = r0 + lane / kGroup;
            float4 vf[kTake];   // the piece that ends the chain (in memory with many rows), on its way early
#pragma unroll
            for (int i = 0; i < kTake; ++i)
                if (closed && r0 + i < rows) vf[i] = first_of(we)[chunk_of(r0 + i, lane)];
            float2 ml = make_float2(-INFINITY, 0.f);
            if ((pieces >> w & 1) && rw < rows) ml = (closed && w == we ? first_ml_of(w) : last_ml_of(w))[rw];
            float m = ml.x;
#pragma unroll
            for (int k = 1; k < kGroup; k <<= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, k));
            const float f = ml.x == -INFINITY ? 0.f : exp2f(ml.x - m);
            float l = f * ml.y;
#pragma unroll
            for (int k = 1; k < kGroup; k <<= 1) l += __shfl_xor_sync(kAll, l, k);
            float4 acc[kTake];
#pragma unroll
            for (int i = 0; i < kTake; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
            const int last_end = closed ? we : last_warp + 1;
#pragma unroll 1
            for (int pw = ws; pw < last_end; pw += 2) {   // last pieces, two at a time
                const bool one = pieces >> pw & 1, two = pw + 1 < last_end && (pieces >> (pw + 1) & 1);
                float4 v[2][kTake];
#pragma unroll
                for (int i = 0; i < kTake; ++i) {
                    v[0][i] = v[1][i] = make_float4(0.f, 0.f, 0.f, 0.f);
                    if (one && r0 + i < rows) v[0][i] = last_of(pw)[chunk_of(r0 + i, lane)];
                    if (two && r0 + i < rows) v[1][i] = last_of(pw + 1)[chunk_of(r0 + i, lane)];
                }
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int i = 0; i < kTake; ++i) {
                        const float fw = __shfl_sync(kAll, f, i * kGroup + ((pw + k) & (kGroup - 1)));
                        const float4 x = v[k][i];
                        if (k ? two : one) {
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
                        store_row4<T>(a.out, row_at(p, first, hh, r) + lane * 4, li, acc[i]);
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
            const int w = P[sg + 1] - P[sg];
            const long long last_unit = (long long)P[sg] * Hkv + (long long)(hh + 1) * w - 1;
            int i = max(0, min((int)((float)last_unit * (float)shares / (float)total), (int)shares - 1));
            while (share_at(i) > last_unit) --i;
            while (share_at(i + 1) <= last_unit) ++i;
            const int near = near_of(w);   // (cuts moved to the segment's end)
            while (last_unit + 1 - share_at(i) <= near && w - (last_unit + 1 - share_at(i)) > kStartUnits + near) --i;
            left.end = i / M::kWarps;
            left.row0 = kMulti ? row0_of[sg] : sg;
            left.rows = (kMulti ? n_of[sg] : 1) * group;
            left.head = hh;
        }
        p.pieces[blockIdx.x] = left;
    }
    if (!kMulti) {   // rows of empty sequences
        for (int e = blockIdx.x; e < S; e += gridDim.x)
            if (lens[e] == 0)
                for (int i = tid; i < a.num_q_heads * kHeadDim / 8; i += M::kThreads)
                    reinterpret_cast<uint4*>(a.out)[(size_t)e * a.num_q_heads * kHeadDim / 8 + i] = make_uint4(0, 0, 0, 0);
    }
}

// Joins the segments cut between CTAs: CTA (c, .) takes the segment whose head is CTA c's last piece; the
// pieces that follow are the first ones of the next CTAs, up to the one that ends it.  A row goes to `split`
// warps (1, 2, 4 or 8), which share its pieces.  Few registers, so that its CTAs are already resident
// beside the attention's and only wait for its end.
constexpr int kJoinWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kJoinWarps * 32, 5) q8_join_kernel(const Q8Launch p, int ctas, int split) {
    const DecodeQ8Args& a = p.a;
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
    if (have) store_row4<T>(a.out, row_at(p, head.row0, head.head, r) + lane * 4, l, acc);
}

inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

long long units_bound(int block_size, int max_blocks, int rows) {   // of one segment
    return ((long long)max_blocks * block_size + kTile - 1) / kTile + start_units((rows + 7) / 8 * 8);
}

// Sequences of one launch: their lengths fit on chip, and the units of a kv head in 31 bits.
int slice_of(int num_seqs, int block_size, int max_blocks, int rows) {
    return (int)max(1LL, min((long long)min(num_seqs, kQ8MaxSeqs), 0x7fffffffLL / units_bound(block_size, max_blocks, rows)));
}

long long line_bound(int num_seqs, int num_kv_heads, int block_size, int max_blocks, int rows) {
    return slice_of(num_seqs, block_size, max_blocks, rows) * num_kv_heads * units_bound(block_size, max_blocks, rows);
}

struct Q8Grid {
    int ctas, warps;
};

// One CTA per SM, fewer for little work: a cut between CTAs costs the joining launch (2.5 us), so at the longest
// contexts the tables allow one CTA takes up to eight units a warp alone, and several take four at least.
Q8Grid q8_grid(int num_seqs, int num_kv_heads, int block_size, int max_blocks, int rows) {
    const long long units = line_bound(num_seqs, num_kv_heads, block_size, max_blocks, rows);
    const int sms = sm_count_current();
    const int warps = rows <= 8 && (long long)num_seqs * num_kv_heads >= 2LL * kFewWarps * sms ? kManyWarps : kFewWarps;
    if (units <= 8 * warps) return Q8Grid{1, warps};
    return Q8Grid{(int)min((units + 4 * warps - 1) / (4 * warps), (long long)sms), warps};
}

struct Q8Layout {
    size_t firsts, pieces, bytes;
};

Q8Layout q8_layout(const Q8Grid& grid, int rows) {
    Q8Layout w;
    const size_t piece = (size_t)piece_floats(rows) * sizeof(float);
    w.firsts = align256(2 * (size_t)grid.ctas * piece);
    w.pieces = w.firsts + (rows > 16 ? align256((size_t)grid.ctas * grid.warps * piece) : 0);
    w.bytes = w.pieces + align256((size_t)grid.ctas * sizeof(CtaPieces));
    return w;
}

bool encode_q8_map(const void* base, unsigned long long rows, CUtensorMap* out) {
    auto fn = tensor_map_encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)kHeadDim, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)kHeadDim};
    cuuint32_t box[2] = {(cuuint32_t)kHeadDim, (cuuint32_t)kTile};
    cuuint32_t estr[2] = {1u, 1u};
    return fn(out, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T, int NT, int kW, bool kMulti>
cudaError_t launch_nt(const Q8Launch& p, int ctas, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    constexpr size_t smem = 1024 + Q8Smem<NT, kW>::kBytes;
    auto kernel = q8_attend_kernel<T, NT, kW, kMulti>;
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
    e = launch_pdl(kernel, dim3(ctas), dim3(Q8Smem<NT, kW>::kThreads), smem, stream, p, k, v);
    if (e != cudaSuccess || ctas == 1) return e;
    // as many warps to a row as a segment has pieces when all are equally long
    const int pieces = ctas / max(1, min(ctas, p.a.num_seqs * p.a.num_kv_heads));
    const int split = pieces >= 32 ? 8 : pieces >= 16 ? 4 : pieces >= 8 ? 2 : 1;
    const int grid_y = (p.rows * split + kJoinWarps - 1) / kJoinWarps;
    return launch_pdl(q8_join_kernel<T>, dim3(ctas - 1, grid_y), dim3(kJoinWarps * 32), 0, stream, p, ctas, split);
}

template <typename T, bool kMulti>
cudaError_t launch_rows(const Q8Launch& p, const Q8Grid& grid, const CUtensorMap& k, const CUtensorMap& v,
                        cudaStream_t stream) {
    const int ctas = grid.ctas;
    if (grid.warps == kManyWarps) return launch_nt<T, 1, kManyWarps, kMulti>(p, ctas, k, v, stream);
    switch ((p.rows + 7) / 8) {
        case 1: return launch_nt<T, 1, kFewWarps, kMulti>(p, ctas, k, v, stream);
        case 2: return launch_nt<T, 2, kFewWarps, kMulti>(p, ctas, k, v, stream);
        case 3: return launch_nt<T, 3, kFewWarps, kMulti>(p, ctas, k, v, stream);
        default: return launch_nt<T, 4, kFewWarps, kMulti>(p, ctas, k, v, stream);
    }
}

}  // namespace

size_t q8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int max_q, int block_size,
                          int max_blocks_per_seq) {
    if (num_seqs == 0) return 0;
    const int rows = num_q_heads / num_kv_heads * max_q;
    const Q8Grid grid = q8_grid(num_seqs, num_kv_heads, block_size, max_blocks_per_seq, rows);
    return grid.ctas == 1 && rows <= 16 ? 0 : q8_layout(grid, rows).bytes;
}

bool q8_line_fits(int num_seqs, int num_kv_heads, int block_size, int max_blocks_per_seq) {
    const Q8Grid grid = q8_grid(num_seqs, num_kv_heads, block_size, max_blocks_per_seq, kQ8MaxRows);
    return line_bound(num_seqs, num_kv_heads, block_size, max_blocks_per_seq, kQ8MaxRows) / (grid.ctas * kFewWarps) <
           (1LL << 30);
}

cudaError_t launch_decode_q8(const DecodeQ8Args& a, int dtype, void* workspace, cudaStream_t stream) {
    CUtensorMap k, v;
    const unsigned long long pool_rows = (unsigned long long)a.num_blocks * a.num_kv_heads * a.block_size;
    if (!encode_q8_map(a.k_cache, pool_rows, &k)) {
        // a host thread that has made no CUDA call yet has no current context, which the encoding asks for
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess ||
            !encode_q8_map(a.k_cache, pool_rows, &k))
            return cudaErrorInvalidValue;
    }
    if (!encode_q8_map(a.v_cache, pool_rows, &v)) return cudaErrorInvalidValue;
    Q8Launch p;
    p.group = a.num_q_heads / a.num_kv_heads;
    p.group_inv = (65536u + p.group - 1) / p.group;
    p.rows = p.group * a.max_q;
    const Q8Grid grid = q8_grid(a.num_seqs, a.num_kv_heads, a.block_size, a.max_blocks_per_seq, p.rows);
    const Q8Layout w = q8_layout(grid, p.rows);
    char* ws = static_cast<char*>(workspace);
    p.parts = reinterpret_cast<float*>(ws);
    p.firsts = reinterpret_cast<float*>(ws + w.firsts);
    p.pieces = reinterpret_cast<CtaPieces*>(ws + w.pieces);
    // larger batches go in slices, one after another
    const int slice = slice_of(a.num_seqs, a.block_size, a.max_blocks_per_seq, p.rows);
    for (int s0 = 0; s0 < a.num_seqs; s0 += slice) {
        p.a = a;
        p.a.num_seqs = min(slice, a.num_seqs - s0);
        p.a.block_tables += (size_t)s0 * a.max_blocks_per_seq;
        p.a.context_lens += s0;
        if (a.q_start) {
            p.a.q_start += s0;
        } else {
            const size_t rows = (size_t)s0 * a.num_q_heads * kHeadDim;
            p.a.q = static_cast<const uint16_t*>(a.q) + rows;
            p.a.out = static_cast<uint16_t*>(a.out) + rows;
        }
        cudaError_t e;
        if (dtype == PA_BF16)
            e = a.q_start ? launch_rows<__nv_bfloat16, true>(p, grid, k, v, stream)
                          : launch_rows<__nv_bfloat16, false>(p, grid, k, v, stream);
        else
            e = a.q_start ? launch_rows<__half, true>(p, grid, k, v, stream)
                          : launch_rows<__half, false>(p, grid, k, v, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace pa
