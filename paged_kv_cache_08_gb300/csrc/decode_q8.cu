// Attention over the 8-bit paged cache: one query token per sequence, or several attending causally.
//
// What it computes ("显存虚拟化革命：PagedAttention 内存池管理与显存碎片终结", §五.1, over codes and
// exponents): for query row i of sequence s at position p = L - n + i and query head h,
//   out = sum_{t <= p} softmax_t(scale * q . (2^ke K_t)) * 2^ve V_t
// with K_t, V_t the codes of token t and ke, ve its block's exponents.  Tokens of a block whose table
// entry lies outside the pool are left out.
//
// The exponents cost one add each: with x_t = scale log2(e) 2^ke (q . K_t) + ve and a base b,
//   P_t = 2^(x_t - b),  O = sum P_t V_t (codes),  l = sum P_t 2^-ve,  out = O / l,
// so V is never scaled, P_t stays in fp16's range whatever the blocks' scales (the base follows the
// maximum of x_t, not of the score), and b cancels.  Codes become fp16 exactly; P is rounded to fp16
// for the PV product (2^-11 of a weight, averaged over the tokens; fp32 sums).  bf16 queries are scaled
// by a power of two per row into fp16's range (exact down to 2^-29 of the row's largest element).
//
// Work split: a segment is a (sequence, kv head); its 16-token tiles and one unit for its start lie on a
// line, segment after segment, and every warp of the grid takes an equal, contiguous share of the line.
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
// The base moves only when a score exceeds it by 2^8 (then O and l are rescaled), so most tiles need
// no shuffle.  Bound by HBM (one byte per cached element).
#include <type_traits>

#include "decode_common.cuh"
#include "q8.cuh"

namespace pa {

namespace {

constexpr int kQ8Warps = 8;
constexpr int kQ8Threads = kQ8Warps * 32;
constexpr int kTile = 16;                       // tokens per tile
constexpr uint32_t kTileHalf = kTile * kHeadDim;   // 2 KB of K, 2 KB of V
constexpr uint32_t kTileBytes = 2 * kTileHalf;
constexpr int kStartUnits = 1;                  // share of a segment's start and end, in tiles
constexpr int kQ8MaxSeqs = 1024;                // sequences of one launch (their lengths stay on chip)
constexpr float kBaseSlack = 8.f;               // log2: P stays below 2^8

// Floats of a piece of `rows` rows: O, then (base, sum) of each row; a multiple of 16 bytes.
__host__ __device__ constexpr int piece_floats(int rows) { return rows * kHeadDim + (2 * rows + 3) / 4 * 4; }

// Partial results of one CTA for the joining launch.
struct CtaPieces {
    int first;      // slot 0: 0 none, 1 ends here, 2 the whole CTA is inside one segment, 3 no work
    int last;       // slot 1 holds the head of a segment that goes on in the next CTA
    int seq;        // of the head
    int head;
};

struct Q8Launch {
    DecodeQ8Args a;
    float* parts;         // [grid][2] pieces of `rows` rows
    float* firsts;        // [grid * warps] pieces, when they do not fit in shared memory
    CtaPieces* pieces;    // [grid]
    int rows;             // query rows of a segment at most (max_q * group)
};

template <int NT>
struct Q8Smem {
    static constexpr int kRows = NT * 8;
    static constexpr bool kQInSmem = NT >= 3;              // Q fragments (16 registers per 8 rows) leave the registers
    static constexpr bool kFirstInSmem = NT <= 2;
    static constexpr int kStages = NT == 1 ? 5 : 4;
    static constexpr uint32_t kRing = kStages * kTileBytes;  // per warp
    static constexpr uint32_t kOffFirst = kQ8Warps * kRing;
    static constexpr uint32_t kOffLastMl = kOffFirst + (kFirstInSmem ? kQ8Warps * piece_floats(kRows) * 4 : 0);
    static constexpr uint32_t kOffQ = kOffLastMl + kQ8Warps * kRows * 8;
    static constexpr uint32_t kOffP = kOffQ + (kQInSmem ? kQ8Warps * NT * 16 * 32 * 4 : 0);
    static constexpr uint32_t kOffLen = kOffP + (kQ8MaxSeqs + 1) * 8;
    static constexpr uint32_t kOffBar = (kOffLen + kQ8MaxSeqs * 4 + 15) / 16 * 16;
    static constexpr uint32_t kOffDesc = kOffBar + kQ8Warps * kStages * 8;
    static constexpr uint32_t kBytes = kOffDesc + kQ8Warps * 32 + 64;
    static_assert(kRing >= kRows * kHeadDim * 4, "a warp's last piece is kept in its ring");
    static_assert(1024 + kBytes <= 227 * 1024, "shared memory of one CTA");
};

// What a warp leaves for the end of its CTA.
struct WarpPieces {
    int first;       // slot: a piece of a segment begun before the warp's share, ended in it
    int last;        // slot: a piece of a segment that goes on; 2: it also began before
    int empty;       // no units
    int first_seq, first_head, last_seq, last_head;
    int pad;
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
    const float f0 = m == -INFINITY ? 0.f : ex2(m - m2), f1 = ml.x == -INFINITY ? 0.f : ex2(ml.x - m2);
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

// Rows (query token, group member) of a segment.
struct Seg {
    int s, h, L;
    int row0, n;     // first query row, new tokens
    int p0;          // position of the first
};

template <bool kMulti>
__device__ __forceinline__ Seg segment(const DecodeQ8Args& a, int s, int h, int L) {
    Seg g{s, h, L, s, 1, L - 1};
    if (kMulti) {
        const NewRows nr = new_rows(a.q_start, a.q_rows, a.max_q, s, L);
        g.row0 = nr.row0;
        g.n = nr.n;
        g.p0 = L - nr.n;
    }
    return g;
}

__device__ __forceinline__ size_t row_offset(const DecodeQ8Args& a, const Seg& g, int group, int r) {
    return ((size_t)(g.row0 + r / group) * a.num_q_heads + (size_t)g.h * group + r % group) * kHeadDim;
}

// One unit of the line as the lane that owns it sees it.
struct Unit {
    int y;           // pool row of the tile's first token; -1 no tile, -2 block outside the pool
    int t0;          // its position
    int seg;         // s << 16 | h
    int flags;       // 1 the segment's first unit, 2 its last
    int ke, ve;
};

__device__ __forceinline__ Unit unit_at(const DecodeQ8Args& a, const long long* P, const int* lens, long long u,
                                        long long end) {
    Unit x{-1, 0, 0, 0, 0, 0};
    if (u >= end) return x;
    const int Hkv = a.num_kv_heads;
    int lo = 0, hi = a.num_seqs;                  // the last s with Hkv * P[s] <= u
    while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (P[mid] * Hkv <= u) lo = mid;
        else hi = mid;
    }
    const long long w = P[lo + 1] - P[lo], rem = u - P[lo] * Hkv;
    int h, r;
    if (rem <= 0x7fffffffLL) {
        h = (int)((uint32_t)rem / (uint32_t)w);
        r = (int)((uint32_t)rem - (uint32_t)h * (uint32_t)w);
    } else {
        h = (int)(rem / w);
        r = (int)(rem - h * w);
    }
    x.seg = lo << 16 | h;
    x.flags = (r == 0 ? 1 : 0) | (r == w - 1 ? 2 : 0);
    if (r < kStartUnits) return x;
    x.t0 = (r - kStartUnits) * kTile;
    const int B = a.block_size;
    const int id = __ldg(a.block_tables + (size_t)lo * a.max_blocks_per_seq + x.t0 / B);
    if (id < 0 || id >= a.num_blocks) {
        flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
        x.y = -2;
        return x;
    }
    const int tile = id * Hkv + h;                // fits: num_blocks * Hkv * B < 2^31
    x.y = tile * B + x.t0 % B;
    x.ke = a.k_exp[tile];
    x.ve = a.v_exp[tile];
    return x;
}

template <typename T, int NT, bool kMulti>
__global__ void __launch_bounds__(kQ8Threads, 1)
    q8_attend_kernel(const Q8Launch p, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using M = Q8Smem<NT>;
    constexpr int kStages = M::kStages;
    const DecodeQ8Args& a = p.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane / 4, t = lane % 4;
    long long* P = reinterpret_cast<long long*>(smem + M::kOffP);
    int* lens = reinterpret_cast<int*>(smem + M::kOffLen);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + M::kOffBar) + warp * kStages;
    WarpPieces* wp = reinterpret_cast<WarpPieces*>(smem + M::kOffDesc);
    const uint32_t ring = smem_u32(smem) + warp * M::kRing;

    if (lane < kStages) {
        mbar_init(&bars[lane], 1);
        fence_mbar_init();
    }
    if (lane == 0) {
        prefetch_map(&kmap);
        prefetch_map(&vmap);
    }
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- lengths and the line's prefix sums ----
    const int S = a.num_seqs, group = a.num_q_heads / a.num_kv_heads;
    {
        constexpr int kPer = kQ8MaxSeqs / kQ8Threads;
        __shared__ long long warp_sum_of[kQ8Warps];
        long long mine[kPer], sum = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int s = tid * kPer + i;
            long long w = 0;
            if (s < S) {
                bool bad;
                const int L = clamped_len(a.context_lens, s, a.max_blocks_per_seq, a.block_size, &bad);
                int n = 1;
                if (kMulti) {
                    const NewRows nr = new_rows(a.q_start, a.q_rows, a.max_q, s, L);
                    n = nr.n;
                    bad |= nr.bad;
                }
                if (bad && blockIdx.x == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
                lens[s] = L;
                if (L > 0 && n > 0) w = (L + kTile - 1) / kTile + kStartUnits;
            }
            mine[i] = sum;
            sum += w;
        }
        long long incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sum_of[warp] = incl;
        __syncthreads();
        long long before = incl - sum;
        for (int i = 0; i < warp; ++i) before += warp_sum_of[i];
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            if (tid * kPer + i <= S) P[tid * kPer + i] = before + mine[i];
        if (tid == kQ8Threads - 1 && S == kQ8MaxSeqs) P[S] = before + sum;
        __syncthreads();
    }
    if (!kMulti) {   // rows of empty sequences
        for (int s = blockIdx.x; s < S; s += gridDim.x)
            if (lens[s] == 0)
                for (int i = tid; i < a.num_q_heads * kHeadDim / 8; i += kQ8Threads)
                    reinterpret_cast<uint4*>(a.out)[(size_t)s * a.num_q_heads * kHeadDim / 8 + i] = make_uint4(0, 0, 0, 0);
    }

    const long long total = P[S] * a.num_kv_heads;
    const long long shares = (long long)gridDim.x * kQ8Warps, me = (long long)blockIdx.x * kQ8Warps + warp;
    const long long u0 = total / shares * me + total % shares * me / shares;
    const long long u1 = total / shares * (me + 1) + total % shares * (me + 1) / shares;
    const int units = (int)(u1 - u0);

    // ---- per-lane fragment addresses inside a tile (128-byte swizzle: 16-byte unit ^ (row & 7)) ----
    const uint32_t k_off0 = g * 128 + ((uint32_t)((2 * t) ^ g) << 4);
    const uint32_t k_off1 = g * 128 + ((uint32_t)((2 * t + 1) ^ g) << 4);
    const uint32_t v_off0 = kTileHalf + (2 * t) * 128 + ((uint32_t)(g ^ (2 * t)) << 4);
    const uint32_t v_off1 = kTileHalf + (2 * t + 1) * 128 + ((uint32_t)(g ^ (2 * t + 1)) << 4);

    float o[NT][8][4];
    float base[NT][2], sum[NT][2], qf[NT][2];
    int lim[NT][2];
    uint32_t qreg[M::kQInSmem ? 1 : NT][16];
    uint32_t* qsm = reinterpret_cast<uint32_t*>(smem + M::kOffQ) + warp * NT * 16 * 32 + lane;
    Seg seg{0, 0, 0, 0, 0, 0};
    int nrows = 0;
    bool open_start = false, have = false;
    uint32_t phases = 0;
    bool dead = false;
    WarpPieces mine{0, 0, units == 0 ? 1 : 0, 0, 0, 0, 0, 0};

    auto clear_state = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][i][c] = 0.f;
            base[nt][0] = base[nt][1] = -INFINITY;
            sum[nt][0] = sum[nt][1] = 0.f;
        }
    };

    // Q fragments of the segment, their scales, and the positions the rows see.
    auto begin_segment = [&](int s, int h) {
        seg = segment<kMulti>(a, s, h, lens[s]);
        nrows = seg.n * group;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int r = nt * 8 + g;
            uint4 w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = make_uint4(0, 0, 0, 0);
            if (r < nrows) {
                const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.q) +
                                                                  row_offset(a, seg, group, r) + 32 * t);
#pragma unroll
                for (int i = 0; i < 4; ++i) w[i] = __ldg(src + i);
            }
            uint32_t* x = reinterpret_cast<uint32_t*>(w);
            float scale = 1.f;
            if (std::is_same<T, __nv_bfloat16>::value) {
                float amax = 0.f;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = Elem<T>::to_float2(x[i]);
                    amax = fmaxf(amax, fmaxf(finite_abs(f.x), finite_abs(f.y)));
                }
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                // largest element into [2^14, 2^15)
                const int up = max(-126, min(126, 14 - ((__float_as_int(amax) >> 23) - 127)));
                const float mul = exp2_int(up);
                scale = exp2_int(-up);
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const float2 f = Elem<T>::to_float2(x[i]);
                    x[i] = Elem<__half>::pack2(f.x * mul, f.y * mul);
                }
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                if (M::kQInSmem) qsm[(nt * 16 + i) * 32] = x[i];
                else qreg[M::kQInSmem ? 0 : nt][i] = x[i];
            }
            // this lane's score columns are rows 2 t and 2 t + 1
            qf[nt][0] = __shfl_sync(0xffffffffu, scale, (2 * t) * 4) * a.scale_log2;
            qf[nt][1] = __shfl_sync(0xffffffffu, scale, (2 * t + 1) * 4) * a.scale_log2;
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const int col = nt * 8 + 2 * t + c;
                lim[nt][c] = kMulti && col < nrows ? seg.p0 + col / group : seg.L - 1;
            }
        }
        clear_state();
        have = true;
    };

    // Sum over the lanes that share a column.
    auto finish_sums = [&]() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
#pragma unroll
                for (int m = 4; m < 32; m <<= 1) sum[nt][c] += __shfl_xor_sync(0xffffffffu, sum[nt][c], m);
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
                    float* dst = slot + r * kHeadDim;
#pragma unroll
                    for (int i = 0; i < 8; i += 2)
                        *reinterpret_cast<float4*>(dst + g * 16 + 2 * i) =
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
                    uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + row_offset(a, seg, group, r) +
                                                          g * 16);
                    dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
                    dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
    };

    // pieces of warp w: the first in memory of its own, the last in its ring (every copy has landed)
    const int slot_rows = M::kFirstInSmem ? M::kRows : p.rows;
    auto first_of = [&](int w) {
        return M::kFirstInSmem ? reinterpret_cast<float*>(smem + M::kOffFirst) + w * piece_floats(M::kRows)
                               : p.firsts + ((size_t)blockIdx.x * kQ8Warps + w) * piece_floats(p.rows);
    };
    auto last_of = [&](int w) { return reinterpret_cast<float*>(smem + w * M::kRing); };
    auto first_ml_of = [&](int w) { return reinterpret_cast<float2*>(first_of(w) + slot_rows * kHeadDim); };
    auto last_ml_of = [&](int w) { return reinterpret_cast<float2*>(smem + M::kOffLastMl) + w * M::kRows; };

    // ---- the stream ----
    if (units > 0) {
        __syncwarp();
        Unit A = unit_at(a, P, lens, u0 + lane, u1), Bn{-1, 0, 0, 0, 0, 0};
        auto issue = [&](int j, int y) {   // by the lane that owns unit j
            const int st = j % kStages;
            const uint32_t dst = ring + st * kTileBytes;
            mbar_arrive_expect_tx(&bars[st], kTileBytes);
            tma_load_2d(dst, &kmap, 0, y, &bars[st]);
            tma_load_2d(dst + kTileHalf, &vmap, 0, y, &bars[st]);
        };
        if (lane < kStages && A.y >= 0) issue(lane, A.y);
        {   // the share may begin inside a segment
            const int sh = __shfl_sync(0xffffffffu, A.seg, 0), fl = __shfl_sync(0xffffffffu, A.flags, 0);
            open_start = !(fl & 1);
            if (open_start) {
                begin_segment(sh >> 16, sh & 0xffff);
                mine.first_seq = seg.s;
                mine.first_head = seg.h;
            }
        }
        int i = 0;
        for (; i < units; ++i) {
            const int w = i & 31;
            if (w == 0) {
                if (i > 0) A = Bn;
                if (i + 32 < units) Bn = unit_at(a, P, lens, u0 + i + 32 + lane, u1);
            }
            const int y = __shfl_sync(0xffffffffu, A.y, w), flags = __shfl_sync(0xffffffffu, A.flags, w);
            if (flags & 1) {
                const int sh = __shfl_sync(0xffffffffu, A.seg, w);
                begin_segment(sh >> 16, sh & 0xffff);
            }
            if (y >= 0) {
                const int t0 = __shfl_sync(0xffffffffu, A.t0, w);
                const int ke = clamp_exp(__shfl_sync(0xffffffffu, A.ke, w)), ve = clamp_exp(__shfl_sync(0xffffffffu, A.ve, w));
                const int st = i % kStages;
                if (!mbar_wait_bounded(&bars[st], (phases >> st) & 1)) {
                    flag_status(a.status, PA_DEV_TIMEOUT);
                    dead = true;
                }
                dead = __any_sync(0xffffffffu, dead);
                if (dead) break;
                phases ^= 1u << st;
                const uint32_t tile = ring + st * kTileBytes;

                // S = K Q^T
                float x[NT][4];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) x[nt][0] = x[nt][1] = x[nt][2] = x[nt][3] = 0.f;
                {
                    const uint4 k0 = lds128(tile + k_off0), k1 = lds128(tile + k_off1);
                    const uint4 k2 = lds128(tile + k_off0 + 1024), k3 = lds128(tile + k_off1 + 1024);
                    const uint32_t ka[8] = {k0.x, k0.y, k0.z, k0.w, k1.x, k1.y, k1.z, k1.w};
                    const uint32_t kb[8] = {k2.x, k2.y, k2.z, k2.w, k3.x, k3.y, k3.z, k3.w};
#pragma unroll
                    for (int s = 0; s < 8; ++s) {
                        const uint32_t a0 = lo_f16x2(ka[s]), a1 = lo_f16x2(kb[s]), a2 = hi_f16x2(ka[s]),
                                       a3 = hi_f16x2(kb[s]);
#pragma unroll
                        for (int nt = 0; nt < NT; ++nt) {
                            const uint32_t b0 = M::kQInSmem ? qsm[(nt * 16 + 2 * s) * 32] : qreg[M::kQInSmem ? 0 : nt][2 * s];
                            const uint32_t b1 =
                                M::kQInSmem ? qsm[(nt * 16 + 2 * s + 1) * 32] : qreg[M::kQInSmem ? 0 : nt][2 * s + 1];
                            mma16816<__half>(x[nt], a0, a1, a2, a3, b0, b1);
                        }
                    }
                }
                uint4 v0 = lds128(tile + v_off0), v1 = lds128(tile + v_off1);
                uint4 v2 = lds128(tile + v_off0 + 1024), v3 = lds128(tile + v_off1 + 1024);

                // x = score in log2 units + ve; positions a row does not see to -inf
                const float ks = exp2_int(ke), vef = (float)ve, unscale = exp2_int(-ve);
                const bool masked = t0 + kTile > seg.p0 + 1;
                bool nan_v = false;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 4; ++c) x[nt][c] = fmaf(x[nt][c], qf[nt][c & 1] * ks, vef);
                if (masked) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 4; ++c)
                            if (t0 + g + (c >> 1) * 8 > lim[nt][c & 1]) x[nt][c] = -INFINITY;
                    // rows behind the last token hold anything: zero codes
                    const int left = seg.L - t0;
                    if (2 * t >= left) v0 = make_uint4(0, 0, 0, 0);
                    if (2 * t + 1 >= left) v1 = make_uint4(0, 0, 0, 0);
                    if (2 * t + 8 >= left) v2 = make_uint4(0, 0, 0, 0);
                    if (2 * t + 9 >= left) v3 = make_uint4(0, 0, 0, 0);
                    if (kMulti) {
                        // a NaN of a token that some rows do not see must not reach them through 0 * NaN
                        auto nans = [](uint32_t w) { return __vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu); };
                        auto any4 = [&](const uint4& v) { return nans(v.x) | nans(v.y) | nans(v.z) | nans(v.w); };
                        nan_v = __any_sync(0xffffffffu, (any4(v0) | any4(v1) | any4(v2) | any4(v3)) != 0);
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
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        move |= fmaxf(x[nt][c], x[nt][c + 2]) > base[nt][c] + kBaseSlack;
                if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            float m = fmaxf(x[nt][c], x[nt][c + 2]);
#pragma unroll
                            for (int k = 4; k < 32; k <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, k));
                            m = fmaxf(m, base[nt][c]);
                            const float f = base[nt][c] == -INFINITY ? 0.f : ex2(base[nt][c] - m);
                            base[nt][c] = m;
                            sum[nt][c] *= f;
#pragma unroll
                            for (int k = 0; k < 8; ++k) {
                                o[nt][k][c] *= f;
                                o[nt][k][c + 2] *= f;
                            }
                        }
                }
                uint32_t b0[NT], b1[NT];
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    float pr[4];
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        pr[c] = ex2(x[nt][c] - base[nt][c & 1]);
                        if (masked && t0 + g + (c >> 1) * 8 > lim[nt][c & 1]) pr[c] = 0.f;
                    }
                    sum[nt][0] = fmaf(pr[0] + pr[2], unscale, sum[nt][0]);
                    sum[nt][1] = fmaf(pr[1] + pr[3], unscale, sum[nt][1]);
                    b0[nt] = movmatrix_trans(Elem<__half>::pack2(pr[0], pr[1]));
                    b1[nt] = movmatrix_trans(Elem<__half>::pack2(pr[2], pr[3]));
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
                        for (int nt = 0; nt < NT; ++nt) mma16816<__half>(o[nt][2 * q + e], a0, a1, a2, a3, b0[nt], b1[nt]);
                    }
                }
                if (kMulti && nan_v) {
                    // rare: NaN into the dims and rows that see such a token
                    for (int j = 0; j < min(kTile, seg.L - t0); ++j) {
                        const uint4 v = lds128(tile + kTileHalf + j * 128 + ((uint32_t)(g ^ (j & 7)) << 4));
                        const uint32_t vw[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int d = 0; d < 16; ++d)
                            if (((vw[d / 4] >> (8 * (d % 4))) & 0x7f) == 0x7f)
#pragma unroll
                                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                                    for (int c = 0; c < 2; ++c)
                                        if (t0 + j <= lim[nt][c]) o[nt][d / 2][c + 2 * (d % 2)] = __int_as_float(0x7fffffff);
                    }
                }
            }
            // every lane has the tile in registers: its stage takes the unit kStages further on
            __syncwarp();
            const int j = i + kStages;
            if (j < units && lane == (j & 31)) {
                const int yj = (j >> 5) == (i >> 5) ? A.y : Bn.y;
                if (yj >= 0) issue(j, yj);
            }
            if (flags & 2) {
                if (open_start) {
                    store_piece(first_of(warp), first_ml_of(warp));
                    mine.first = 1;
                } else {
                    store_out();
                }
                open_start = false;
                have = false;
            }
        }
        if (dead) {   // let the copies in flight land (again with a limit) before the CTA's memory is given up
            for (int j = i; j < min(units, i + kStages); ++j) {
                const int yj = __shfl_sync(0xffffffffu, (j >> 5) == (i >> 5) ? A.y : Bn.y, j & 31);
                if (yj >= 0) mbar_wait_bounded(&bars[j % kStages], (phases >> (j % kStages)) & 1);
            }
            have = false;
            __syncwarp();
        }
        if (have) {
            store_piece(last_of(warp), last_ml_of(warp));
            mine.last = open_start ? 2 : 1;
            mine.last_seq = seg.s;
            mine.last_head = seg.h;
        }
    }
    if (lane == 0) wp[warp] = mine;
    __syncthreads();

    // ---- join the pieces of cut segments ----
    // Warps in order: a first piece ends the chain that is open (or one from before this CTA), a last
    // piece goes on with it (2) or opens one (1).  Of a chain ws .. we, warp we gives its first piece if
    // the chain ends there, every other warp its last.
    CtaPieces left{3, 0, 0, 0};
    auto join = [&](int ws, int we, bool before, bool closed, int s, int h) {
        const Seg sg = segment<kMulti>(a, s, h, lens[s]);
        float* to = p.parts + ((size_t)blockIdx.x * 2 + (before ? 0 : 1)) * piece_floats(p.rows);
        for (int e = tid; e < sg.n * group * 32; e += kQ8Threads) {
            const int r = e / 32, d = e % 32 * 4;
            float m = -INFINITY, l = 0.f;
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int w = ws; w <= we; ++w) {
                if (wp[w].empty) continue;
                const bool first = closed && w == we;
                add_piece(m, l, acc, (first ? first_ml_of(w) : last_ml_of(w))[r],
                          *reinterpret_cast<const float4*>((first ? first_of(w) : last_of(w)) + r * kHeadDim + d));
            }
            if (closed && !before) {
                store_row4<T>(a.out, row_offset(a, sg, group, r) + d, l, acc);
            } else {
                *reinterpret_cast<float4*>(to + r * kHeadDim + d) = acc;
                if (d == 0) reinterpret_cast<float2*>(to + p.rows * kHeadDim)[r] = make_float2(m, l);
            }
        }
        if (before) {
            left.first = closed ? 1 : 2;
        } else if (!closed) {
            left.last = 1;
            left.seq = s;
            left.head = h;
        }
    };
    int ws = -1;
    bool before = false;
    for (int w = 0; w < kQ8Warps; ++w) {
        const WarpPieces x = wp[w];
        if (x.empty) continue;
        if (left.first == 3) left.first = 0;
        if ((x.first || x.last == 2) && ws < 0) {
            ws = w;
            before = true;
        }
        if (x.first) {
            join(ws, w, before, true, x.first_seq, x.first_head);
            ws = -1;
        }
        if (x.last == 1) {
            ws = w;
            before = false;
        }
    }
    if (ws >= 0) join(ws, kQ8Warps - 1, before, false, wp[ws].last_seq, wp[ws].last_head);
    if (tid == 0 && gridDim.x > 1) p.pieces[blockIdx.x] = left;
}

// Joins a segment cut between CTAs: CTA (c, r) takes row r of the segment whose head is CTA c's last
// piece; the pieces that follow are the first ones of the next CTAs, up to the one that ends it.
constexpr int kJoinWarps = 4;

template <typename T, bool kMulti>
__global__ void __launch_bounds__(kJoinWarps * 32) q8_join_kernel(const Q8Launch p, int ctas) {
    const DecodeQ8Args& a = p.a;
    __shared__ int end_of;
    __shared__ float4 acc_of[kJoinWarps][32];
    __shared__ float2 ml_of[kJoinWarps];
    grid_dependency_wait();
    grid_launch_dependents();
    const int c = blockIdx.x, r = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const CtaPieces head = p.pieces[c];
    if (!head.last) return;
    bool bad;
    const int L = clamped_len(a.context_lens, head.seq, a.max_blocks_per_seq, a.block_size, &bad);
    const Seg sg = segment<kMulti>(a, head.seq, head.head, L);
    const int group = a.num_q_heads / a.num_kv_heads;
    if (r >= sg.n * group) return;
    if (threadIdx.x == 0) end_of = ctas - 1;
    __syncthreads();
    for (int i = c + 1 + threadIdx.x; i < ctas; i += kJoinWarps * 32)
        if (p.pieces[i].first < 2) atomicMin(&end_of, i);
    __syncthreads();
    const int end = end_of;
    float m = -INFINITY, l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    constexpr int kBatch = 8;
    for (int i0 = c + warp; i0 <= end; i0 += kJoinWarps * kBatch) {
        float2 ml[kBatch];
        float4 v[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = i0 + k * kJoinWarps;
            ml[k] = make_float2(-INFINITY, 0.f);
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (i <= end && (i == c || p.pieces[i].first != 3)) {
                const float* piece = p.parts + ((size_t)i * 2 + (i == c ? 1 : 0)) * piece_floats(p.rows);
                ml[k] = reinterpret_cast<const float2*>(piece + p.rows * kHeadDim)[r];
                v[k] = *reinterpret_cast<const float4*>(piece + r * kHeadDim + lane * 4);
            }
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) add_piece(m, l, acc, ml[k], v[k]);
    }
    acc_of[warp][lane] = acc;
    if (lane == 0) ml_of[warp] = make_float2(m, l);
    __syncthreads();
    if (warp > 0) return;
    for (int w = 1; w < kJoinWarps; ++w) add_piece(m, l, acc, ml_of[w], acc_of[w][lane]);
    store_row4<T>(a.out, row_offset(a, sg, group, r) + lane * 4, l, acc);
}

inline size_t align256(size_t n) { return (n + 255) & ~size_t(255); }

long long line_bound(int num_seqs, int num_kv_heads, int block_size, int max_blocks) {
    const long long tiles = ((long long)max_blocks * block_size + kTile - 1) / kTile;
    return (long long)min(num_seqs, kQ8MaxSeqs) * num_kv_heads * (tiles + kStartUnits);
}

// One CTA per SM, fewer for little work: a cut between CTAs costs the joining launch, so a CTA's share
// is at least four tiles a warp of the longest contexts the tables allow.
int q8_ctas(int num_seqs, int num_kv_heads, int block_size, int max_blocks) {
    const long long want = (line_bound(num_seqs, num_kv_heads, block_size, max_blocks) + 4 * kQ8Warps - 1) / (4 * kQ8Warps);
    return (int)max(1LL, min(want, (long long)sm_count_current()));
}

struct Q8Layout {
    size_t firsts, pieces, bytes;
};

Q8Layout q8_layout(int ctas, int rows) {
    Q8Layout w;
    const size_t piece = (size_t)piece_floats(rows) * sizeof(float);
    w.firsts = align256(2 * ctas * piece);
    w.pieces = w.firsts + (rows > 16 ? align256((size_t)ctas * kQ8Warps * piece) : 0);
    w.bytes = w.pieces + align256(ctas * sizeof(CtaPieces));
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

template <typename T, int NT, bool kMulti>
cudaError_t launch_nt(const Q8Launch& p, int ctas, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    constexpr size_t smem = 1024 + Q8Smem<NT>::kBytes;
    auto kernel = q8_attend_kernel<T, NT, kMulti>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(kernel, dim3(ctas), dim3(kQ8Threads), smem, stream, p, k, v);
    if (e != cudaSuccess || ctas == 1) return e;
    return launch_pdl(q8_join_kernel<T, kMulti>, dim3(ctas - 1, p.rows), dim3(kJoinWarps * 32), 0, stream, p, ctas);
}

template <typename T, bool kMulti>
cudaError_t launch_rows(const Q8Launch& p, int ctas, const CUtensorMap& k, const CUtensorMap& v, cudaStream_t stream) {
    switch ((p.rows + 7) / 8) {
        case 1: return launch_nt<T, 1, kMulti>(p, ctas, k, v, stream);
        case 2: return launch_nt<T, 2, kMulti>(p, ctas, k, v, stream);
        case 3: return launch_nt<T, 3, kMulti>(p, ctas, k, v, stream);
        default: return launch_nt<T, 4, kMulti>(p, ctas, k, v, stream);
    }
}

}  // namespace

size_t q8_workspace_bytes(int num_seqs, int num_q_heads, int num_kv_heads, int max_q, int block_size,
                          int max_blocks_per_seq) {
    if (num_seqs == 0) return 0;
    const int ctas = q8_ctas(num_seqs, num_kv_heads, block_size, max_blocks_per_seq);
    const int rows = num_q_heads / num_kv_heads * max_q;
    return ctas == 1 && rows <= 16 ? 0 : q8_layout(ctas, rows).bytes;
}

bool q8_line_fits(int num_seqs, int num_kv_heads, int block_size, int max_blocks_per_seq) {
    const int ctas = q8_ctas(num_seqs, num_kv_heads, block_size, max_blocks_per_seq);
    return line_bound(num_seqs, num_kv_heads, block_size, max_blocks_per_seq) / (ctas * kQ8Warps) < (1LL << 30);
}

cudaError_t launch_decode_q8(const DecodeQ8Args& a, int dtype, void* workspace, cudaStream_t stream) {
    CUtensorMap k, v;
    const unsigned long long pool_rows = (unsigned long long)a.num_blocks * a.num_kv_heads * a.block_size;
    if (!encode_q8_map(a.k_cache, pool_rows, &k) || !encode_q8_map(a.v_cache, pool_rows, &v))
        return cudaErrorInvalidValue;
    Q8Launch p;
    p.rows = a.num_q_heads / a.num_kv_heads * a.max_q;
    const int ctas = q8_ctas(a.num_seqs, a.num_kv_heads, a.block_size, a.max_blocks_per_seq);
    const Q8Layout w = q8_layout(ctas, p.rows);
    char* ws = static_cast<char*>(workspace);
    p.parts = reinterpret_cast<float*>(ws);
    p.firsts = reinterpret_cast<float*>(ws + w.firsts);
    p.pieces = reinterpret_cast<CtaPieces*>(ws + w.pieces);
    // lengths of kQ8MaxSeqs sequences fit on chip: larger batches go in slices, one after another
    for (int s0 = 0; s0 < a.num_seqs; s0 += kQ8MaxSeqs) {
        p.a = a;
        p.a.num_seqs = min(kQ8MaxSeqs, a.num_seqs - s0);
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
            e = a.q_start ? launch_rows<__nv_bfloat16, true>(p, ctas, k, v, stream)
                          : launch_rows<__nv_bfloat16, false>(p, ctas, k, v, stream);
        else
            e = a.q_start ? launch_rows<__half, true>(p, ctas, k, v, stream)
                          : launch_rows<__half, false>(p, ctas, k, v, stream);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace pa
