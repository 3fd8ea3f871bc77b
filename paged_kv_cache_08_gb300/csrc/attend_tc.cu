// Attention of many query rows on the fifth-generation tensor cores: chunks of new tokens with capped, biased and masked
// scores, and the part of a batch's attention that reads a shared prefix.
//
// What it computes: attend.cuh, by the running-maximum softmax of "显存虚拟化革命：PagedAttention 内存池管理与显存碎片终结",
// §五.1, in log2 units: x = log2(e) z, O = sum 2^(x_t - b) V_t, l = sum 2^(x_t - b), out = O / l.
//
// A unit is what reads one list of blocks: a sequence, or a group of sequences that share a prefix, whose query rows
// then stand side by side in the tiles, so that the prefix passes through the tensor cores once for all of them.  A CTA
// takes 256 query rows of a unit and kv head (two tiles of 128) and a part of the keys that any of them sees; rows
// r = i * G + g (token i, group member g).  Where rows alone do not fill the GPU, the keys are split into `splits` parts
// and the pieces joined by a second launch.
//   warps 0-3, 4-7  softmax of tile 0, tile 1: a thread owns a row (tensor-memory lane)
//   warp 8          copies of 64-token K and V stages into a ring of four
//   warps 9, 10     products of tile 0, tile 1: S = Q K^T, O += P V (P in tensor memory), issued by one lane each
//   warp 11         makes a stage's V fit for products with weights of zero (below)
// Tensor memory and the order of its buffers are those of prefill_tc.cu.
//
// Masks: every row has an interval of keys.  Stages that no row of the CTA sees are not read, a tile passes over those
// that none of its rows sees, and where every row of a warp sees a whole stage there is nothing to mask.  A masked weight
// is zero, and 0 * V is not where V holds an infinity or a NaN (a token of another document, a slot behind the context):
// warp 11 looks through V in stages that some row does not see whole and puts zero in such places and in rows of blocks
// outside the pool; a row that does see a non-finite value takes it at its end, from memory.
//
// Caps: tanh is a polynomial on the FMA units for scores within 3/4 of the cap, else 1 - 2 / (1 + e^2y) on the
// special-function unit, which the softmax's own exponentials already fill.
// P is rounded to fp16, or taken as a high and a low bf16 part (two products): 8 bits of a weight would be the largest error
// of the result.
//
// What bounds it: a CTA's stage of 64 tokens (two tiles) takes about 2050 cycles in fp16 without options, of which its
// products need 1024 (bf16 1536, for P's two parts) and the shared memory that feeds them about 1540 (Q is read again for
// every 64 keys, K and V by both tiles); the rest is the softmax's chain, two warps a scheduler.  A cap adds seven packed
// operations to every pair of scores, a bias by distance one and the groups' offsets.  16 sequences with 512 new of 4096
// tokens, 32 heads: 465 us in fp16 without options (1.11 PFLOP/s), 590 in bf16, 609 with a cap, 304 for packed documents of
// 2048 tokens with one; prompts of 1025 to 2048 tokens behind an image, 32 heads in bf16 with a bias: 286 us.  A CTA's start
// and end take 6 us (unit and intervals, Q, first copies, 64 to 128 KB of results at what one SM stores).
#include <atomic>

#include "attend.cuh"
#include "tc_common.cuh"

namespace pa {

namespace {

constexpr int kTRows = 128;
constexpr int kTiles = 2;
constexpr int kCtaRows = kTiles * kTRows;
constexpr int kTileWarps = 4;                                // softmax warps of a tile: a thread owns a row
constexpr int kSoftWarps = kTileWarps * kTiles;
constexpr int kProdWarp = kSoftWarps;
constexpr int kMmaWarp = kSoftWarps + 1;
constexpr int kCheckWarp = kMmaWarp + kTiles;
constexpr int kTThreads = (kCheckWarp + 1) * 32;
constexpr uint32_t kQHalf = kTRows * 128;                    // 128 rows x 64 dims
constexpr uint32_t kQTile = 2 * kQHalf;
constexpr uint32_t kKVHalf = kStageTokens * 128;             // 64 tokens x 64 dims
constexpr uint32_t kKBytes = 2 * kKVHalf;
constexpr uint32_t kStage = 2 * kKBytes;
constexpr int kTStages = 4;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffRing = kTiles * kQTile;
constexpr int kNumBars = 3 * kTStages + 12 + kTiles + 1;
constexpr uint32_t kOffBar = kOffRing + kTStages * kStage;
constexpr uint32_t kOffValid = kOffBar + kNumBars * 8;       // [stage] the tokens whose rows a copy brings
constexpr uint32_t kOffMisc = kOffValid + kTStages * 8;
constexpr uint32_t kMiscInts = 40;
constexpr size_t kSmem = 1024 + kOffMisc + kMiscInts * 4;
static_assert(kSmem <= 227 * 1024, "one CTA's shared memory must fit in 227 KB");
constexpr uint32_t kTmemCols = 512;                          // per tile: S at +0, P at +64, O at +128
constexpr uint32_t kTileCols = 256;
constexpr uint32_t kColP = 64, kColO = 128;                  // P: fp16 two buffers in turn, bf16 the high and the low part
// log2 of P: a new base puts the largest at 2^top_new, and moves when one would exceed 2^top_most.  fp16: weights keep 11
// bits down to 2^-21 of the row's largest and steps of 2^-31 of it below.  bf16 has fp32's range, and O = sum P V must stay
// in it, too: weights up to 2^8 leave room for |V| up to 2^118, and from 2^-40 on for |V| down to 2^-80.  (A move costs about
// 1000 cycles, for it waits for the tile's products; with 2^8 between the two one stage in four of a warp moved, scores of
// standard deviation 4, and a steep bias moves the base every few stages: prompts with one 290 us with 2^24, 280 with 2^48.)
template <typename T>
__host__ __device__ constexpr float top_new() { return std::is_same<T, __half>::value ? 7.f : -40.f; }
template <typename T>
__host__ __device__ constexpr float top_most() { return std::is_same<T, __half>::value ? 15.9f : 8.f; }
// Scores (in log2 units) beyond which a stage's are rounded before the base is taken from them: from about 2^28 on the
// rounding of a maximum alone, which the exponents' FMA does not share, would put weights out of fp16's range.
constexpr float kLargeScore = 0x1p18f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint32_t kAll = 0xffffffffu;

struct Maps {
    CUtensorMap k, v;
};

struct TcLaunch {
    AttendArgs a;
    int keys;        // AttendKeys
    int units;       // sequences, or groups
    int splits;
    int slot0;
    int R_log2;      // log2 of a box's rows
};

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
    return v;
}

__device__ __forceinline__ float lds32(uint32_t addr) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts32(uint32_t addr, float v) {
    asm volatile("st.shared.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ uint16_t lds16(uint32_t addr) {
    uint16_t v;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t addr, uint16_t v) {
    asm volatile("st.shared.u16 [%0], %1;" ::"r"(addr), "h"(v) : "memory");
}

// Halves of w whose exponent is all ones, as 0x8000 each.
template <typename T>
__device__ __forceinline__ uint32_t non_finite(uint32_t w) {
    constexpr uint32_t kExp = std::is_same<T, __half>::value ? 0x7c007c00u : 0x7f807f80u;
    constexpr uint32_t kOne = std::is_same<T, __half>::value ? 0x04000400u : 0x00800080u;
    return ((w & kExp) + kOne) & 0x80008000u;
}

// The larger magnitudes of two pairs, NaN where either is.
template <typename T>
__device__ __forceinline__ uint32_t max_abs2(uint32_t a, uint32_t b) {
    using T2 = typename std::conditional<std::is_same<T, __half>::value, __half2, __nv_bfloat162>::type;
    const T2 m = __hmax2_nan(*reinterpret_cast<T2*>(&a), __habs2(*reinterpret_cast<T2*>(&b)));
    return *reinterpret_cast<const uint32_t*>(&m);
}

// mbarriers by shared-memory address (32 bits: the softmax has no registers to spare).
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void bar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}
// false if phase `parity` has not completed after about kWaitLimitNs.  (The global timer takes some hundred cycles to read:
// not before many tries have failed.)
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity) {
    unsigned long long t0 = 0;
    for (uint32_t i = 1; !bar_try(bar, parity); ++i) {
        if ((i & 255u) == 0) {
            const unsigned long long now = global_timer_ns();
            if (t0 == 0) t0 = now;
            else if (now - t0 > kWaitLimitNs) return false;
        }
    }
    return true;
}
// Arrive once every tcgen05 operation this thread has issued so far is complete.
__device__ __forceinline__ void bar_commit(uint32_t bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_load(uint32_t dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], "
        "[%4];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// One lane of a converged warp, the same at every call.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}" : "=r"(p));
    return p != 0;
}

// The query tokens of unit u: rows row0 .. row0+n-1 of q, and for a sequence its length.
struct Unit {
    int row0, n, L;
    bool bad;
};

__device__ __forceinline__ Unit unit_of(const TcLaunch& p, int u) {
    const AttendArgs& a = p.a;
    if (p.keys == kPrefixKeys) {
        const int b = a.group_start[u], e = a.group_start[u + 1];
        const int s0 = max(0, min(b, a.num_seqs)), s1 = max(s0, min(e, a.num_seqs));
        const int len = a.prefix_lens[u];
        Unit x{s0, s1 - s0, 0, b != s0 || e != s1 || len < 0 || len > a.max_prefix_blocks * a.block_size};
        if (a.q_start && s1 > s0) {
            x.row0 = max(0, min(a.q_start[s0], a.q_rows));
            x.n = max(0, min(a.q_start[s1], a.q_rows) - x.row0);
        }
        return x;
    }
    bool bad;
    const int L = clamped_len(a.context_lens, u, a.max_blocks_per_seq, a.block_size, &bad);
    const NewRows r = rows_of(a, u, L);
    return Unit{r.row0, r.n, L, bad || r.bad};
}

template <typename T, bool kCap, bool kBias>
__global__ void __launch_bounds__(kTThreads, 1)
    attend_tc_kernel(const TcLaunch p, const __grid_constant__ Maps maps) {
    constexpr bool kSplitP = std::is_same<T, __nv_bfloat16>::value;
    extern __shared__ unsigned char smem_raw[];
    const AttendArgs& a = p.a;
    const uint32_t raw = smem_u32(smem_raw);
    const uint32_t base = (raw + 1023u) & ~1023u;
    unsigned char* bp = smem_raw + (base - raw);
    // mbarriers, by shared-memory address
    const uint32_t kv_full = base + kOffBar;             // [stage] K and V landed
    const uint32_t kv_empty = kv_full + kTStages * 8;    // [stage] the products reading it are done
    const uint32_t v_ready = kv_empty + kTStages * 8;    // [stage] its V has been looked through
    const uint32_t s_full = v_ready + kTStages * 8;      // [tile] S is in tensor memory
    const uint32_t s_free = s_full + 16;                 // [tile] the softmax holds S in registers
    const uint32_t p_full = s_free + 16;                 // [tile][2] P is in tensor memory
    const uint32_t pv_done = p_full + 32;                // [tile][2] O += P V is complete
    const uint32_t q_ready = pv_done + 32;               // [tile]
    const uint32_t drain = q_ready + kTiles * 8;
    volatile uint64_t* valid = reinterpret_cast<volatile uint64_t*>(bp + kOffValid);
    int* misc = reinterpret_cast<int*>(bp + kOffMisc);
    volatile uint32_t* tslot = reinterpret_cast<volatile uint32_t*>(misc);
    volatile int* abort_flag = misc + 1;
    volatile int* issued_count = misc + 2;
    int* found_unit = misc + 3;                  // unit and tile pair of this CTA
    int* found_pair = misc + 4;
    volatile int* bad_first = misc + 5;          // stages in which a V value was not finite: first and last
    volatile int* bad_last = misc + 6;
    int* lo_max = misc + 7;                      // over the CTA's rows that see any key: the intervals' extremes
    int* hi_min = misc + 8;
    int* lo_min = misc + 9;                      // [tile]
    int* hi_max = misc + 11;                     // [tile]
    int* warp_sum = misc + 16;                   // [kTThreads / 32]

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int item = blockIdx.x / p.splits, split = blockIdx.x - item * p.splits, hk = blockIdx.y;
    const int G = a.num_q_heads / a.num_kv_heads;

    // tensor memory, while the loads below are on their way; freed on every path
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(
                         const_cast<uint32_t*>(tslot))),
                     "n"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    auto free_tmem = [&]() {   // after a barrier of the CTA
        if (warp == kMmaWarp) {
            tc_fence_after();
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(*tslot), "n"(kTmemCols) : "memory");
        }
    };
    if (tid == 0) {
        prefetch_map(&maps.k);
        prefetch_map(&maps.v);
    }
    grid_dependency_wait();
    grid_launch_dependents();
    // ---- this CTA's unit and rows: the item-th pair of tiles of all units' ----
    if (tid == 0) *found_unit = -1;
    for (int u0 = 0, before = 0; u0 < p.units; u0 += kTThreads) {
        const int u = u0 + tid;
        int pairs = 0;
        if (u < p.units) {
            const Unit x = unit_of(p, u);
            if (x.bad && blockIdx.x == 0 && hk == 0) flag_status(a.status, PA_DEV_BAD_CONTEXT);
            pairs = (int)(((long long)x.n * G + kCtaRows - 1) / kCtaRows);
        }
        int incl = pairs;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(kAll, incl, o);
            if (lane >= o) incl += v;
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        int mine = before + incl - pairs;
#pragma unroll
        for (int w = 0; w < kTThreads / 32; ++w) {
            const int x = warp_sum[w];
            if (w < warp) mine += x;
            before += x;
        }
        if (item >= mine && item < mine + pairs) {
            *found_unit = u;
            *found_pair = item - mine;
        }
        __syncthreads();
        // (CTA 0 of the first kv head goes on through all units, whose faults it reports)
        if (before > item && !(blockIdx.x == 0 && hk == 0)) break;
    }
    if (tid == 0) {
        *lo_max = 0;
        *hi_min = INT_MAX;
        lo_min[0] = lo_min[1] = INT_MAX;
        hi_max[0] = hi_max[1] = 0;
        *bad_first = INT_MAX;
        *bad_last = -1;
        *abort_flag = 0;
        *issued_count = 0;
    }
    tc_fence_before();
    __syncthreads();
    const int unit = *found_unit;
    if (unit < 0) {
        free_tmem();
        return;
    }
    const Unit un = unit_of(p, unit);
    const int r0 = *found_pair * kCtaRows, rows = un.n * G;
    const int ntiles = min(kTiles, (rows - r0 + kTRows - 1) / kTRows);
    if (tid == kProdWarp * 32) {
        for (int i = 0; i < kTStages; ++i) {
            bar_init(kv_full + i * 8, 1);
            bar_init(kv_empty + i * 8, ntiles);
            bar_init(v_ready + i * 8, 1);
        }
        for (int b = 0; b < 2 * kTiles; ++b) {
            if (b < kTiles) {
                bar_init(s_full + b * 8, 1);
                bar_init(s_free + b * 8, kTileWarps);
                bar_init(q_ready + b * 8, kTileWarps);
            }
            bar_init(p_full + b * 8, kTileWarps);
            bar_init(pv_done + b * 8, 1);
        }
        bar_init(drain, ntiles);
        fence_mbar_init();
    }
    const int32_t* table_row = p.keys == kPrefixKeys ? a.prefix_tables + (size_t)unit * a.max_prefix_blocks
                                                     : a.block_tables + (size_t)unit * a.max_blocks_per_seq;

    // ---- the row of a softmax thread: where it lies, its position, and the keys lo .. hi-1 that it sees ----
    const int st = warp / kTileWarps, wt = (warp & 3) * 32 + lane;
    const int r = r0 + st * kTRows + wt;
    bool row_ok = warp < kSoftWarps && r < rows;
    int lo = 0, hi = INT_MAX, pos = 0;
    int row_at = 0;                                  // row of [T * Hq]
    float slope = 0.f;
    if (row_ok) {
        const int tok = un.row0 + r / G, head = hk * G + r % G;
        row_at = tok * a.num_q_heads + head;
        if (p.keys == kPrefixKeys) {
            int s = tok;
            if (a.q_start) {   // the last sequence of the group that begins at or before this row
                int b = max(0, min(a.group_start[unit], a.num_seqs)), e = max(b, min(a.group_start[unit + 1], a.num_seqs)) - 1;
                while (b < e) {
                    const int mid = (b + e + 1) / 2;
                    if (a.q_start[mid] <= tok) b = mid;
                    else e = mid - 1;
                }
                s = b;
            }
            bool bad;
            const int L = clamped_len(a.context_lens, s, a.max_blocks_per_seq, a.block_size, &bad);
            const NewRows nr = rows_of(a, s, L);
            row_ok = tok >= nr.row0 && tok < nr.row0 + nr.n;
            pos = L - nr.n + tok - nr.row0;
            hi = min(pos + 1, prefix_len(a, unit));
        } else {
            pos = un.L - un.n + r / G;
            hi = pos + 1;
            if (a.bidirectional) hi = max(hi, min(a.bidirectional[unit], un.L));
            if (p.keys == kTailKeys) lo = prefix_of(a, unit);
            else if (a.first_key) lo = max(0, a.first_key[tok]);
        }
        if (kBias) slope = a.slopes[head] * kLog2e;
    }
    if (warp < kSoftWarps) {
        if (row_ok && lo >= hi) lo = hi = 0;
        const bool sees = row_ok && lo < hi;
        const int a_lo = __reduce_min_sync(kAll, sees ? lo : INT_MAX), b_lo = __reduce_max_sync(kAll, sees ? lo : 0);
        const int a_hi = __reduce_max_sync(kAll, sees ? hi : 0), b_hi = __reduce_min_sync(kAll, sees ? hi : INT_MAX);
        if (lane == 0 && a_hi > 0) {
            atomicMin(&lo_min[st], a_lo);
            atomicMax(&hi_max[st], a_hi);
            atomicMax(lo_max, b_lo);
            atomicMin(hi_min, b_hi);
        }
        if (!row_ok) {   // a row that is nobody's: nothing to mask
            lo = 0;
            hi = INT_MAX;
        }
    }
    __syncthreads();
    // stages st_begin .. st_begin + nst - 1 of 64 tokens are this CTA's; tile t sees those from tile_lo to tile_hi - 1
    const int k_lo = min(lo_min[0], lo_min[1]), k_hi = max(hi_max[0], hi_max[1]);
    int st_begin = 0, nst = 0;
    if (k_hi > k_lo) {
        const int s0 = k_lo / kStageTokens, cnt = (k_hi + kStageTokens - 1) / kStageTokens - s0;
        st_begin = s0 + (int)((unsigned)cnt * split / p.splits);   // (at most 2^24 stages, 2^7 splits)
        nst = s0 + (int)((unsigned)cnt * (split + 1) / p.splits) - st_begin;
    }
    auto tile_lo = [&](int t) { return hi_max[t] == 0 ? nst : max(0, min(nst, lo_min[t] / kStageTokens - st_begin)); };
    auto tile_hi = [&](int t) {
        return max(tile_lo(t), min(nst, (hi_max[t] + kStageTokens - 1) / kStageTokens - st_begin));
    };
    const size_t all_rows = (size_t)a.q_rows * a.num_q_heads;
    auto part_at = [&](int row) { return (size_t)(p.slot0 + split) * all_rows + row; };
    if (nst == 0) {   // uniform: no key for any row here
        if (row_ok) {
            if (a.part_o) {
                a.part_ml[part_at(row_at)] = make_float2(-INFINITY, 0.f);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + (size_t)row_at * kHeadDim);
                for (int c = 0; c < kHeadDim / 8; ++c) dst[c] = make_uint4(0, 0, 0, 0);
            }
        }
        free_tmem();
        return;
    }

    tc_fence_after();
    const uint32_t tmem = *tslot;

    auto give_up = [&]() {
        flag_status(a.status, PA_DEV_TIMEOUT);
        *abort_flag = 1;
    };

    if (warp == kProdWarp) {
        // ---------------- copies: one lane keeps the ring full ----------------
        if (lane == 0) {
            const int B = a.block_size, R = 1 << p.R_log2;
            const uint64_t box = R == 64 ? ~0ull : (1ull << R) - 1;
            // the blocks that hold tokens of stage i (up to four): their ids, read a stage ahead
            auto first_of = [&](int i) { return max((st_begin + i) * kStageTokens, k_lo) / B; };
            auto last_of = [&](int i) { return (min((st_begin + i + 1) * kStageTokens, k_hi) - 1) / B; };
            int ids[4];
            auto look = [&](int i) {
                const int first = first_of(i), last = last_of(i);
#pragma unroll
                for (int j = 0; j < 4; ++j) ids[j] = first + j <= last ? table_row[first + j] : 0;
            };
            look(0);
            int i = 0;
            for (; i < nst; ++i) {
                const int sl = i % kTStages;
                if (i >= kTStages && !bar_wait(kv_empty + sl * 8, (uint32_t)((i / kTStages) - 1) & 1u)) {
                    give_up();
                    break;
                }
                if (*abort_flag) break;
                // K and V, each 64-dim half of a block's R rows to [half][token]
                const int s0 = (st_begin + i) * kStageTokens, first = first_of(i), last = last_of(i);
                const int within = B > kStageTokens ? s0 % B : 0;
                int now[4];
                uint32_t bytes = 0;
                uint64_t ok = 0;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    now[j] = -1;
                    if (first + j <= last) {
                        if (ids[j] >= 0 && ids[j] < a.num_blocks) {
                            now[j] = ids[j];
                            bytes += 4u * (uint32_t)R * 128u;
                            ok |= box << (B > kStageTokens ? 0 : (first + j) * B - s0);
                        } else {
                            flag_status(a.status, PA_DEV_BAD_BLOCK_ID);
                        }
                    }
                }
                valid[sl] = ok;
                bar_expect(kv_full + sl * 8, bytes);
                const uint32_t dst = base + kOffRing + (uint32_t)sl * kStage;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    if (now[j] >= 0) {
                        const int row = (now[j] * a.num_kv_heads + hk) * B + within;
                        const uint32_t off = (uint32_t)(B > kStageTokens ? 0 : (first + j) * B - s0) * 128u;
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            bar_load(dst + h * kKVHalf + off, &maps.k, 64 * h, row, kv_full + sl * 8);
                            bar_load(dst + kKBytes + h * kKVHalf + off, &maps.v, 64 * h, row, kv_full + sl * 8);
                        }
                    }
                }
                if (i + 1 < nst) look(i + 1);
            }
            *issued_count = i;
        }
    } else if (warp == kCheckWarp) {
        // ---------------- V made fit for weights of zero ----------------
        const int all_lo = *lo_max, all_hi = *hi_min;
        for (int i = 0; i < nst; ++i) {
            const int sl = i % kTStages;
            if (!__all_sync(kAll, bar_wait(kv_full + sl * 8, (uint32_t)(i / kTStages) & 1u))) {
                if (lane == 0) give_up();
                break;
            }
            if (__any_sync(kAll, *abort_flag != 0)) break;
            const int s0 = (st_begin + i) * kStageTokens;
            const uint64_t ok = valid[sl];
            if (ok != ~0ull || s0 < all_lo || s0 + kStageTokens > all_hi) {
                const uint32_t v = base + kOffRing + (uint32_t)sl * kStage + kKBytes;
                // rows that no copy brought, or behind the last key: zero ([half][token][8 vectors])
                if (ok != ~0ull || s0 + kStageTokens > k_hi)
                    for (int k = lane; k < (int)kKBytes / 16; k += 32)
                        if (!(ok >> (k >> 3 & 63) & 1) || s0 + (k >> 3 & 63) >= k_hi) st_shared_v4(v + k * 16, make_uint4(0, 0, 0, 0));
                __syncwarp();
                bool wrong = false;
#pragma unroll 1
                for (int k0 = lane; k0 < (int)kKBytes / 16; k0 += 8 * 32) {
                    uint4 w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) w[k] = lds128(v + (k0 + k * 32) * 16);
                    uint32_t m[4] = {0, 0, 0, 0};   // the largest magnitudes, NaN above all
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        m[0] = max_abs2<T>(m[0], w[k].x);
                        m[1] = max_abs2<T>(m[1], w[k].y);
                        m[2] = max_abs2<T>(m[2], w[k].z);
                        m[3] = max_abs2<T>(m[3], w[k].w);
                    }
                    if (non_finite<T>(max_abs2<T>(max_abs2<T>(m[0], m[1]), max_abs2<T>(m[2], m[3])))) {
                        wrong = true;
                        for (int k = 0; k < 8; ++k) {
                            uint4 u = lds128(v + (k0 + k * 32) * 16);
                            u.x &= ~((non_finite<T>(u.x) >> 15) * 0xffffu);
                            u.y &= ~((non_finite<T>(u.y) >> 15) * 0xffffu);
                            u.z &= ~((non_finite<T>(u.z) >> 15) * 0xffffu);
                            u.w &= ~((non_finite<T>(u.w) >> 15) * 0xffffu);
                            st_shared_v4(v + (k0 + k * 32) * 16, u);
                        }
                    }
                }
                if (__any_sync(kAll, wrong) && lane == 0) {
                    *bad_first = min(*bad_first, i);
                    *bad_last = i;
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) bar_arrive(v_ready + sl * 8);
        }
    } else if (warp >= kMmaWarp) {
        // ---------------- products: one thread per tile, in warps on different schedulers ----------------
        // (the whole warp runs the loop, so that descriptors stay in uniform registers; one elected lane issues)
        const int t = __shfl_sync(kAll, warp, 0) - kMmaWarp;
        if (t < ntiles) {
            constexpr uint32_t kIdS = idesc<T>(kStageTokens, false);
            constexpr uint32_t kIdPV = idesc<T>(kHeadDim, true);
            const uint64_t dq = sdesc(base + kOffQ + t * kQTile, 16, 1024);
            const uint64_t dk0 = sdesc(base + kOffRing, 16, 1024);
            const uint64_t dv0 = sdesc(base + kOffRing + kKBytes, kKVHalf, 1024);
            const uint32_t d = tmem + (uint32_t)t * kTileCols;
            const int j0 = tile_lo(t), n = tile_hi(t) - j0;
            bool ok = true;
            auto wait = [&](uint32_t bar, uint32_t parity) { return __all_sync(kAll, bar_wait(bar, parity)) != 0; };
            // a stage that no row of the tile sees is released as soon as it has been looked through
            auto pass = [&](int j) {
                if (__any_sync(kAll, *abort_flag != 0) || !wait(v_ready + (j % kTStages) * 8, (uint32_t)(j / kTStages) & 1u))
                    return false;
                if (lane == 0) bar_arrive(kv_empty + (j % kTStages) * 8);
                return true;
            };
            for (int j = 0; j < j0 && ok; ++j) ok = pass(j);
            // S_k = Q K^T of the tile's k-th stage
            auto issue_s = [&](int k) -> bool {
                const int j = j0 + k, sl = j % kTStages;
                if (!wait(kv_full + sl * 8, (uint32_t)(j / kTStages) & 1u)) return false;
                if (k >= 1 && !wait(s_free + t * 8, (uint32_t)(k - 1) & 1u)) return false;
                tc_fence_after();
                const uint64_t dk = dk0 + (uint64_t)(((uint32_t)sl * kStage) >> 4);
                if (elect_one()) {
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            umma(d, dq + (uint64_t)((h * kQHalf + kk * 32) >> 4), dk + (uint64_t)((h * kKVHalf + kk * 32) >> 4),
                                 kIdS, (h | kk) != 0 ? 1u : 0u);
                    bar_commit(s_full + t * 8);
                }
                __syncwarp();
                return true;
            };
            if (ok && n > 0) {
                ok = wait(q_ready + t * 8, 0u);
                tc_fence_after();
                if (ok) ok = issue_s(0);
            }
            for (int k = 0; k < n && ok; ++k) {
                if (k + 1 < n && !issue_s(k + 1)) {
                    ok = false;
                    break;
                }
                const int j = j0 + k, sl = j % kTStages;
                if (!wait(p_full + (t * 2 + (k & 1)) * 8, (uint32_t)(k >> 1) & 1u) ||
                    !wait(v_ready + sl * 8, (uint32_t)(j / kTStages) & 1u)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint64_t dv = dv0 + (uint64_t)(((uint32_t)sl * kStage) >> 4);
                const uint32_t pt = d + kColP + (kSplitP ? 0u : (uint32_t)(k & 1) * 32u);
                if (elect_one()) {
#pragma unroll
                    for (int kt = 0; kt < 4; ++kt) {
                        const uint64_t v = dv + (uint64_t)((kt * 2048) >> 4);
                        umma_ts(d + kColO, pt + (uint32_t)(kt * 8), v, kIdPV, (k > 0 || kt > 0) ? 1u : 0u);
                        if (kSplitP) umma_ts(d + kColO, pt + 32u + (uint32_t)(kt * 8), v, kIdPV, 1u);
                    }
                    bar_commit(pv_done + (t * 2 + (k & 1)) * 8);
                    bar_commit(kv_empty + sl * 8);
                }
                __syncwarp();
            }
            for (int j = j0 + n; j < nst && ok; ++j) ok = pass(j);
            if (!ok && lane == 0) give_up();
            // nothing of this CTA's may still run on the tensor cores when it frees its memory (the commit is the electing
            // lane's, whose operations it waits for)
            if (elect_one()) bar_commit(drain);
            __syncwarp();
            (void)wait(drain, 0u);
        }
    } else if (st < ntiles) {
        // ------- softmax: four warps a tile, a thread owns a row -------
        const int t = st;
        const uint32_t lane_addr = tmem + (uint32_t)t * kTileCols + ((uint32_t)((warp & 3) * 32) << 16);
        // 16-byte chunk c of row r of this warp's 32 in the Q tile: also where results are turned from a thread's rows to
        // whole rows of memory (when all products with Q are done)
        const uint32_t warp_rows = base + kOffQ + t * kQTile + (warp & 3) * 32 * 128;
        auto row_chunk = [&](int r, int c) { return warp_rows + (c >> 3) * kQHalf + r * 128 + (((c ^ r) & 7) << 4); };
        const uint32_t t_s_full = s_full + t * 8;
        const uint32_t t_p_full = p_full + t * 16;
        const uint32_t t_pv_done = pv_done + t * 16;
        {
            // The scale's sign goes into Q (and a scale of zero makes it zero), so that the order of the scores is z's.  Half a
            // warp loads a row, for whole sectors.
            const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
            uint4 w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                const int from = 2 * i + (lane >> 4), at = __shfl_sync(kAll, row_at, from);
                const bool some = __shfl_sync(kAll, row_ok, from) && a.scale != 0.f;
                w[i] = some ? __ldg(reinterpret_cast<const uint4*>(static_cast<const T*>(a.q) + (size_t)at * kHeadDim) + (lane & 15))
                            : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                w[i].x ^= flip;
                w[i].y ^= flip;
                w[i].z ^= flip;
                w[i].w ^= flip;
                st_shared_v4(row_chunk(2 * i + (lane >> 4), lane & 15), w[i]);
            }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) bar_arrive(q_ready + t * 8);

        auto warp_wait = [&](uint32_t bar, uint32_t parity) -> bool {
            return __all_sync(kAll, bar_wait(bar, parity));
        };
        // log2(e) times the score: xs * S, or with a cap capl tanh(y), y = ks S (while |y| <= kTanhReach a polynomial)
        const float scale = fabsf(a.scale), ks = kCap ? scale / a.cap : 0.f, xs = a.scale == 0.f ? 1.f : scale * kLog2e;
        const float capl = a.cap * kLog2e, c1 = kTanh1 * capl, c2 = kTanh2 * capl, c3 = kTanh3 * capl, c4 = kTanh4 * capl;
        auto capped2 = [&](float2 y) {
            const float2 y2 = ffma2(y, y, make_float2(0.f, 0.f));
            float2 q = ffma2(make_float2(c4, c4), y2, make_float2(c3, c3));
            q = ffma2(q, y2, make_float2(c2, c2));
            q = ffma2(q, y2, make_float2(c1, c1));
            q = ffma2(q, y2, make_float2(capl, capl));
            return ffma2(y, q, make_float2(0.f, 0.f));
        };
        auto capped_far = [&](float y) { return capl - __fdividef(2.f * capl, 1.f + ex2(y * (2.f * kLog2e))); };
        float2 step2[kBias ? 4 : 1];     // the bias of eight keys from the first one's on
        if (kBias)
#pragma unroll
            for (int c = 0; c < 4; ++c) step2[kBias ? c : 0] = make_float2(slope * (2 * c), slope * (2 * c + 1));
        float m_run = -INFINITY, l_run = 0.f;
        bool dead = false;
        const int j0 = tile_lo(t), n = tile_hi(t) - j0;
        for (int k = 0; k < n; ++k) {
            const int j = j0 + k;
            if (!warp_wait(t_s_full, (uint32_t)k & 1u)) {
                dead = true;
                break;
            }
            tc_fence_after();
            float x[64];
            tmem_ld64(lane_addr, x);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(s_free + t * 8);
            const int t0 = (st_begin + j) * kStageTokens;
            const uint64_t there = valid[j % kTStages];
            const bool whole = __all_sync(kAll, t0 >= lo && t0 + 64 <= hi && there == ~0ull);
            // the keys of the stage that the row sees
            uint32_t vis[2] = {~0u, ~0u};
            if (!whole) {
                const int from = max(lo - t0, 0), to = min(hi - t0, 64);
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int f = from - 32 * e, n = to - 32 * e;
                    const uint32_t behind = n >= 32 ? 0u : n <= 0 ? ~0u : ~0u << n, before = f >= 32 ? ~0u : f <= 0 ? 0u : ~(~0u << f);
                    vis[e] = (uint32_t)(there >> (32 * e)) & ~behind & ~before;
                }
            }
            // A cap: log2 units in the place of S.  A score's own size chooses the form of its tanh, so that nothing else can
            // change its bits; the vote spares the exponentials where no score of the warp's stage wants one.
            if (kCap) {
                float m4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                for (int c = 0; c < 64; c += 2) {
                    const float2 y = ffma2(make_float2(x[c], x[c + 1]), make_float2(ks, ks), make_float2(0.f, 0.f));
                    x[c] = y.x;
                    x[c + 1] = y.y;
                    m4[c >> 1 & 3] = fmax3(m4[c >> 1 & 3], fabsf(y.x), fabsf(y.y));
                }
                if (__any_sync(kAll, fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) > kTanhReach)) {
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const float2 y = make_float2(x[c], x[c + 1]), z = capped2(y);
                        const float e0 = capped_far(y.x), e1 = capped_far(y.y);
                        x[c] = fabsf(y.x) > kTanhReach ? e0 : z.x;
                        x[c + 1] = fabsf(y.y) > kTanhReach ? e1 : z.y;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const float2 z = capped2(make_float2(x[c], x[c + 1]));
                        x[c] = z.x;
                        x[c + 1] = z.y;
                    }
                }
            }
            float f = kBias || kCap ? 1.f : xs;   // the factor still to apply
            float bias0 = 0.f, bias8 = 0.f;       // what the registers lack of the bias: bias0, and bias8 times the group of eight keys
            if (kBias) {
                const float far = (float)(t0 - pos), to_log2 = kCap ? 1.f : xs;
                // no key lies behind its row, and the bias can be taken apart
                const bool before = __all_sync(kAll, (t0 + 63 <= pos && fabsf(slope * far) <= kLargeScore) || !row_ok);
                if (before) {
                    bias0 = slope * far;
                    bias8 = 8.f * slope;
#pragma unroll
                    for (int c = 0; c < 64; c += 2) {
                        const float2 y = ffma2(make_float2(x[c], x[c + 1]), make_float2(to_log2, to_log2), step2[kBias ? (c >> 1 & 3) : 0]);
                        x[c] = y.x;
                        x[c + 1] = y.y;
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] = fmaf(x[c], to_log2, -slope * fabsf(far + (float)c));
                }
            }
            if (!whole) {
#pragma unroll
                for (int c = 0; c < 64; ++c) x[c] = vis[c >> 5] & (1u << (c & 31)) ? x[c] : -INFINITY;
            }
            // the maximum by groups of eight, as trees of three-input steps
            float m8[8];
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                float m = fmax3(x[8 * g], x[8 * g + 1], x[8 * g + 2]);
                m = fmax3(m, x[8 * g + 3], x[8 * g + 4]);
                m = fmax3(m, x[8 * g + 5], x[8 * g + 6]);
                m8[g] = fmaxf(m, x[8 * g + 7]);
                if (kBias) m8[g] += fmaf(bias8, (float)g, bias0);
            }
            float mx = fmax3(fmax3(m8[0], m8[1], m8[2]), fmax3(m8[3], m8[4], m8[5]), fmaxf(m8[6], m8[7]));
            if (!kBias && !kCap && mx != -INFINITY) mx *= f;
            // The base moves when a score would put its weight above 2^top_most (the distance is compared, and a new base
            // rounded towards the maximum: scores of 2^24 and more leave few bits for such offsets).
            const bool move = mx - m_run > top_most<T>();
            const bool large = (kBias || !kCap) && fabsf(mx) > kLargeScore && mx != -INFINITY;   // (capped ones are rounded)
            if (__any_sync(kAll, move || large)) {
                if (large) {
#pragma unroll
                    for (int c = 0; c < 64; ++c) x[c] = kBias ? x[c] + fmaf(bias8, (float)(c >> 3), bias0) : x[c] * f;
                    bias0 = bias8 = 0.f;
                    f = 1.f;
                }
                const float m_new = !move ? m_run : top_new<T>() > 0.f ? __fadd_ru(mx, -top_new<T>()) : __fadd_rd(mx, -top_new<T>());
                if (__any_sync(kAll, move && k > 0 && m_run != -INFINITY)) {
                    // O holds the stages before this one once their last product is complete
                    if (!warp_wait(t_pv_done + ((k - 1) & 1) * 8, (uint32_t)((k - 1) >> 1) & 1u)) {
                        dead = true;
                        break;
                    }
                    tc_fence_after();
                    const float alpha = (move && m_run != -INFINITY) ? exp2f(m_run - m_new) : 1.f;
#pragma unroll 1
                    for (int c0 = 0; c0 < kHeadDim; c0 += 16) {   // few at a time: the scores are in registers, too
                        float o[16];
                        uint32_t u[16];
                        tmem_ld16(lane_addr + kColO + c0, o);
#pragma unroll
                        for (int c = 0; c < 16; ++c) u[c] = __float_as_uint(o[c] * alpha);
                        tmem_st16u(lane_addr + kColO + c0, u);
                    }
                    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                    l_run *= alpha;
                }
                m_run = m_new;
            }
            const float m_use = (m_run == -INFINITY) ? 0.f : m_run;
            float2 rs2[4] = {{0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}, {0.f, 0.f}};
            // P goes to tensor memory in parts of kPart words.  fp16: the buffer was last read by the product of two stages
            // before, which was issued before this stage's S: it is complete, since the arrival on s_full waits for all that
            // was issued before it.  bf16: the one buffer is free once the last stage's product is complete.
            constexpr int kPart = kSplitP ? 16 : 32;
            const uint32_t p_at = lane_addr + kColP + (kSplitP ? 0u : (uint32_t)(k & 1) * 32u);
            uint32_t w[kPart];
            auto weights = [&](auto exponent) {
#pragma unroll
                for (int part = 0; part < 32; part += kPart) {
                    uint32_t low[kPart];
#pragma unroll
                    for (int c = 0; c < kPart; ++c) {
                        const int c2 = part + c;
                        const float2 e2 = exponent(c2, make_float2(x[2 * c2], x[2 * c2 + 1]));
                        const float p0 = ex2(e2.x), p1 = ex2(e2.y);
                        w[c] = kSplitP ? high_part2(p0, p1) : Elem<T>::pack2(p0, p1);
                        if (kSplitP) {
                            const float2 d = ffma2(make_float2(p0, p1), make_float2(kLowPart, kLowPart), Elem<T>::to_float2(w[c] ^ 0x80008000u));
                            low[c] = Elem<T>::pack2(d.x, d.y);
                        }
                        rs2[c2 & 3] = fadd2(rs2[c2 & 3], make_float2(p0, p1));
                    }
                    if constexpr (kSplitP) {
                        if (part == 0 && k > 0) {
                            if (!warp_wait(t_pv_done + ((k - 1) & 1) * 8, (uint32_t)((k - 1) >> 1) & 1u)) dead = true;
                            tc_fence_after();
                        }
                        tmem_st16u(p_at + part, w);
                        tmem_st16u(p_at + 32 + part, low);
                    }
                }
            };
            const float2 nm2 = make_float2(-m_use, -m_use);
            if (kBias) {
                float2 from[8];   // the base less what the bias of a group lacks
#pragma unroll
                for (int g = 0; g < 8; ++g) from[g].x = from[g].y = fmaf(bias8, (float)g, bias0) - m_use;
                weights([&](int c2, float2 y) { return fadd2(y, from[c2 >> 2]); });
            } else if (!kCap) {
                weights([&](int, float2 s) { return ffma2(s, make_float2(f, f), nm2); });
            } else {
                weights([&](int, float2 y) { return fadd2(y, nm2); });
            }
            if (kSplitP && dead) break;
            if constexpr (!kSplitP) tmem_st32u(p_at, w);
            l_run += ((rs2[0].x + rs2[0].y) + (rs2[1].x + rs2[1].y)) + ((rs2[2].x + rs2[2].y) + (rs2[3].x + rs2[3].y));
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tc_fence_before();
            __syncwarp();
            if (lane == 0) bar_arrive(t_p_full + (k & 1) * 8);
        }
        // ---- the row's result ----
        if (!dead && n > 0 && !warp_wait(t_pv_done + ((n - 1) & 1) * 8, (uint32_t)((n - 1) >> 1) & 1u)) dead = true;
        if (!dead) {
            tc_fence_after();
            const float inv = a.part_o ? 1.f : l_run == 0.f ? 0.f : 1.f / l_run;
            const int wrong0 = *bad_first, wrong1 = *bad_last;   // (warp 11 is past every stage of this tile)
            const bool none = m_run == -INFINITY;                // (its weights of zero may have met anything)
            if (row_ok && a.part_o) a.part_ml[part_at(row_at)] = make_float2(m_run, l_run);
            const uint32_t rows_ok = __ballot_sync(kAll, row_ok);
            // Rare: values that are not finite, of tokens the row sees, taken out of the products above (those left in them
            // count twice, which changes nothing), into the row as it lies in shared memory, from dim d0 on.
            auto add_non_finite = [&](int d0) {
                const int dims = a.part_o ? 64 : kHeadDim;
#pragma unroll 1
                for (int tok = max((st_begin + wrong0) * kStageTokens, lo);
                     tok < min((st_begin + wrong1 + 1) * kStageTokens, min(hi, k_hi)); ++tok) {
                    const int id = table_row[tok / a.block_size];
                    if (id < 0 || id >= a.num_blocks) continue;
                    const uint16_t* v = static_cast<const uint16_t*>(a.v_cache) + d0 +
                                        (((size_t)id * a.num_kv_heads + hk) * a.block_size + tok % a.block_size) * kHeadDim;
#pragma unroll 1
                    for (int d = 0; d < dims; ++d) {
                        if (!non_finite<T>(v[d])) continue;
                        const float x = Elem<T>::to_float(v[d]);
                        const uint32_t at = a.part_o ? row_chunk(lane, d / 4) + d % 4 * 4 : row_chunk(lane, d / 8) + d % 8 * 2;
                        if (a.part_o) {
                            sts32(at, lds32(at) + x);
                        } else {
                            sts16(at, (uint16_t)Elem<T>::pack2(Elem<T>::to_float(lds16(at)) + x, 0.f));
                        }
                    }
                }
            };
#pragma unroll 1
            for (int c0 = 0; c0 < kHeadDim; c0 += 32) {
                float o[32];
                __syncwarp();
                if (n > 0) tmem_ld32(lane_addr + kColO + c0, o);
                if (n == 0 || none) {
#pragma unroll
                    for (int c = 0; c < 32; ++c) o[c] = 0.f;
                }
                if (a.part_o) {
#pragma unroll
                    for (int c = 0; c < 8; ++c)
                        st_shared_v4(row_chunk(lane, (c0 & 32) / 4 + c),
                                     make_uint4(__float_as_uint(o[4 * c]), __float_as_uint(o[4 * c + 1]),
                                                __float_as_uint(o[4 * c + 2]), __float_as_uint(o[4 * c + 3])));
                } else {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        st_shared_v4(row_chunk(lane, c0 / 8 + c),
                                     make_uint4(Elem<T>::pack2(o[c * 8 + 0] * inv, o[c * 8 + 1] * inv),
                                                Elem<T>::pack2(o[c * 8 + 2] * inv, o[c * 8 + 3] * inv),
                                                Elem<T>::pack2(o[c * 8 + 4] * inv, o[c * 8 + 5] * inv),
                                                Elem<T>::pack2(o[c * 8 + 6] * inv, o[c * 8 + 7] * inv)));
                }
                if (c0 == kHeadDim - 32 || (a.part_o && c0 == kHeadDim / 2 - 32)) {   // 256 bytes of every row are there
                    if (wrong0 <= wrong1) add_non_finite(a.part_o ? c0 & 64 : 0);
                    __syncwarp();
                    char* out = (a.part_o ? reinterpret_cast<char*>(a.part_o + part_at(0) * kHeadDim + (c0 & 64))
                                          : static_cast<char*>(a.out)) + (lane & 15) * 16;
                    const int bytes = kHeadDim * (a.part_o ? 4 : 2);
#pragma unroll 1
                    for (int i0 = 0; i0 < 16; i0 += 8) {
                        uint4 v[8];
                        char* to[8];
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const int from = 2 * (i0 + i) + (lane >> 4);
                            to[i] = out + (size_t)__shfl_sync(kAll, row_at, from) * bytes;
                            v[i] = lds128(row_chunk(from, lane & 15));
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i)
                            if (rows_ok >> (2 * (i0 + i) + (lane >> 4)) & 1) *reinterpret_cast<uint4*>(to[i]) = v[i];
                    }
                    __syncwarp();
                }
            }
        } else {
            give_up();
        }
    }

    // ---- teardown: nothing in flight on the tensor cores or the copy engine, then free ----
    tc_fence_before();
    __syncthreads();
    if (*abort_flag && tid == 0) {
        // let every copy still in flight land before the CTA's shared memory is released
        const int n = *issued_count;
        for (int sl = 0; sl < kTStages; ++sl) {
            int last = -1;
            for (int i = sl; i < n; i += kTStages) last = i;
            if (last >= 0) (void)bar_wait(kv_full + sl * 8, (uint32_t)(last / kTStages) & 1u);
        }
    }
    __syncthreads();
    free_tmem();
}

// Joins the pieces of a row, one warp each: lane l weighs slots l, l + 32, .., then has four elements of every piece.
constexpr int kCombineWarps = 8;

template <typename T>
__global__ void __launch_bounds__(kCombineWarps * 32) attend_combine_kernel(const AttendArgs a, int own, int shared) {
    const int lane = threadIdx.x % 32;
    const long long row = (long long)blockIdx.x * kCombineWarps + threadIdx.x / 32;
    const long long all_rows = (long long)a.q_rows * a.num_q_heads;
    grid_dependency_wait();
    grid_launch_dependents();
    if (row >= all_rows) return;
    const int tok = (int)(row / a.num_q_heads);
    // the slots' bases and sums, the prefix's too before it is known whether the row has one
    float2 ml[kMostSlots / 32];
#pragma unroll
    for (int i = 0; i < kMostSlots / 32; ++i) {
        const int slot = i * 32 + lane;
        ml[i] = slot < own + shared ? a.part_ml[(size_t)slot * all_rows + row] : make_float2(-INFINITY, 0.f);
    }
    // ... and so the first eight pieces
    constexpr int kAhead = 8;
    const float* at = a.part_o + (size_t)row * kHeadDim + lane * 4;
    float4 ahead[kAhead];
#pragma unroll
    for (int e = 0; e < kAhead; ++e)
        ahead[e] = e < own + shared ? ld_cg4(at + (size_t)e * all_rows * kHeadDim) : make_float4(0.f, 0.f, 0.f, 0.f);
    int s = tok;
    if (a.q_start) {
        s = last_not_above(a.q_start, a.num_seqs, tok);
        bool bad;
        const int L = clamped_len(a.context_lens, s, a.max_blocks_per_seq, a.block_size, &bad);
        const NewRows nr = rows_of(a, s, L);
        if (tok < nr.row0 || tok >= nr.row0 + nr.n) return;   // nobody's row stays as it was
    }
    int slots = own;
    if (shared) {
        const int g = last_not_above(a.group_start, a.num_groups, s);
        if (a.group_start[g] <= s && s < a.group_start[g + 1]) slots += shared;
    }
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < kMostSlots / 32; ++i) {
        if (i * 32 + lane >= slots) ml[i] = make_float2(-INFINITY, 0.f);
        m = (ml[i].x != ml[i].x) ? ml[i].x : fmaxf(m, ml[i].x);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kAll, m, o));
    float l = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kMostSlots / 32; ++i) {
        const float f = join_factor(ml[i].x, m);
        l += f * ml[i].y;
        const int here = min(32, slots - i * 32);
        if (i == 0) {
#pragma unroll
            for (int e = 0; e < kAhead; ++e) {
                const float w = __shfl_sync(kAll, f, e);
                if (e < here && __shfl_sync(kAll, ml[0].x, e) != -INFINITY) {
                    acc.x = fmaf(w, ahead[e].x, acc.x);
                    acc.y = fmaf(w, ahead[e].y, acc.y);
                    acc.z = fmaf(w, ahead[e].z, acc.z);
                    acc.w = fmaf(w, ahead[e].w, acc.w);
                }
            }
        }
        for (int j = i == 0 ? kAhead : 0; j < here; j += 4) {
            float4 v[4];
            float w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                w[e] = __shfl_sync(kAll, f, (j + e) & 31);
                const bool some = j + e < here && __shfl_sync(kAll, ml[i].x, (j + e) & 31) != -INFINITY;
                v[e] = some ? ld_cg4(at + (size_t)(i * 32 + j + e) * all_rows * kHeadDim) : make_float4(0.f, 0.f, 0.f, 0.f);
                if (!some) w[e] = 0.f;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                acc.x = fmaf(w[e], v[e].x, acc.x);
                acc.y = fmaf(w[e], v[e].y, acc.y);
                acc.z = fmaf(w[e], v[e].z, acc.z);
                acc.w = fmaf(w[e], v[e].w, acc.w);
            }
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(kAll, l, o);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint2 w;
    w.x = Elem<T>::pack2(acc.x * inv, acc.y * inv);
    w.y = Elem<T>::pack2(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(static_cast<T*>(a.out) + (size_t)row * kHeadDim + lane * 4) = w;
}

template <typename T, bool kCap, bool kBias>
cudaError_t launch_kind(const TcLaunch& p, const Maps& maps, dim3 grid, cudaStream_t stream) {
    static std::atomic<unsigned long long> allowed{0};   // devices on which the kernel may have its shared memory
    auto kernel = attend_tc_kernel<T, kCap, kBias>;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (dev > 63 || !(allowed.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        allowed.fetch_or(dev > 63 ? 0 : bit);
    }
    return launch_pdl(kernel, grid, dim3(kTThreads), kSmem, stream, p, maps);
}

template <typename T>
cudaError_t launch_type(const TcLaunch& p, const Maps& maps, dim3 grid, cudaStream_t stream) {
    if (p.a.cap > 0.f)
        return p.a.slopes ? launch_kind<T, true, true>(p, maps, grid, stream) : launch_kind<T, true, false>(p, maps, grid, stream);
    return p.a.slopes ? launch_kind<T, false, true>(p, maps, grid, stream) : launch_kind<T, false, false>(p, maps, grid, stream);
}

}  // namespace

TcSplits tc_splits(long long rows_bound, int units, int num_kv_heads, long long max_keys, int most, int sms) {
    // every unit may end in the middle of a pair of tiles; how many do is not known here
    const long long items = (rows_bound + (long long)(kCtaRows - 1) * units) / kCtaRows;
    const long long whole = (rows_bound + kCtaRows - 1) / kCtaRows;
    const long long likely = max(1LL, min(items, max((long long)units, whole + (units - 1) / 2)) * num_kv_heads);
    const long long stages = max(1LL, (max_keys + kStageTokens - 1) / kStageTokens);
    const long long splits = max(1LL, min(min((long long)most, stages), sms / likely));
    return TcSplits{(int)items, (int)splits};
}

cudaError_t launch_attend_tc(const AttendArgs& a, int dtype, AttendKeys keys, TcSplits grid, int slot0,
                             cudaStream_t stream) {
    TcLaunch p;
    p.a = a;
    p.keys = keys;
    p.units = keys == kPrefixKeys ? a.num_groups : a.num_seqs;
    p.splits = grid.splits;
    p.slot0 = slot0;
    p.R_log2 = 0;
    const int R = min(a.block_size, kStageTokens);
    while ((1 << p.R_log2) < R) ++p.R_log2;
    const unsigned long long rows = (unsigned long long)a.num_blocks * a.num_kv_heads * a.block_size;
    Maps maps;
    if (!encode_pool_map(a.k_cache, rows, R, &maps.k)) {
        // a host thread that has made no CUDA call yet has no current context, which the encoding asks for
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || cudaSetDevice(dev) != cudaSuccess ||
            !encode_pool_map(a.k_cache, rows, R, &maps.k))
            return cudaErrorInvalidValue;
    }
    if (!encode_pool_map(a.v_cache, rows, R, &maps.v)) return cudaErrorInvalidValue;
    const dim3 g((unsigned)(grid.items * grid.splits), a.num_kv_heads);
    return dtype == PA_BF16 ? launch_type<__nv_bfloat16>(p, maps, g, stream) : launch_type<__half>(p, maps, g, stream);
}

cudaError_t launch_attend_combine(const AttendArgs& a, int dtype, int own, int shared, cudaStream_t stream) {
    const long long rows = (long long)a.q_rows * a.num_q_heads;
    const dim3 grid((unsigned)((rows + kCombineWarps - 1) / kCombineWarps)), block(kCombineWarps * 32);
    return dtype == PA_BF16 ? launch_pdl(attend_combine_kernel<__nv_bfloat16>, grid, block, 0, stream, a, own, shared)
                            : launch_pdl(attend_combine_kernel<__half>, grid, block, 0, stream, a, own, shared);
}

}  // namespace pa
