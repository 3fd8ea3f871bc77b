// What a CTA of the 8-bit attention joins at its end, from what its warps left of cut segments.  Plain C++: the
// kernel's decisions can be checked on the host.
#pragma once

#ifdef __CUDACC__
#define PA_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define PA_HOST_DEVICE inline
#endif

namespace pa {

// Flags of a warp.
constexpr int kHasFirst = 1;    // a piece of a segment begun before the warp's share, ended in it
constexpr int kHasLast = 2;     // a piece of a segment that goes on
constexpr int kThrough = 4;     // ... and that also began before the share
constexpr int kNoUnits = 8;
constexpr int kGaveUp = 16;     // a copy did not come in time: the warp's pieces are missing

PA_HOST_DEVICE int lowest_bit(unsigned x) {    // x != 0
#ifdef __CUDA_ARCH__
    return __ffs((int)x) - 1;
#else
    return __builtin_ctz(x);
#endif
}

PA_HOST_DEVICE int highest_bit(unsigned x) {   // x != 0
#ifdef __CUDA_ARCH__
    return 31 - __clz((int)x);
#else
    return 31 - __builtin_clz(x);
#endif
}

// One chain of pieces: warps from .. to, of which `to` gives its first piece if the chain ends there (to < warps), every
// other warp its last.  `before`: the chain's segment began in an earlier CTA.
struct JoinChain {
    int from, to;
    bool before;
};

struct CtaJoin {
    unsigned some;      // warps with units
    unsigned opens;     // warps whose last piece opens a chain
    unsigned events;    // chains by where they end: at a warp's first piece, or (bit `warps`) open at the CTA's end
    int warps;
    int last_warp;      // the last of `some`
    int left_first;     // CtaPieces::first and ::last
    int left_last;

    // The chain of the lowest bit of `ev`, a tail of `events`.
    PA_HOST_DEVICE JoinChain chain(unsigned ev) const {
        const int to = lowest_bit(ev);
        const unsigned below = events & ((1u << to) - 1);
        const unsigned opener = opens & ((1u << to) - 1) & ~((1u << (below ? highest_bit(below) : 0)) - 1);
        return JoinChain{opener ? lowest_bit(opener) : 0, to, opener == 0};
    }
};

// A first piece ends the chain of pieces that is open (or one from before this CTA), a last piece goes on with it
// (kThrough) or opens one.  The arguments are masks of the CTA's warps by flag.  Where a warp gave up, its pieces are
// missing and a chain could take one from before the CTA for its own: nothing is joined then, and later CTAs are told
// that this one had no work.
PA_HOST_DEVICE CtaJoin cta_join(unsigned idle, unsigned firsts, unsigned lasts, unsigned through, unsigned gave_up,
                                int warps) {
    CtaJoin j;
    j.some = ~idle & ((1u << warps) - 1);
    j.opens = lasts & ~through;
    j.warps = warps;
    j.last_warp = j.some ? highest_bit(j.some) : 0;
    j.events = firsts | ((lasts >> j.last_warp & 1) << warps);
    j.left_first = j.some ? 0 : 3;
    j.left_last = 0;
    if (gave_up) {
        j.events = 0;
        j.left_first = 3;
    }
    if (j.events) {
        const int e = lowest_bit(j.events);
        if (!(j.opens & ((1u << e) - 1))) j.left_first = e < warps ? 1 : 2;
    }
    if ((j.events >> warps) && (j.opens >> (firsts ? highest_bit(firsts) : 0))) j.left_last = 1;
    return j;
}

}  // namespace pa
