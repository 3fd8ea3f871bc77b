"""What a CTA of the 8-bit attention joins at its end (csrc/q8_join.h), on the host: every cut segment once and from its
own pieces, and nothing when a warp's copy wait ran out, whose pieces are then missing."""
import ctypes
import subprocess
from pathlib import Path

import numpy as np
import pytest

CSRC = Path(__file__).resolve().parent.parent / "paged_kv_cache_08_gb300" / "csrc"
HARNESS = """
#include "q8_join.h"
extern "C" void join(const int* flags, int warps, int* out) {   // out: first, last, chains, then (from, to, before) of each
    unsigned m[5] = {0, 0, 0, 0, 0};
    const int bit[5] = {pa::kNoUnits, pa::kHasFirst, pa::kHasLast, pa::kThrough, pa::kGaveUp};
    for (int w = 0; w < 32; ++w)
        for (int i = 0; i < 5; ++i)
            if ((w < warps ? flags[w] : pa::kNoUnits) & bit[i]) m[i] |= 1u << w;
    const pa::CtaJoin j = pa::cta_join(m[0], m[1], m[2], m[3], m[4], warps);
    out[0] = j.left_first;
    out[1] = j.left_last;
    int n = 0;
    for (unsigned ev = j.events; ev; ev &= ev - 1, ++n) {
        const pa::JoinChain c = j.chain(ev);
        out[3 + 3 * n] = c.from;
        out[4 + 3 * n] = c.to;
        out[5 + 3 * n] = c.before;
    }
    out[2] = n;
}
"""
FIRST, LAST, THROUGH, NONE, GAVE_UP = 1, 2, 4, 8, 16


@pytest.fixture(scope="module")
def join(tmp_path_factory):
    d = tmp_path_factory.mktemp("join")
    (d / "join.cpp").write_text(HARNESS)
    subprocess.run(["g++", "-O1", "-Wall", "-Werror", "-fPIC", "-shared", "-I", str(CSRC), str(d / "join.cpp"), "-o",
                    str(d / "join.so")], check=True)
    lib = ctypes.CDLL(str(d / "join.so"))

    def call(flags):
        a, out = (ctypes.c_int * len(flags))(*flags), (ctypes.c_int * 64)()
        lib.join(a, len(flags), out)
        return out[0], out[1], [tuple(out[3 + 3 * i:6 + 3 * i]) for i in range(out[2])]

    return call


def _flags(cuts, ends):
    """Flags of the warps whose shares are cuts[w] .. cuts[w + 1] of a line on which segments end at `ends` (ascending,
    the last is the line's end), as the kernel sets them."""
    ends, flags = np.asarray(ends), []
    for a, b in zip(cuts[:-1], cuts[1:]):
        f, at = (NONE if a == b else 0), a
        while at < b:
            i = int(np.searchsorted(ends, at, side="right"))
            begin, end = (int(ends[i - 1]) if i else 0), int(ends[i])
            if end > b:
                f |= LAST | (THROUGH if begin < at else 0)
            elif begin < at:
                f |= FIRST
            at = min(end, b)
        flags.append(f)
    return flags


def _line(rng, shares):
    """Cuts of a random line into shares, some empty, and the ends of its segments."""
    total = int(rng.integers(1, 40 * shares))
    cuts = np.sort(np.concatenate([[0, total], rng.integers(0, total + 1, shares - 1)])).tolist()
    ends = np.unique(np.concatenate([[total], rng.integers(1, total + 1, int(rng.choice([1, 4, shares, 4 * shares])))]))
    return cuts, ends.tolist()


@pytest.mark.parametrize("warps", [8, 12])
def test_cut_segments_are_joined_once(join, warps):
    rng = np.random.default_rng(warps)
    for _ in range(3000):
        ctas = int(rng.integers(1, 4))
        cuts, ends = _line(rng, ctas * warps)
        begins = [0] + ends[:-1]
        flags = _flags(cuts, ends)
        for c in range(ctas):
            mine = cuts[c * warps:(c + 1) * warps + 1]
            first, last, chains = join(flags[c * warps:(c + 1) * warps])
            want = []          # segments in two shares and more, by the part of them inside this CTA
            for a, b in zip(begins, ends):
                lo, hi = max(a, mine[0]), min(b, mine[-1])
                if lo >= hi:
                    continue
                ws = [w for w in range(warps) if max(lo, mine[w]) < min(hi, mine[w + 1])]
                if len(ws) > 1 or a < mine[0] or b > mine[-1]:
                    want.append((0 if a < mine[0] else ws[0], warps if b > mine[-1] else ws[-1], int(a < mine[0])))
            assert sorted(chains) == sorted(want)
            before = [b for _, b, x in want if x]
            assert first == (3 if mine[0] == mine[-1] else 0 if not before else 2 if before[0] == warps else 1)
            assert last == any(b == warps and not x for _, b, x in want)
            if ctas == 1:      # such a grid has no workspace: nothing may be left for other CTAs
                assert (first, last) in ((0, 0), (3, 0)) and not any(x for _, _, x in chains)


@pytest.mark.parametrize("warps", [8, 12])
def test_nothing_is_joined_where_a_warp_gave_up(join, warps):
    rng = np.random.default_rng(100 + warps)
    for _ in range(1000):
        cuts, ends = _line(rng, warps)
        flags = _flags(cuts, ends)
        busy = [w for w in range(warps) if flags[w] != NONE]
        for dead in [[w] for w in busy] + [busy]:
            assert join([GAVE_UP if w in dead else f for w, f in enumerate(flags)]) == (3, 0, [])
