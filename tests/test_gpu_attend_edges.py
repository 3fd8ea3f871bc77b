"""Attention with other scores, masks and shared prefixes at the edges of what its calls may be given, on the GPU
against the definition in 64 bits."""
import math

import pytest
import torch

import attend_reference as ref
import paged_kv_cache_08_gb300 as pa
from paged_kv_cache_08_gb300 import _native
from test_gpu_attend import BF16, DEV, F16, clean, make, run, slopes_of, status, window  # noqa: F401 (status: every test's)

pytestmark = pytest.mark.gpu


def as_single_tokens(case):
    """The rows of a call with several tokens, each as a sequence of one token at the same position: the same definition,
    with the bound of weights that enter the products with 11 (fp16) or 16 bits (bf16)."""
    tables, lens, rows = [], [], []
    for s in range(len(case["lens"])):
        r0, n, L = ref.rows_of(case, s)
        tables += [case["tables"][s]] * n
        lens += list(range(L - n + 1, L + 1))
        rows += list(range(r0, r0 + n))
    one = dict(case, q=case["q"][rows], tables=torch.stack(tables), lens=torch.tensor(lens, dtype=torch.int32), start=None,
               max_q=1)
    if case.get("first") is not None:
        one["first"] = case["first"][rows]
    for name in ("prefix_tables", "prefix_lens", "group_start"):   # (the sequences' own tables name the prefix, too)
        one.pop(name, None)
    return one, rows


def copies(case, n):
    """The batch n times over the same blocks: so many rows that no row's keys are split among CTAs."""
    S = len(case["lens"])
    many = dict(case, q=case["q"].repeat(n, 1, 1), tables=case["tables"].repeat(n, 1), lens=case["lens"].repeat(n))

    def ends(x, step):
        return torch.cat([x[:1]] + [x[1:] + i * step for i in range(n)]).to(torch.int32)

    if case["start"] is not None:
        many["start"] = ends(case["start"], int(case["start"][-1]))
    if case.get("first") is not None:
        many["first"] = case["first"].repeat(n)
    if case.get("group_start") is not None:   # (the groups hold all sequences)
        many.update(prefix_tables=case["prefix_tables"].repeat(n, 1), prefix_lens=case["prefix_lens"].repeat(n),
                    group_start=ends(case["group_start"], S))
    return many


def check_copies(case, n=160):
    out = run(copies(case, n)).reshape(n, *case["q"].shape)
    assert torch.isfinite(out).all()
    for i in (0, n // 2, n - 1):            # (shares of a stream are cut anywhere: copies differ in their last bits)
        ref.check(out[i], case)


# ---- counts above max_q ----------------------------------------------------------------------

@pytest.mark.parametrize("Hq,Hkv,max_q,new,groups", [
    (6, 1, 1, [1000, 1, 1, 1], [(0, 4, 130)]),                   # the tails streamed
    (1, 1, 4, [1000, 4], [(0, 1, 130), (1, 2, 130)]),
    (12, 2, 5, [900, 5, 2, 5], [(0, 2, 70), (2, 4, 140)]),       # ... in tiles
    (6, 1, 1, [1, 700, 1, 700, 1], [(0, 3, 40), (3, 5, 200)])])
@pytest.mark.parametrize("dtype", [F16, BF16])
def test_counts_above_max_q_leave_other_rows_alone(Hq, Hkv, max_q, new, groups, dtype):
    """A count is clamped and flagged; the rows of all sequences, its own first ones too, are as without the surplus."""
    lens = [300 + 7 * i for i in range(len(new))]
    case = make(lens, new, Hq=Hq, Hkv=Hkv, block=32, dtype=dtype, seed=max_q, groups=groups)
    case["max_q"] = max_q
    T, S = case["q"].shape[0], len(lens)
    need = pa.attend_workspace_size(S, T, max_q, Hq, Hkv, 128, 32, case["tables"].shape[1], len(groups),
                                    case["prefix_tables"].shape[1])
    out = torch.full_like(case["q"], 7.0).to(DEV)
    run(case, workspace=torch.full((need,), 255, dtype=torch.uint8, device=DEV), out=out)   # (NaN in fp32)
    ref.check(out, case)
    owned = ref.attention(case)[2]
    assert (out.cpu()[~owned] == 7).all()
    assert clean() == _native.DEV_BAD_CONTEXT


@pytest.mark.parametrize("Hq,max_q,new", [(2, 3, [400, 3, 2]), (2, 20, [400, 3, 20]), (24, 20, [400, 20, 7])])
def test_counts_above_max_q_of_scored_calls(Hq, max_q, new):
    case = make([500, 300, 90], new, Hq=Hq, Hkv=2, seed=max_q)
    case["max_q"], case["cap"] = max_q, 9.0
    out = torch.full_like(case["q"], 7.0).to(DEV)
    run(case, out=out)
    ref.check(out, case)
    assert (out.cpu()[~ref.attention(case)[2]] == 7).all()
    assert clean() == _native.DEV_BAD_CONTEXT


# ---- how many bits the weights keep ----------------------------------------------------------

CHUNKS = [dict(lens=[150, 64, 200], new=[40, 64, 3], Hq=8, Hkv=2), dict(lens=[130], new=[130], Hq=2, Hkv=2),
          dict(lens=[300, 257, 90], new=[20, 3, 40], Hq=12, Hkv=2, groups=[(0, 2, 129)]),
          dict(lens=[300, 257, 90], new=[2, 3, 1], Hq=6, Hkv=2, groups=[(0, 3, 80)]),
          dict(lens=[300, 257, 90], Hq=12, Hkv=2, groups=[(0, 3, 80)]),
          dict(lens=[200, 77], Hq=40, Hkv=1)]


@pytest.mark.parametrize("call", range(len(CHUNKS)))
@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("cap", [0.0, 7.0])
def test_weights_keep_their_bits_in_tiles(call, dtype, cap):
    """The bound of the streamed calls (bf16: 2^-16 of a weight) holds for chunks and shared prefixes."""
    case = make(**CHUNKS[call], block=16, dtype=dtype, seed=40 + call)
    if "groups" not in CHUNKS[call]:
        case["cap"], case["slopes"] = cap, slopes_of(CHUNKS[call]["Hq"])
    out = run(case).cpu()
    if case["start"] is None and CHUNKS[call]["Hq"] // CHUNKS[call]["Hkv"] > 32:
        return split_heads(out, case)
    one, rows = as_single_tokens(case)
    ref.check(out[rows], one)


@pytest.mark.parametrize("new", [None, [2, 3]])
def test_weights_keep_their_bits_where_a_prefix_is_not_shared(new):
    """Tables so small that the prefix is read for every sequence."""
    case = make([300, 257], new, Hq=6, Hkv=2, dtype=BF16, seed=47, groups=[(0, 2, 80)], wide=False)
    one, rows = as_single_tokens(case)
    ref.check(run(case).cpu()[rows], one)


def split_heads(out, case):
    """A kv head with more than 32 query heads as two of them, so that the bound is that of few rows."""
    half = case["q"].shape[1] // 2
    for i in range(2):
        part = dict(case, q=case["q"][:, i * half:(i + 1) * half])
        if case.get("slopes") is not None:
            part["slopes"] = case["slopes"][i * half:(i + 1) * half]
        ref.check(out[:, i * half:(i + 1) * half], part)


@pytest.mark.parametrize("kind", ["chunk", "shared", "shared several", "many heads"])
def test_bf16_weights_just_below_one(kind):
    """Half of the tokens have weight 1 and value 1, half weight 1 - 0.45 / 256 and value -1: 8 bits of a weight cannot tell
    them apart, and the result would be zero."""
    new = [64] if kind == "chunk" else [2, 3] if kind == "shared several" else None
    lens = [256] if kind == "chunk" else [256, 256]
    case = make(lens, new, Hq=2 if kind != "many heads" else 40, Hkv=1, dtype=BF16, seed=3,
                groups=[(0, 2, 200)] if "shared" in kind else None)
    gap = -math.log1p(-0.45 / 256)
    case["q"][:] = 1.0
    case["scale"] = gap / 128
    case["k_cache"][:] = 0
    case["k_cache"][:, :, ::2] = 1.0
    case["v_cache"][:] = -1.0
    case["v_cache"][:, :, ::2] = 1.0
    out = run(case).cpu()
    one, rows = as_single_tokens(case)
    if kind == "many heads":
        return split_heads(out, case)
    ref.check(out[rows], one)


@pytest.mark.parametrize("new", [None, [3], [40]])
def test_fp16_weights_far_below_the_largest(new):
    """2000 tokens of weight 22.5 * 2^-29 beside one of weight 1 and value 0: a weight is off by no more than 2^-32, half a
    step of fp16's smallest numbers with the largest weight at 2^7 or more."""
    case = make([2000], new, Hq=2, Hkv=1, block=128, seed=8)
    case["q"][:] = 0.25
    case["k_cache"][:] = 0
    at = (int(case["tables"][0, 3]), 0, 5)
    case["k_cache"][at] = 4.0
    case["scale"] = math.log(2.0 ** 29 / 22.5) / 128
    case["v_cache"][:] = 1.0
    case["v_cache"][at] = 0
    n = 160
    out = run(copies(case, n)).reshape(n, -1, 2, 128).cpu().double()
    tail = torch.arange(2000 - out.shape[1], 2000)[:, None, None].double()
    w = 22.5 * 2.0 ** -29
    want = tail * w / (1 + tail * w)
    # Products and sums of the score are exact (0.25 * 4 * 128), so that its factor's two roundings count, 2^-23 of 24.5 in
    # log2 units: 2^-18 of a weight; the exponential, the sums and the division as in the reference 2^-20; half a step of fp16.
    bound = tail * 2.0 ** -32 + want * (2.0 ** -18 + 2.0 ** -20 + 2.0 ** -11) + 2.0 ** -25
    assert ((out - want).abs() <= bound).all()


# ---- values and scores of any size -----------------------------------------------------------

@pytest.mark.parametrize("kind", ["single", "several", "chunk", "shared", "shared several"])
@pytest.mark.parametrize("cap", [0.0, 1000.0])
@pytest.mark.parametrize("size", [2.0 ** 108, 2.0 ** -80])
@pytest.mark.parametrize("rise", [0.0, 38.0])
def test_values_of_any_size(kind, cap, size, rise):
    """bf16 values of about 2^109 and 2^-80 under scores that grow by 38 (55 in log2 units) along the context, or do not."""
    new = dict(several=[3], chunk=[64]).get(kind, [2, 3] if kind == "shared several" else None)
    shared = "shared" in kind
    if shared and cap:
        return
    case = make([300, 300] if shared else [300], new, Hq=2, Hkv=1, dtype=BF16, seed=6, groups=[(0, 2, 250)] if shared else None)
    case["cap"], case["scale"] = cap, rise / 128
    case["q"][:] = 1.0
    t = torch.arange(300)
    for table, n in [(row, 300) for row in case["tables"]] + [(row, 250) for row in case.get("prefix_tables", [])]:
        case["k_cache"][table.long()[t[:n] // 16], 0, t[:n] % 16] = (t[:n] / 300).bfloat16()[:, None]
    case["v_cache"] = (case["v_cache"].double() * size).bfloat16()
    if shared:
        for s in range(2):                  # the whole last block of the prefix, as its own rows
            n = 250 % 16
            src, dst = int(case["prefix_tables"][0, 15]), int(case["tables"][s, 15])
            case["v_cache"][dst, :, :n] = case["v_cache"][src, :, :n]
    check_copies(case)

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", ["single", "several", "chunk", "shared", "biased", "biased backwards", "capped"])
@pytest.mark.parametrize("scale", [1.0, 1e4, 1e8, 1e12])
def test_scores_of_any_size_row_by_row(dtype, kind, scale):
    """The token with the largest score wins each row where it leads by more than fp32 can lose; elsewhere the result lies
    between the smallest and the largest value."""
    new = {"several": [2, 3], "single": None, "shared": None}.get(kind, [64, 40])
    case = make([700, 333], new, Hq=2, Hkv=2, dtype=dtype, seed=5, size=100.0, groups=[(0, 2, 300)] if kind == "shared" else None)
    case["scale"] = scale
    if "biased" in kind:
        case["slopes"] = torch.tensor([scale, 0.01 * scale]) * (1 if kind == "biased" else -1)
    if kind == "capped":
        case["cap"] = scale * 500
    n = 80
    outs = run(copies(case, n)).reshape(n, *case["q"].shape).cpu().double()
    assert torch.isfinite(outs).all()
    slopes, cap = case.get("slopes"), case.get("cap") or 0.0
    # The winner's weight is rounded for its product (2^-11, bf16 2^-16) and not in the sum; the rest is 700 e^-30; the sums
    # and the division 2^-20; half a step of the result (2^-11, bf16 2^-8).
    rel = 2.0 ** -10 + 2.0 ** -19 if dtype == F16 else 2.0 ** -8 + 2.0 ** -15
    won = 0
    for s in range(2):
        r0, n_new, L = ref.rows_of(case, s)
        t = torch.arange(L)
        blk = case["tables"][s].long()[t // 16]
        p = torch.arange(L - n_new, L)
        for h in range(2):
            K, V = case["k_cache"][blk, h, t % 16].double(), case["v_cache"][blk, h, t % 16].double()
            Q = case["q"][r0:r0 + n_new, h].double()
            z = Q @ K.T * scale
            e = 2.0 ** -16 * (Q.abs() @ K.abs().T) * scale + 2.0 ** -21 * z.abs()      # as in attend_reference.py
            if cap:
                z = cap * torch.tanh(z / cap)
                e = e + 2.0 ** -21 * cap
            if slopes is not None:
                bias = slopes[h].double() * (p[:, None] - t)
                z, e = z - bias, e + 2.0 ** -21 * bias.abs()
            seen = t <= p[:, None]
            best = torch.where(seen, z, -math.inf).argmax(-1, keepdim=True)
            behind = (z - e).gather(-1, best) - (z + e)
            lead = torch.where(seen & (t != best), behind, math.inf).amin(-1)
            for out in (outs[0], outs[n // 2], outs[-1]):
                o = out[r0:r0 + n_new, h]
                lo = torch.where(seen[..., None], V, math.inf).amin(1)
                hi = torch.where(seen[..., None], V, -math.inf).amax(1)
                slack = rel * torch.maximum(lo.abs(), hi.abs())
                assert ((o >= lo - slack) & (o <= hi + slack)).all()
                sure = lead > 30
                won += int(sure.sum())
                want = V[best[:, 0]]
                assert ((o - want).abs() <= rel * want.abs() + 2.0 ** -25)[sure].all()
    assert won > 0 or kind == "capped" or "biased" in kind


@pytest.mark.parametrize("new", [None, [3, 2], [50, 40]])
@pytest.mark.parametrize("cap", [0.0, 30.0])
@pytest.mark.parametrize("shared", [False, True])
def test_keys_of_the_types_lowest_value(new, cap, shared):
    """Scores below fp32's range (here -4e40, of the first 40 tokens) leave no weight."""
    if shared and cap:
        return
    case = make([150, 77], new, Hq=4, Hkv=2, dtype=BF16, seed=21, groups=[(0, 2, 45)] if shared else None)
    case["cap"] = cap
    case["q"] = case["q"].abs() + 0.5
    lowest = torch.finfo(BF16).min
    for s in range(2):
        t = torch.arange(40)
        case["k_cache"][case["tables"][s].long()[t // 16], :, t % 16] = lowest
    if shared:
        case["k_cache"][case["prefix_tables"][0].long()[t // 16], :, t % 16] = lowest
    ref.check(run(case), case)


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("new", [None, [3, 2], [50, 40]])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("cap", [1e-300, 1e-40, 1e-30, 1e-6, 1e6, 1e20, 3e38])
def test_caps_of_any_size(dtype, new, biased, cap):
    """A tiny cap leaves all scores alike, a huge one changes none."""
    case = make([150, 77], new, Hq=4, Hkv=2, dtype=dtype, seed=22)
    case["q"][0, 0] = 0                      # scores of exactly zero, too
    case["cap"] = cap
    if biased:
        case["slopes"] = slopes_of(4)
    out = run(case)
    # the bound's 2^-21 of the cap is what the exponential may lose; at such sizes the cap changes nothing
    ref.check(out, dict(case, cap=cap if cap < 1e4 else 0.0))


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("kind", ["single", "several", "chunk", "shared"])
@pytest.mark.parametrize("size", [0.3, 2.0])
def test_infinite_values_that_every_row_sees(dtype, kind, size):
    """They are infinities of the result, and NaN only where both signs meet or a NaN is among them."""
    new = dict(several=[3, 2], chunk=[70, 40]).get(kind)
    case = make([400, 390], new, Hq=4, Hkv=2, block=32, dtype=dtype, seed=31, size=size,
                groups=[(0, 2, 300)] if kind == "shared" else None)
    values = ((100, 0, 3, math.inf), (150, 1, 7, -math.inf), (151, 1, 9, math.nan), (170, 0, 11, math.inf), (171, 0, 11, -math.inf))
    for s in range(2):
        for at, h, d, x in values:
            case["v_cache"][int(case["tables"][s, at // 32]), h, at % 32, d] = x
    out = run(case)
    ref.check(out, case)
    assert torch.isinf(out).any() and torch.isnan(out).any()


# ---- what a row does not see -----------------------------------------------------------------

OPTIONS = [dict(), dict(cap=9.0), dict(biased=True), dict(cap=9.0, biased=True), dict(scale=3e4), dict(scale=3e4, cap=3e5)]


def with_options(case, cap=0.0, biased=False, scale=None):
    case["cap"] = cap
    if biased:
        case["slopes"] = slopes_of(case["q"].shape[1])
    if scale is not None:
        case["scale"] = scale
    return case


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("new,options", [(n, o) for n in ([8, 5], [16, 9], [70, 40]) for o in range(len(OPTIONS))])
@pytest.mark.parametrize("times", [3.0, -40.0])
def test_what_later_rows_see_changes_no_bit_of_earlier_ones(dtype, new, options, times):
    """The newest token of each sequence, which its last row alone sees, with larger scores."""
    case = with_options(make([150, 77], new, Hq=4, Hkv=2, block=32, dtype=dtype, seed=12), **OPTIONS[options])
    want = run(case)
    for s, L in enumerate([150, 77]):
        at = (int(case["tables"][s, (L - 1) // 32]), slice(None), (L - 1) % 32)
        case["k_cache"][at] *= times
        case["v_cache"][at] *= times
    got = run(case)
    last = torch.tensor([new[0] - 1, sum(new) - 1])
    others = torch.ones(sum(new), dtype=torch.bool)
    others[last] = False
    assert torch.equal(got[others.to(DEV)], want[others.to(DEV)])
    assert not torch.equal(got[last.to(DEV)], want[last.to(DEV)])


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("new", [None, [3, 2], [8, 5], [70, 40]])
@pytest.mark.parametrize("options", range(len(OPTIONS)))
def test_garbage_nobody_sees_changes_no_bit(dtype, new, options):
    """Anything behind the context, before the window, in unused blocks: the same bits."""
    case = with_options(make([150, 77], new, Hq=4, Hkv=2, block=32, dtype=dtype, seed=11), **OPTIONS[options])
    case["first"] = torch.full((case["q"].shape[0],), 40, dtype=torch.int32)
    want = run(case)
    used = torch.zeros(case["k_cache"].shape[0], 32, dtype=torch.bool)
    for s, L in enumerate([150, 77]):
        t = torch.arange(40, L)
        used[case["tables"][s].long()[t // 32], t % 32] = True
    free = ~used
    for bad in (math.nan, math.inf, -math.inf, 60000.0, -300.0, 0.0):
        for cache in ("k_cache", "v_cache"):
            x = case[cache].permute(0, 2, 1, 3).clone()
            x[free] = bad
            case[cache] = x.permute(0, 2, 1, 3).contiguous()
        assert torch.equal(run(case), want), bad
    assert all(torch.equal(run(case), want) for _ in range(5))


@pytest.mark.parametrize("dtype", [F16, BF16])
def test_garbage_behind_shared_prefixes_changes_no_bit(dtype):
    case = make([150, 77, 300], Hq=12, Hkv=2, block=32, dtype=dtype, seed=13, groups=[(0, 3, 70)])
    want = run(case)
    used = torch.zeros(case["k_cache"].shape[0], 32, dtype=torch.bool)
    for s, L in enumerate([150, 77, 300]):
        t = torch.arange(L)
        used[case["tables"][s].long()[t // 32], t % 32] = True
    t = torch.arange(70)
    used[case["prefix_tables"][0].long()[t // 32], t % 32] = True
    for bad in (math.nan, math.inf, 60000.0, 0.0):
        for cache in ("k_cache", "v_cache"):
            x = case[cache].permute(0, 2, 1, 3).clone()
            x[~used] = bad
            case[cache] = x.permute(0, 2, 1, 3).contiguous()
        assert torch.equal(run(case), want), bad


# ---- many query heads a kv head --------------------------------------------------------------

@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("Hq,Hkv,block", [(40, 1, 16), (66, 2, 64), (300, 1, 128)])
@pytest.mark.parametrize("cap,biased,span", [(0.0, False, 0), (5.0, True, 0), (0.0, True, 30), (2.0, False, 30)])
def test_more_than_32_query_heads_a_kv_head(dtype, Hq, Hkv, block, cap, biased, span):
    """Single tokens in tiles."""
    case = make([1, 0, 7, 64, 65, 255, 700, 33], Hq=Hq, Hkv=Hkv, block=block, dtype=dtype, seed=Hq)
    case["cap"] = cap
    if biased:
        case["slopes"] = slopes_of(Hq)
    if span:
        case["first"] = window(case, span)
        case["first"][3] = 10**9
    out = run(case)
    ref.check(out, case)
    assert not out[1].any() and (not span or not out[3].any())
    assert clean() == 0


@pytest.mark.parametrize("dtype", [F16, BF16])
@pytest.mark.parametrize("wide", [False, True])
def test_more_than_32_query_heads_share_a_prefix(dtype, wide):
    case = make([90, 0, 300, 64, 500, 41], Hq=80, Hkv=2, block=16, dtype=dtype, seed=2, groups=[(0, 2, 64), (2, 5, 130)],
                wide=wide)
    ref.check(run(case), case)
    assert clean() == 0
