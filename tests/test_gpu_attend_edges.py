"""Attention with other scores, masks and shared prefixes at the edges of what its calls may be given, on the GPU
against the definition in 64 bits."""
import math

import pytest
import torch

import attend_reference as ref
import paged_kv_cache_08_gb300 as pa
from paged_kv_cache_08_gb300 import _native
from test_gpu_attend import BF16, DEV, F16, clean, make, run, slopes_of, status  # noqa: F401 (status: every test's)

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
