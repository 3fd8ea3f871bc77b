"""Attention with other scores, masks and shared prefixes at the edges of what its calls may be given, on the GPU
against the definition in 64 bits."""
import pytest
import torch

import attend_reference as ref
import paged_kv_cache_08_gb300 as pa
from paged_kv_cache_08_gb300 import _native
from test_gpu_attend import BF16, DEV, F16, clean, make, run, status  # noqa: F401 (status: every test's)

pytestmark = pytest.mark.gpu


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
