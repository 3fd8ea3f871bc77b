"""Small softmax weights beside a large one in the attention over the 8-bit cache: they enter the product with V in fp16,
so far below the row's largest they are subnormal there, and what is left of them has to carry contexts of many tokens."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_08_gb300 as pa
import q8_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
# A weight times its block's scale is held to 11 bits from 2^-23 of the row's largest on, below that in steps of 2^-33:
# the largest lies at 2^9 of fp16 at least, whose normal numbers begin at 2^-14 and whose steps below are 2^-24.
STEP = 2.0 ** -33


def _expect(q, kc, vc, ks, vs, scale):
    """(out, bound) of query rows [R, D] over codes' values kc, vc [L, D] and the scales ks, vs [L] of their blocks: the
    bound's terms are q8_reference.attention's, with the weights' step as above."""
    qk = q @ kc.T
    score = qk * ks * scale
    w = np.exp(score - score.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    ds = 132 * 2.0 ** -24 * (np.abs(q) @ np.abs(kc).T * ks * abs(scale)).max(-1, keepdims=True)
    rel = 2.0 ** -11 + 2 * ds + 2.0 ** -20 + (len(kc) / 16 + 64) * 2.0 ** -22
    small = STEP / 2 * np.abs(vc).sum(0) * (w * vs).max(-1, keepdims=True)
    return (w * vs) @ vc, rel * ((w * vs) @ np.abs(vc)) + small


@pytest.mark.parametrize("at", [0, 70000, 131069])
@pytest.mark.parametrize("group,new", [(1, 0), (6, 0), (4, 4), (8, 3)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_a_sink_over_a_long_context(dtype, group, new, at):
    """One token takes e^16 times the weight of each of the 131,071 others, 98.5 % of all, and has a small value.  In the
    first head the others' scores are alike, so that the weights' roundings do not cancel, in the others they differ.
    A thousand sequences share the context's blocks: then most of a context, or all, lies in one warp's share."""
    L, S, block = 131072, 1000, 64
    rng = np.random.default_rng(at + group)
    nb = L // block
    ids = rng.permutation(nb)
    k = ref.to_code(0.25 * rng.standard_normal((L, ref.D)))
    k[:, 0] = 0
    k[at] = 0
    k[at, 0] = ref.to_code(np.array(16.0))
    v = ref.to_code(rng.uniform(0.5, 2.0, (L, ref.D)))       # of one sign: no sum cancels
    v[at] = ref.to_code(np.array(2.0 ** -6))
    rows = max(1, new)
    q = torch.from_numpy(0.3 * rng.standard_normal((rows, group, ref.D))).to(dtype)
    q[:, :, 0] = 1.0
    q[:, 0, 1:] = 0

    def pool(c):
        blocks = np.empty((nb, 1, block, ref.D), dtype=np.uint8)
        blocks[ids] = c.reshape(nb, 1, block, ref.D)
        return torch.from_numpy(blocks).to(DEV).view(torch.float8_e4m3fn)

    exps = [torch.zeros((nb, 1), dtype=torch.int8, device=DEV) for _ in range(2)]
    args = [q.repeat(S, 1, 1).to(DEV), pool(k), pool(v), *exps,
            torch.from_numpy(ids[None].astype(np.int32)).to(DEV).repeat(S, 1),
            torch.full((S,), L - 1, dtype=torch.int32, device=DEV)]      # the last block's last row is no token
    if new:
        out = pa.multi_query_q8(*args, new * torch.arange(S + 1, dtype=torch.int32, device=DEV), 1.0, 1, new)
    else:
        out = pa.decode_q8(*args, 1.0, 1)
    torch.cuda.synchronize()
    assert pa.read_device_status(clear=True) == 0
    got, kv, vv = ref.f64(out).reshape(S, rows, group, ref.D), ref.CODE_VALUES[k], ref.CODE_VALUES[v]
    for i in range(rows):
        n = L - 1 - (rows - 1 - i)
        want, bound = _expect(ref.f64(q[i]), kv[:n], vv[:n], np.ones(n), np.ones(n), 1.0)
        excess = np.abs(got[:, i] - want) - (bound + ref.half_step(np.abs(want) + bound, dtype))
        assert excess.max() <= 0, f"beyond the bound by {excess.max():.3e}, values from {np.abs(want).min():.3e}"


@pytest.mark.parametrize("scale", [1.0, 40.0])
def test_weights_at_the_top_of_their_range(scale):
    """Scores that climb from token to token, so that the largest weight of a tile comes near the point where the base
    moves, and by steps of several bits: nothing overflows."""
    L, block = 4096, 16
    rng = np.random.default_rng(7)
    nb = L // block
    climb = np.linspace(0, 440, L) + rng.uniform(0, 8, L)
    k = np.zeros((L, ref.D), dtype=np.uint8)
    k[:, 0] = ref.to_code(climb)
    v = ref.to_code(rng.standard_normal((L, ref.D)) * 200)
    q = torch.zeros((1, 8, ref.D), dtype=torch.float16)
    q[0, :, 0] = torch.linspace(0.01, 1.0, 8)
    pool = lambda c: torch.from_numpy(c.reshape(nb, 1, block, ref.D)).to(DEV).view(torch.float8_e4m3fn)  # noqa: E731
    e = rng.integers(-20, 20, (2, nb, 1)).astype(np.int8)
    e[0] = 0
    out = pa.decode_q8(q.to(DEV), pool(k), pool(v), *(torch.from_numpy(x).to(DEV) for x in e),
                       torch.arange(nb, dtype=torch.int32, device=DEV)[None], torch.tensor([L], dtype=torch.int32, device=DEV),
                       scale, 1)
    torch.cuda.synchronize()
    vs = np.repeat(np.exp2(e[1, :, 0].astype(np.float64)), block)
    want, bound = _expect(ref.f64(q[0]), ref.CODE_VALUES[k], ref.CODE_VALUES[v], np.ones(L), vs, scale)
    ref.check_attention(out, want[None], bound[None], np.ones(1, dtype=bool))
    assert math.isfinite(float(out.float().abs().max())) or (np.abs(want) > 65504).any()


@pytest.mark.parametrize("log2_top", [20, 23, 24, 25, 26, 27])
@pytest.mark.parametrize("v_exp", [-20, 0, 14])
@pytest.mark.parametrize("dtype,new", [(torch.float16, 0), (torch.bfloat16, 0), (torch.float16, 3)])
def test_scores_too_large_for_their_differences(dtype, new, v_exp, log2_top):
    """Scores of 2^20 to 2^27 that differ by a few units: fp32 holds their differences in steps of up to 16, so that the
    weights are nobody's to say, but every output is a mean of V's values, which lie in [1, 1.875] x 2^v_exp."""
    L, block = 1500, 16
    nb = -(-L // block)
    rng = np.random.default_rng(log2_top)
    k = np.zeros((nb * block, ref.D), dtype=np.uint8)
    k[:, 0] = ref.to_code(np.array(256.0))
    k[:, 1] = ref.to_code(np.linspace(0, 400, nb * block))          # climbing differences
    k[:, 2] = ref.to_code(rng.uniform(-16, 16, nb * block))
    v = ref.to_code(rng.integers(8, 16, (nb * block, ref.D)) / 8.0)
    rows = max(1, new)
    q = torch.zeros((rows, 5, ref.D), dtype=dtype)
    q[:, :, 0] = 2.0 ** 10
    q[:, :, 1:3] = torch.tensor([0.25, 0.5, 1.0, 2.0, 4.0])[:, None] * 2.0 ** (18 - log2_top)
    scale = 2.0 ** (log2_top - 18)
    pool = lambda c: torch.from_numpy(c.reshape(nb, 1, block, ref.D)).to(DEV).view(torch.float8_e4m3fn)  # noqa: E731
    exps = [torch.full((nb, 1), e, dtype=torch.int8, device=DEV) for e in (0, v_exp)]
    args = [q.to(DEV), pool(k), pool(v), *exps, torch.arange(nb, dtype=torch.int32, device=DEV)[None],
            torch.tensor([L], dtype=torch.int32, device=DEV)]
    if new:
        out = pa.multi_query_q8(*args, torch.tensor([0, new], dtype=torch.int32, device=DEV), scale, 1, new)
    else:
        out = pa.decode_q8(*args, scale, 1)
    torch.cuda.synchronize()
    y = ref.f64(out) * 2.0 ** -v_exp
    # a weight's rounding to fp16 (2^-11 of it, or a step below 2^-14 beside a largest one of 2^(9 - 16) at least) and
    # the output's own (2^-8 in bf16, in fp16's subnormals 2^-25 x 2^20)
    assert np.isfinite(y).all()
    assert y.min() >= 1 - 2.0 ** -4 and y.max() <= 1.875 + 2.0 ** -4
