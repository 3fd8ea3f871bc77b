"""Rotary positions on the GPU against the formula in 64 bits with exactly reduced angles."""
import numpy as np
import pytest
import torch

import paged_kv_cache_08_gb300 as pa
import q8_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


def _inputs(T, Hq, Hkv, D, dtype, seed, far=4096, fused=False):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=gen).to(dtype).to(DEV)
    if fused:      # slices of one projection's output
        q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    else:
        q, k = x[:, :Hq].contiguous(), x[:, Hq:Hq + Hkv].contiguous()
    return q, k, torch.randint(0, far, (T,), generator=gen)


def _check(got, x, positions, inv_freq, magnitude, interleaved):
    want, bound = ref.rope(ref.f64(x), positions.tolist(), inv_freq.tolist(), magnitude, interleaved)
    R = 2 * len(inv_freq)
    y = ref.f64(got)
    assert np.array_equal(y[..., R:], want[..., R:])
    excess = np.abs(y - want)[..., :R] - (bound + ref.half_step(np.abs(want) + bound, got.dtype))[..., :R]
    assert excess.size == 0 or excess.max() <= 0, f"beyond the bound by {excess.max():.3e}"


@pytest.mark.parametrize("T,Hq,Hkv,D,R", [(1, 12, 2, 128, 128), (5, 1, 1, 128, 16), (64, 12, 2, 128, 64),
                                          (7, 8, 8, 128, 96), (3, 5, 1, 64, 64), (33, 4, 2, 80, 32),
                                          (2, 3, 3, 256, 256), (200, 32, 8, 128, 128), (1, 1, 1, 1024, 1024),
                                          (9, 20, 4, 24, 16)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rope(T, Hq, Hkv, D, R, dtype, interleaved):
    q, k, pos = _inputs(T, Hq, Hkv, D, dtype, seed=T * 7 + R)
    f, m = pa.rope_frequencies(R)
    oq, ok = pa.rope(q, k, pos.to(DEV), f, interleaved=interleaved)
    torch.cuda.synchronize()
    _check(oq, q, pos, f, m, interleaved)
    _check(ok, k, pos, f, m, interleaved)


@pytest.mark.parametrize("scaling", ["linear", "ntk", "yarn"])
def test_rope_far_positions(scaling):
    q, k, _ = _inputs(24, 4, 1, 128, torch.float16, seed=3)
    f, m = pa.rope_frequencies(128, scaling=scaling, factor=32.0, original_context=4096)
    pos = torch.tensor([0, 1, -1, 4095, 131071, 131072, 999999, 1000001, -1000003, 2**24 + 1, 2**31 - 1, -2**31,
                        2**31 + 5, 2**33 + 7] + [10007 * i * i for i in range(10)])
    oq, ok = pa.rope(q, k, pos.to(DEV), f, magnitude=m)
    torch.cuda.synchronize()
    _check(oq, q, pos, f, m, False)
    _check(ok, k, pos, f, m, False)


def test_rope_int32_positions_and_any_frequency():
    q, k, _ = _inputs(40, 2, 2, 128, torch.bfloat16, seed=5)
    gen = torch.Generator().manual_seed(6)
    f = torch.randn(24, generator=gen, dtype=torch.float64) * 20       # above a turn per position, negative too
    f[0], f[1], f[2] = 0.0, 2 * np.pi, -1e-12
    pos = torch.randint(-(2**31), 2**31 - 1, (40,), generator=gen)
    pos[0] = 0
    oq, ok = pa.rope(q, k, pos.to(torch.int32).to(DEV), f.to(DEV), magnitude=-0.5, interleaved=True)
    torch.cuda.synchronize()
    _check(oq, q, pos, f, -0.5, True)
    _check(ok, k, pos, f, -0.5, True)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("R", [48, 128])
def test_rope_in_place_on_a_fused_projection(interleaved, R):
    T, Hq, Hkv, D = 37, 12, 2, 128
    gen = torch.Generator().manual_seed(9)
    x = torch.randn((T, Hq + 2 * Hkv, D), generator=gen).to(torch.float16).to(DEV)
    before = x.clone()
    q, k = x[:, :Hq], x[:, Hq:Hq + Hkv]
    pos = torch.randint(0, 5000, (T,), generator=gen)
    f, m = pa.rope_frequencies(R)
    oq, ok = pa.rope(q, k, pos.to(DEV), f, interleaved=interleaved, out_q=q, out_k=k)
    torch.cuda.synchronize()
    assert oq is q and ok is k
    _check(q, before[:, :Hq], pos, f, m, interleaved)
    _check(k, before[:, Hq:Hq + Hkv], pos, f, m, interleaved)
    assert torch.equal(x[:, Hq + Hkv:], before[:, Hq + Hkv:])
    # the same out of place, from the slices
    oq, ok = pa.rope(before[:, :Hq], before[:, Hq:Hq + Hkv], pos.to(DEV), f, interleaved=interleaved)
    assert torch.equal(oq, q) and torch.equal(ok, k)


def test_rope_without_k_and_without_tokens():
    q, _, pos = _inputs(6, 3, 1, 128, torch.float16, seed=11)
    f, m = pa.rope_frequencies(64)
    oq, ok = pa.rope(q, None, pos.to(DEV), f)
    torch.cuda.synchronize()
    assert ok is None
    _check(oq, q, pos, f, m, False)
    oq, ok = pa.rope(q[:0], q[:0], pos[:0].to(DEV), f)
    assert oq.shape == (0, 3, 128) and ok.shape == (0, 3, 128)


def test_rope_keeps_infinities_and_nan_in_their_pairs():
    q, k, pos = _inputs(4, 2, 1, 128, torch.float16, seed=13)
    q[1, 0, 3], q[2, 1, 100] = float("inf"), float("nan")
    f, m = pa.rope_frequencies(96)
    oq, _ = pa.rope(q, k, pos.to(DEV), f)
    torch.cuda.synchronize()
    bad = ~torch.isfinite(oq).cpu()
    want = torch.zeros_like(bad)
    want[1, 0, 3] = want[1, 0, 3 + 48] = want[2, 1, 100] = True
    assert torch.equal(bad, want)


def test_rope_on_a_stream_and_in_a_graph():
    q, k, pos = _inputs(64, 12, 2, 128, torch.bfloat16, seed=15)
    p = pos.to(DEV)
    f, m = pa.rope_frequencies(128)
    want = pa.rope(q, k, p, f)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = pa.rope(q, k, p, f, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = pa.rope(q, k, p, f)
    p.add_(17)
    g.replay()
    torch.cuda.synchronize()
    _check(out[0], q, pos + 17, f, m, False)


def test_rope_every_way_to_call_gives_the_same():
    q, k, pos = _inputs(21, 12, 2, 128, torch.float16, seed=19, fused=True)
    p = pos.to(DEV)
    f, m = pa.rope_frequencies(64)
    want = pa.rope(q, k, p, f)
    _check(want[0], q, pos, f, m, False)
    assert want[0].is_contiguous() and want[1].is_contiguous()
    got = [pa.rope(q, k, p, f, stream=torch.cuda.current_stream()), pa.rope(q, k, p.int(), f),
           pa.rope(torch.nn.Parameter(q, requires_grad=False), k, p, f),
           (pa.rope(q, None, p, f)[0], pa.rope(k, None, p, f)[0])]
    outs = torch.empty((21, 14, 128), dtype=torch.float16, device=DEV)
    pa.rope(q, k, p, f, out_q=outs[:, :12], out_k=outs[:, 12:])
    torch.cuda.synchronize()
    for a, b in got + [(outs[:, :12], outs[:, 12:])]:
        assert torch.equal(a, want[0]) and torch.equal(b, want[1])


def test_rope_beyond_32_bit_offsets():
    T, H = 530000, 32                                 # 2.17e9 elements
    x = torch.zeros((T, H, 128), dtype=torch.bfloat16, device=DEV)
    gen = torch.Generator(device=DEV).manual_seed(21)
    x[-3:] = torch.randn((3, H, 128), generator=gen, device=DEV)
    pos = torch.arange(T, device=DEV)
    f, m = pa.rope_frequencies(128)
    before = x[-3:].clone()
    pa.rope(x, None, pos, f, out_q=x)
    torch.cuda.synchronize()
    _check(x[-3:], before, pos[-3:].cpu(), f, m, False)
    assert not x[:-3].any()


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_of_the_widest_head_and_many_tokens(interleaved):
    """Several tokens of a CTA, whose cosines and sines fill what shared memory it may have."""
    q, k, pos = _inputs(12500, 1, 1, 1024, torch.bfloat16, seed=21)
    f, m = pa.rope_frequencies(1024)
    oq, ok = pa.rope(q, k, pos.to(DEV), f, interleaved=interleaved)
    torch.cuda.synchronize()
    for at in (slice(0, 40), slice(6230, 6270), slice(12460, 12500)):
        _check(oq[at], q[at], pos[at], f, m, interleaved)
        _check(ok[at], k[at], pos[at], f, m, interleaved)


def test_rope_refuses():
    q, k, pos = _inputs(4, 2, 1, 128, torch.float16, seed=17)
    p = pos.to(DEV)
    f, _ = pa.rope_frequencies(128)
    for call, error in ((lambda: pa.rope(q.float(), None, p, f), TypeError),
                        (lambda: pa.rope(q, k.bfloat16(), p, f), TypeError),
                        (lambda: pa.rope(q, k, p.float(), f), TypeError),
                        (lambda: pa.rope(q, k, p, f.float()), TypeError),
                        (lambda: pa.rope(q, k[:2], p, f), ValueError),
                        (lambda: pa.rope(q, k, p[:3], f), ValueError),
                        (lambda: pa.rope(q.transpose(0, 1), None, p[:2], f), ValueError),
                        (lambda: pa.rope(q[:, :, ::2], None, p, f), ValueError),
                        (lambda: pa.rope(q, None, p, f, out_k=k), ValueError),
                        (lambda: pa.rope(q, k, p, f, out_q=k), ValueError),
                        (lambda: pa.rope(q, k, p, f[:60].contiguous()), pa.PAError),      # 120 = no multiple of 16
                        (lambda: pa.rope(q, q, p, f, out_q=q, out_k=q), pa.PAError),      # two outputs in one place
                        (lambda: pa.rope(q, k, p, torch.ones(72, dtype=torch.float64, device=DEV)), pa.PAError)):
        with pytest.raises(error):
            call()
