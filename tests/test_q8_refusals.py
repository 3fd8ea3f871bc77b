"""Rotary positions and the 8-bit cache without a GPU: the C ABI refuses bad arguments before any CUDA
call, the binding refuses tensors that are not what it takes, the frequencies follow their formulas, and
the 64-bit reference agrees with torch's e4m3."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_08_gb300 as pa
import q8_reference as ref
from paged_kv_cache_08_gb300 import _native

E = {v: k for k, v in _native.STATUS.items()}
BAD, UNSUPPORTED, WORKSPACE = E["PA_ERR_INVALID_ARG"], E["PA_ERR_UNSUPPORTED"], E["PA_ERR_WORKSPACE"]


@pytest.fixture(scope="module")
def lib():
    return _native.load()


def _rope(lib, **kw):
    # far apart, so that nothing overlaps unless a case says so
    a = dict(oq=1 << 30, ok=2 << 30, q=3 << 30, k=4 << 30, oqs=1536, oks=256, qs=1536, ks=256, pos=64, pb=8, f=64, m=1.0,
             T=4, hq=12, hkv=2, d=128, r=128, inter=0, dtype=0)
    a.update(kw)
    return lib.pa_rope(*a.values(), None)


def test_rope_rejects_before_launch(lib):
    assert _rope(lib, T=0) == 0
    for kw in (dict(dtype=2), dict(pb=2), dict(T=-1), dict(hq=0), dict(hkv=-1), dict(d=0), dict(r=0), dict(r=144),
               dict(q=None), dict(oq=None), dict(k=None), dict(ok=None), dict(pos=None), dict(f=None),
               dict(q=(3 << 30) + 8), dict(oq=(1 << 30) + 2), dict(k=(4 << 30) + 4), dict(pos=68, pb=8), dict(f=68),
               dict(qs=1540), dict(oqs=1528), dict(oks=128), dict(ks=-256), dict(qs=-8), dict(oks=260)):
        assert _rope(lib, **kw) == BAD, kw
    for kw in (dict(d=132, r=128), dict(r=24), dict(r=8), dict(d=1032, r=1024)):
        assert _rope(lib, **kw) == UNSUPPORTED, kw


def test_rope_rejects_overlaps(lib):
    q = 3 << 30
    row = 1536 * 2
    assert _rope(lib, oq=q + 16) == BAD                             # shifted onto itself
    assert _rope(lib, oq=q, oqs=2048) == BAD                        # another stride in place
    assert _rope(lib, ok=q) == BAD                                  # k's output over q
    assert _rope(lib, oq=4 << 30) == BAD                            # q's output over k
    assert _rope(lib, oq=1 << 30, ok=(1 << 30) + row - 16) == BAD   # outputs over one another
    # one projection's output, [q | k | v] per token, with k begun inside q
    assert _rope(lib, q=q, k=q + row - 16, oq=q, ok=q + row - 16, qs=2048, ks=2048, oqs=2048, oks=2048) == BAD


def _append(lib, **kw):
    a = dict(k=16, v=16, ks=256, vs=256, kc=16, vc=16, ke=16, ve=16, bt=16, cl=16, qs=16, S=2, T=4, mq=2, hkv=2, d=128,
             b=16, nb=4, maxb=4, dtype=0)
    a.update(kw)
    return lib.pa_cache_append_q8(*a.values(), None)


def test_append_rejects_before_launch(lib):
    assert _append(lib, T=0) == 0
    assert _append(lib, S=0, T=0) == 0
    for kw in (dict(dtype=-1), dict(T=-1), dict(mq=0), dict(S=-1), dict(hkv=0), dict(nb=0), dict(maxb=-1),
               dict(qs=None), dict(k=None), dict(v=None), dict(kc=None), dict(vc=None), dict(ke=None), dict(ve=None),
               dict(bt=None), dict(cl=None), dict(k=24), dict(v=8), dict(kc=24), dict(vc=17), dict(bt=18), dict(cl=17),
               dict(qs=18), dict(ks=252), dict(vs=-8), dict(b=0)):
        assert _append(lib, **kw) == BAD, kw
    for kw in (dict(d=64), dict(b=8), dict(b=48), dict(S=70000), dict(maxb=1 << 27), dict(nb=1 << 27),
               dict(T=1 << 30, hkv=64, nb=4)):
        assert _append(lib, **kw) == UNSUPPORTED, kw


def _read(lib, **kw):
    a = dict(kc=16, vc=16, ke=16, ve=16, ns=4, dk=16, dv=16, nd=4, src=16, dst=16, n=2, hkv=2, d=128, b=16, dtype=0)
    a.update(kw)
    return lib.pa_read_blocks_q8(*a.values(), None)


def test_read_rejects_before_launch(lib):
    assert _read(lib, n=0) == 0
    for kw in (dict(dtype=3), dict(n=-1), dict(nd=-1), dict(ns=0), dict(hkv=0), dict(kc=None), dict(vc=None),
               dict(ke=None), dict(ve=None), dict(dk=None), dict(dv=None), dict(src=None), dict(dst=None), dict(kc=20),
               dict(dv=24), dict(src=18), dict(dst=17)):
        assert _read(lib, **kw) == BAD, kw
    for kw in (dict(d=96), dict(b=24), dict(ns=1 << 27)):
        assert _read(lib, **kw) == UNSUPPORTED, kw


def _decode(lib, **kw):
    a = dict(out=16, q=16, kc=16, vc=16, ke=16, ve=16, bt=16, cl=16, scale=0.1, hkv=2, S=1, hq=12, d=128, b=16, nb=4,
             maxb=4, dtype=0, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_decode_q8(*a.values(), None)


def _multi(lib, **kw):
    a = dict(out=16, q=16, kc=16, vc=16, ke=16, ve=16, bt=16, cl=16, qs=16, scale=0.1, hkv=2, S=1, T=2, mq=2, hq=12,
             d=128, b=16, nb=4, maxb=4, dtype=0, ws=None, wsb=0)
    a.update(kw)
    return lib.pa_multi_query_q8(*a.values(), None)


@pytest.mark.parametrize("call", [_decode, _multi])
def test_attention_rejects_before_launch(lib, call):
    for kw in (dict(dtype=7), dict(hq=13), dict(hq=0), dict(hkv=0), dict(S=-1), dict(nb=0), dict(out=None), dict(q=None),
               dict(kc=None), dict(vc=None), dict(ke=None), dict(ve=None), dict(bt=None), dict(cl=None), dict(out=24),
               dict(q=8), dict(kc=24), dict(vc=2), dict(bt=18), dict(cl=17), dict(maxb=-1)):
        assert call(lib, **kw) == BAD, kw
    for kw in (dict(d=64), dict(b=256), dict(hq=66), dict(S=70000), dict(maxb=1 << 27), dict(nb=1 << 27)):
        assert call(lib, **kw) == UNSUPPORTED, kw
    assert call(lib, S=0) == 0


def test_several_rows_reject_before_launch(lib):
    for kw in (dict(qs=None), dict(qs=18), dict(mq=0), dict(T=-1)):
        assert _multi(lib, **kw) == BAD, kw
    assert _multi(lib, mq=6) == UNSUPPORTED            # 6 x 6 rows per kv head
    assert _multi(lib, T=0) == 0


def test_workspace_size_is_zero_for_shapes_without_a_kernel(lib):
    size = lib.pa_decode_q8_workspace_size
    assert size(64, 66, 2, 128, 16, 128, 1) == 0
    assert size(64, 12, 2, 64, 16, 128, 1) == 0
    assert size(64, 12, 2, 128, 16, 128, 6) == 0
    need = size(64, 12, 2, 128, 16, 128, 1)
    if need:
        args = dict(S=64, maxb=128)
        assert _decode(lib, **args) == WORKSPACE                              # missing
        assert _decode(lib, **args, ws=16, wsb=need - 1) == WORKSPACE         # short
        assert _decode(lib, **args, ws=24, wsb=need) == WORKSPACE             # misaligned


def test_the_binding_refuses_host_tensors():
    h = torch.zeros((4, 2, 128), dtype=torch.float16)
    c = torch.zeros((4, 2, 16, 128), dtype=torch.float8_e4m3fn)
    e = torch.zeros((4, 2), dtype=torch.int8)
    i = torch.zeros((4, 4), dtype=torch.int32)
    for call in (lambda: pa.rope(h, None, torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.float64)),
                 lambda: pa.cache_append_q8(h, h, c, c, e, e, i, i[0]),
                 lambda: pa.read_blocks_q8(c, c, e, e, h, h, i[0], i[0]),
                 lambda: pa.decode_q8(h, c, c, e, e, i, i[0], 0.1, 2),
                 lambda: pa.multi_query_q8(h, c, c, e, e, i, i[0], i[0], 0.1, 2, 1),
                 lambda: pa.multi_query_q8(h, c, c, e, e, i, i[0], None, 0.1, 2, 1)):
        with pytest.raises(TypeError):
            call()


# ---- frequencies ---------------------------------------------------------------------------

def test_frequencies_follow_their_formulas():
    f, m = pa.rope_frequencies(128, device="cpu")
    assert m == 1.0 and f.dtype == torch.float64
    assert np.allclose(f.numpy(), [10000.0 ** (-2 * i / 128) for i in range(64)], rtol=1e-15)
    g, m = pa.rope_frequencies(64, base=5e5, scaling="linear", factor=4.0, device="cpu")
    assert m == 1.0 and np.allclose(g.numpy(), [5e5 ** (-2 * i / 64) / 4 for i in range(32)], rtol=1e-15)
    # ntk: the fastest pair is unchanged, the slowest is slowed by the factor
    f, _ = pa.rope_frequencies(96, device="cpu")
    g, _ = pa.rope_frequencies(96, scaling="ntk", factor=8.0, device="cpu")
    assert g[0] == 1.0 and math.isclose(float(f[-1] / g[-1]), 8.0, rel_tol=1e-12)


def test_yarn_keeps_fast_pairs_and_slows_slow_ones():
    R, base, trained, factor = 128, 10000.0, 4096, 32.0
    f, _ = pa.rope_frequencies(R, base, device="cpu")
    g, m = pa.rope_frequencies(R, base, scaling="yarn", factor=factor, original_context=trained, device="cpu")
    assert math.isclose(m, 1.0 + 0.1 * math.log(factor))
    turns = (trained * f / (2 * math.pi)).numpy()
    ratio = (g / f).numpy()
    # a pair's distance from the ramp's ends is at most the rounding to whole pairs
    step = base ** (2.0 / R)
    assert np.allclose(ratio[turns > 32.0 * step], 1.0, rtol=1e-12)
    assert np.allclose(ratio[turns < 1.0 / step], 1 / factor, rtol=1e-12)
    assert (np.diff(ratio) <= 1e-15).all()
    ramp = (ratio > 1 / factor + 1e-9) & (ratio < 1 - 1e-9)
    assert np.ptp(np.diff(ratio[ramp])) < 1e-12                 # linear in the pair's index


@pytest.mark.parametrize("kw", [dict(rotary_dim=0), dict(rotary_dim=7), dict(base=1.0), dict(factor=0.5),
                                dict(scaling="other"), dict(scaling="yarn", factor=2.0),
                                dict(rotary_dim=2, scaling="ntk", factor=2.0),
                                dict(scaling="yarn", original_context=64, beta_fast=1.0)])
def test_frequencies_refuse(kw):
    with pytest.raises(ValueError):
        pa.rope_frequencies(**{"rotary_dim": 64, "device": "cpu", **kw})


# ---- the reference -------------------------------------------------------------------------

def test_reference_codes_are_e4m3():
    every = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(every, ref.CODE_VALUES, equal_nan=True)
    x = np.concatenate([np.linspace(-448, 448, 100001), 2.0 ** np.linspace(-14, 8.8, 20001),
                        (ref.CODE_VALUES[:126] + ref.CODE_VALUES[1:127]) / 2, [0.0, -0.0]])
    x = x.astype(np.float32)
    got = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(ref.to_code(x), got)
    assert ref.to_code(np.array([np.inf, -np.inf, 1e9])).tolist() == [0x7E, 0xFE, 0x7E]


def test_reference_exponent_is_the_least():
    assert ref.exponent_for(np.array([448.0])) == 0
    assert ref.exponent_for(np.array([448.5])) == 1
    assert ref.exponent_for(np.array([1.75])) == -8
    assert ref.exponent_for(np.array([0.0, np.nan])) == -60
    assert ref.exponent_for(np.array([np.inf, 7.0])) == -6
    assert ref.exponent_for(np.array([1e38])) == 60
