"""The binding's C part (csrc/marshal.c) without a GPU: built against a stand-in of the library that records its calls, on
host tensors that answer as if they lay on device 0.  What reaches the library are the tensors' own addresses, and a call
with a tensor that has none to give (a batched one inside torch.vmap) goes to the Python code."""
import ctypes
import importlib.machinery
import importlib.util
import shutil
import subprocess
import sysconfig
from pathlib import Path

import numpy as np
import pytest
import torch

import paged_kv_cache_08_gb300 as pa
from paged_kv_cache_08_gb300 import _native, build

ROOT = Path(__file__).resolve().parent.parent
STAND_IN = """
#include "pa.h"
int calls;
uintptr_t seen[16];
static int called(int n, const void *const *p) {
    ++calls;
    for (int i = 0; i < 16; ++i) seen[i] = i < n ? (uintptr_t)p[i] : 0;
    return PA_OK;
}
#define CALLED(...) do { const void *p[] = {__VA_ARGS__}; return called((int)(sizeof p / sizeof *p), p); } while (0)
int pa_rope(void *oq, void *ok, const void *q, const void *k, long long a, long long b, long long c, long long d,
            const void *pos, int pb, const double *f, float m, int T, int hq, int hkv, int D, int R, int in, int dt, void *s) {
    CALLED(q, k, pos, f, oq, ok);
}
int pa_cache_append_q8(const void *k, const void *v, long long ks, long long vs, void *kc, void *vc, int8_t *ke, int8_t *ve,
                       const int32_t *bt, const int32_t *cl, const int32_t *qs, int S, int T, int mq, int hkv, int D, int B,
                       int nb, int mb, int dt, void *s) {
    CALLED(k, v, kc, vc, ke, ve, bt, cl, qs);
}
int pa_read_blocks_q8(const void *kc, const void *vc, const int8_t *ke, const int8_t *ve, int ns, void *dk, void *dv, int nd,
                      const int32_t *src, const int32_t *dst, int n, int hkv, int D, int B, int dt, void *s) {
    CALLED(kc, vc, ke, ve, dk, dv, src, dst);
}
int pa_decode_q8(void *o, const void *q, const void *kc, const void *vc, const int8_t *ke, const int8_t *ve,
                 const int32_t *bt, const int32_t *cl, float sc, int hkv, int S, int hq, int D, int B, int nb, int mb, int dt,
                 void *w, size_t wb, void *s) {
    CALLED(q, kc, vc, ke, ve, bt, cl, o);
}
int pa_multi_query_q8(void *o, const void *q, const void *kc, const void *vc, const int8_t *ke, const int8_t *ve,
                      const int32_t *bt, const int32_t *cl, const int32_t *qs, float sc, int hkv, int S, int T, int mq, int hq,
                      int D, int B, int nb, int mb, int dt, void *w, size_t wb, void *s) {
    CALLED(q, kc, vc, ke, ve, bt, cl, qs, o);
}
size_t pa_decode_q8_workspace_size(int S, int hq, int hkv, int D, int B, int mb, int mq) { return 0; }
"""


@pytest.fixture(scope="module")
def native(tmp_path_factory):
    if not shutil.which("gcc") or not (Path(sysconfig.get_paths()["include"]) / "Python.h").exists():
        pytest.skip("the C part is not built here: no gcc or no Python headers")
    d = tmp_path_factory.mktemp("marshal")
    (d / "lib.c").write_text(STAND_IN)
    lib, mod = d / "libstand_in.so", d / "_marshal.so"
    inc = ["-I", str(ROOT / "include"), "-I", sysconfig.get_paths()["include"]]
    subprocess.run(["gcc", "-fPIC", "-shared", *inc, str(d / "lib.c"), "-o", str(lib)], check=True)
    subprocess.run(["gcc", "-fPIC", "-shared", *inc, str(ROOT / "paged_kv_cache_08_gb300" / "csrc" / "marshal.c"), "-o",
                    str(mod), str(lib)], check=True)
    record = ctypes.CDLL(str(lib))
    loader = importlib.machinery.ExtensionFileLoader("_marshal", str(mod))
    m = importlib.util.module_from_spec(importlib.util.spec_from_loader("_marshal", loader))
    loader.exec_module(m)
    m.setup(torch.Tensor, (torch.float16, torch.bfloat16, torch.float8_e4m3fn, torch.int8, torch.int32, torch.int64,
                           torch.float64), torch.empty_like, lambda dev: 0, lambda: 0, lambda *a: None)
    return m, record


@pytest.fixture()
def device0(monkeypatch):
    monkeypatch.setattr(torch.Tensor, "get_device", lambda self: 0, raising=False)


def _operands(call):
    """Arguments of a call, and what is added behind them (None in the place of an output: the call allocates it)."""
    x = torch.zeros((3, 2, 128), dtype=torch.float16)
    cache = [torch.zeros((4, 2, 16, 128), dtype=torch.float8_e4m3fn) for _ in range(2)]
    cache += [torch.zeros((4, 2), dtype=torch.int8) for _ in range(2)]
    tables = [torch.zeros((3, 2), dtype=torch.int32), torch.ones(3, dtype=torch.int32)]
    start = torch.arange(4, dtype=torch.int32)
    if call == "rope":
        return [x, x.clone(), torch.zeros(3, dtype=torch.int64), torch.ones(64, dtype=torch.float64), 1.0, False, x.clone(),
                x.clone()]
    if call == "append":
        return [x, x.clone(), *cache, *tables, start, 1]
    if call == "read_blocks":
        pool = torch.zeros((5, 2, 16, 128), dtype=torch.float16)
        return [*cache, pool, pool.clone(), torch.zeros(2, dtype=torch.int32), torch.ones(2, dtype=torch.int32)]
    return [x, *cache, *tables, start if call == "several" else None, 0.1, 2, 1, x.clone()]


CALLS = ["rope", "append", "read_blocks", "attention", "several"]


def _call(m, call, args):
    return getattr(m, "attention" if call == "several" else call)(*args)


@pytest.mark.parametrize("call", CALLS)
def test_the_library_is_given_the_tensors_addresses(native, device0, call):
    m, record = native
    calls = ctypes.c_int.in_dll(record, "calls")
    calls.value = 0
    args = _operands(call)
    assert _call(m, call, args) is not None
    assert calls.value == 1
    want = [a.data_ptr() for a in args if isinstance(a, torch.Tensor)]
    assert list((ctypes.c_size_t * 16).in_dll(record, "seen"))[:len(want)] == want


@pytest.mark.parametrize("call,at", [(c, i) for c in CALLS for i, a in enumerate(_operands(c)) if isinstance(a, torch.Tensor)])
def test_a_tensor_without_an_address_is_left_to_python(native, device0, call, at):
    m, record = native
    calls = ctypes.c_int.in_dll(record, "calls")
    calls.value = 0
    args, results = _operands(call), []

    def body(x):
        assert type(x) is torch.Tensor and x.shape == args[at].shape
        results.append(_call(m, call, args[:at] + [x] + args[at + 1:]))
        return torch.zeros(())

    torch.vmap(body)(torch.stack([args[at].view(torch.uint8)] * 2).view(args[at].dtype))
    assert results == [None] and calls.value == 0


def test_the_built_file_is_this_interpreters():
    assert build.MARSHAL == _native.MARSHAL_PATH
    assert build.MARSHAL.name == "_marshal" + sysconfig.get_config_var("EXT_SUFFIX")


@pytest.mark.parametrize("lacks", ["headers", "gcc"])
def test_the_build_goes_on_without_headers_or_compiler(monkeypatch, tmp_path, capsys, lacks):
    monkeypatch.setattr(build, "MARSHAL", tmp_path / "_marshal.so")
    if lacks == "headers":
        monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    else:
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
    assert build.build_marshal() is None
    assert not build.MARSHAL.exists()
    assert ("Python.h" if lacks == "headers" else "gcc") in capsys.readouterr().err


@pytest.fixture()
def not_built(monkeypatch, tmp_path):
    monkeypatch.setattr(_native, "MARSHAL_PATH", tmp_path / "_marshal.so")
    monkeypatch.setattr(pa, "_marshal", None)


def test_calls_are_made_without_it(not_built):
    """Refused by the Python code's checks, not for the missing file."""
    h = torch.zeros((4, 2, 128), dtype=torch.float16)
    with pytest.raises(TypeError):
        pa.rope(h, None, torch.zeros(4, dtype=torch.int32), torch.zeros(64, dtype=torch.float64))
    assert isinstance(pa._marshal, _native.PythonCalls)


@pytest.mark.gpu
def test_results_are_the_same_without_it(monkeypatch):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(3)
    f, _ = pa.rope_frequencies(128)
    lens = torch.tensor([37, 5, 64], dtype=torch.int32, device=dev)
    tables = torch.arange(12, dtype=torch.int32, device=dev).reshape(3, 4)
    start = torch.tensor([0, 3, 5, 6], dtype=torch.int32, device=dev)
    q = torch.randn((6, 12, 128), generator=gen, device=dev).half()
    k, v = (torch.randn((6, 2, 128), generator=gen, device=dev).half() for _ in range(2))

    def step():
        cache = [torch.zeros((12, 2, 16, 128), device=dev).to(torch.float8_e4m3fn) for _ in range(2)]
        cache += [torch.zeros((12, 2), dtype=torch.int8, device=dev) for _ in range(2)]
        a, b = pa.rope(q, k, torch.arange(6, device=dev), f)
        pa.cache_append_q8(b, v, *cache, tables, lens, start, 3)
        pa.cache_append_q8(b[:3], v[:3], *cache, tables, lens)
        out = [a, b, pa.multi_query_q8(a, *cache, tables, lens, start, 0.1, 2, 3),
               pa.decode_q8(a[:3], *cache, tables, lens, 0.1, 2)]
        back = [torch.zeros((12, 2, 16, 128), dtype=torch.float16, device=dev) for _ in range(2)]
        pa.read_blocks_q8(*cache, *back, tables.flatten(), tables.flatten())
        torch.cuda.synchronize()
        return [np.asarray(x.cpu().view(torch.uint8)) for x in out + cache + back]

    want = step()
    monkeypatch.setattr(pa, "_marshal", _native.PythonCalls())
    for a, b in zip(step(), want):
        assert np.array_equal(a, b)
