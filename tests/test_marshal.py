"""The binding's C part (csrc/marshal.c) without a GPU: built against a stand-in of the library that records its calls, on
host tensors that answer as if they lay on device 0.  What reaches the library are the tensors' own addresses, and a call
with a tensor that has none to give (a batched one inside torch.vmap) goes to the Python code."""
import ctypes
import importlib.machinery
import importlib.util
import subprocess
import sysconfig
from pathlib import Path

import pytest
import torch

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
