"""The quantising append and the read-back against their definitions: codes, exponents and values are
compared bit for bit, since every step of theirs is exact or rounds once."""
import numpy as np
import pytest
import torch

import paged_kv_cache_08_gb300 as pa
import q8_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


@pytest.fixture(autouse=True)
def _clean_status():
    pa.read_device_status(clear=True)
    yield


class Cache:
    """An 8-bit cache on the GPU and its reference on the host, filled with every code."""

    def __init__(self, nb, heads, block, seed=0, exps=(-12, 4)):
        rng = np.random.default_rng(seed)
        shape = (nb, heads, block, ref.D)
        self.k = rng.integers(0, 256, shape).astype(np.uint8)
        self.v = rng.integers(0, 256, shape).astype(np.uint8)
        self.ke = rng.integers(exps[0], exps[1], shape[:2]).astype(np.int8)
        self.ve = rng.integers(exps[0], exps[1], shape[:2]).astype(np.int8)
        self.dev = [torch.from_numpy(x.copy()).to(DEV) for x in (self.k, self.v)]
        self.dev = [x.view(torch.float8_e4m3fn) for x in self.dev]
        self.dev += [torch.from_numpy(x.copy()).to(DEV) for x in (self.ke, self.ve)]

    def append(self, k, v, tables, lens, start=None, max_q=1, **kw):
        self.args = [None if x is None else torch.tensor(np.asarray(x), dtype=torch.int32, device=DEV)
                     for x in (tables, lens, start)]
        if kw:
            torch.cuda.synchronize()     # another stream reads them
        pa.cache_append_q8(k, v, *self.dev, *self.args[:2], query_start=self.args[2], max_q=max_q, **kw)
        ref.append(ref.f64(k), ref.f64(v), self.k, self.v, self.ke, self.ve, np.asarray(tables), lens, start, max_q)

    def check(self):
        torch.cuda.synchronize()
        for name, got, want in (("k_exp", self.dev[2], self.ke), ("v_exp", self.dev[3], self.ve)):
            assert np.array_equal(got.cpu().numpy(), want), name
        for name, got, want in (("k", self.dev[0], self.k), ("v", self.dev[1], self.v)):
            got = ref.codes(got)
            nan = (got & 0x7F == 0x7F) & (want & 0x7F == 0x7F)
            assert np.array_equal(np.where(nan, 0, got), np.where(nan, 0, want)), name


def _rows(T, heads, dtype, seed, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((2, T, heads, ref.D), generator=gen) * torch.exp(spread * torch.randn((2, T, heads, 1), generator=gen))
    return x[0].to(dtype).to(DEV), x[1].to(dtype).to(DEV)


def _tables(lens, block, nb, seed):
    rng = np.random.default_rng(seed)
    ids = rng.permutation(nb)
    width = max(1, max(-(-L // block) for L in lens) + 1)
    t = np.full((len(lens), width), -1, dtype=np.int32)
    at = 0
    for s, L in enumerate(lens):
        n = -(-L // block)
        t[s, :n] = ids[at:at + n]
        at += n
    return t


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,dtype", [(1, torch.float16), (3, torch.bfloat16), (8, torch.float16),
                                         (9, torch.bfloat16), (20, torch.float16)])
def test_append_one_row_each(block, heads, dtype):
    lens = [1, 2, 0, block - 1, block, block + 1, 2 * block, 3 * block + 7, 5]
    c = Cache(40, heads, block, seed=block)
    k, v = _rows(len(lens), heads, dtype, seed=1)
    c.append(k, v, _tables(lens, block, 40, 2), lens)
    c.check()
    assert pa.read_device_status(clear=True) == 0


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_ragged(block, dtype):
    lens = [300, 5, 17, 0, 129, 64, 1, 260, 33]
    new = [300, 3, 1, 0, 40, 64, 1, 0, 32]
    start = np.concatenate([[0], np.cumsum(new)])
    c = Cache(80, 2, block, seed=3)
    k, v = _rows(int(start[-1]), 2, dtype, seed=4)
    c.append(k, v, _tables(lens, block, 80, 5), lens, start, max_q=300)
    c.check()
    assert pa.read_device_status(clear=True) == 0


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_long_chunks(block, dtype):
    """Chunks of several blocks, begun and ended inside one."""
    lens, new = [300, 470], [299, 390]
    start = np.array([0, 299, 689])
    c = Cache(64, 3, block, seed=33)
    k, v = _rows(689, 3, dtype, seed=34)
    k[5, 1, 3], v[400, 2, 100], k[688, 0, 0] = float("inf"), float("nan"), 3e4
    c.append(k, v, _tables(lens, block, 64, 35), lens, start, max_q=400)
    c.check()
    assert pa.read_device_status(clear=True) == 0


@pytest.mark.parametrize("S", [1, 33, 700, 1500])
def test_append_many_sequences(S):
    """The search over query_start: batches below and above a warp's and a square of it."""
    rng = np.random.default_rng(S)
    new = rng.integers(0, 4, S)
    lens = new + rng.integers(0, 20, S)
    start = np.concatenate([[0], np.cumsum(new)])
    nb = int(sum(-(-lens // 16))) + 4
    c = Cache(nb, 1, 16, seed=7)
    k, v = _rows(int(start[-1]) + 3, 1, torch.float16, seed=8)      # rows behind the last sequence's are not read
    c.append(k, v, _tables(lens.tolist(), 16, nb, 9), lens.tolist(), start, max_q=4)
    c.check()
    assert pa.read_device_status(clear=True) == 0


def test_append_token_by_token_grows_and_restarts():
    """One block filled a token at a time with rows of growing size, then used again from offset 0."""
    block, heads = 16, 2
    c = Cache(6, heads, block, seed=11)
    table = np.array([[4, 1, 5]], dtype=np.int32)
    for L in range(1, 2 * block + 3):
        k, v = _rows(1, heads, torch.float16, seed=100 + L)
        k *= 1.7 ** (L % 9)
        v *= 0.6 ** (L % 7)
        c.append(k, v, table, [L])
        c.check()
    k, v = _rows(1, heads, torch.float16, seed=200)
    c.append(k * 1e-3, v * 1e-3, table, [1])       # the block starts afresh: its exponents may shrink
    c.check()
    assert c.ke[4].max() < -12


def test_append_takes_back_and_writes_again():
    """Rejected draft tokens: the length goes back and other rows take their slots."""
    c = Cache(8, 2, 16, seed=13)
    table = np.array([[3, 0, 6], [2, 7, 1]], dtype=np.int32)
    for lens, new in (([20, 9], [20, 9]), ([24, 14], [4, 5]), ([22, 10], [1, 1]), ([27, 17], [5, 7])):
        start = np.concatenate([[0], np.cumsum(new)])
        k, v = _rows(int(start[-1]), 2, torch.bfloat16, seed=sum(lens), spread=2.0)
        c.append(k, v, table, lens, start, max_q=20)
        c.check()


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_append_extreme_values(dtype):
    """Infinities, NaN, zeros, the types' largest and smallest values, values at the borders of the grid."""
    info = torch.finfo(dtype)
    c = Cache(12, 1, 16, seed=17)
    k, v = _rows(10, 1, dtype, seed=18)
    k[0] = 0.0
    k[1, 0, ::3] = float("inf")
    k[2, 0, 1::2] = float("nan")
    k[3, 0, :5] = -float("inf")
    k[4] = info.max
    k[5] = info.smallest_normal * info.eps           # the smallest value of all
    k[6] = float("nan")
    k[7] = -float("inf")
    k[8, 0] = torch.from_numpy(ref.CODE_VALUES[:128].copy()).nan_to_num().to(dtype)
    k[9, 0, :126] = torch.from_numpy((ref.CODE_VALUES[:126] + ref.CODE_VALUES[1:127]) / 2).to(dtype)   # ties
    k[9, 0, 126] = 448.0
    v.copy_(k.flip(0))
    lens = [1 + 3 * (i % 2) for i in range(10)]      # offsets 0 (afresh) and 3 (growing)
    c.append(k, v, np.arange(10, dtype=np.int32)[:, None], lens)
    c.check()
    # all rows of one block at once
    c = Cache(2, 1, 16, seed=19)
    c.append(k, v, np.array([[1]], dtype=np.int32), [13], np.array([0, 10]), max_q=16)
    c.check()


def test_append_strided_rows():
    T, heads = 50, 2
    gen = torch.Generator().manual_seed(21)
    x = torch.randn((T, 12 + 2 * heads, ref.D), generator=gen).to(torch.float16).to(DEV)
    k, v = x[:, 12:12 + heads], x[:, 12 + heads:]
    c = Cache(8, heads, 16, seed=22)
    c.append(k, v, _tables([60], 16, 8, 23), [60], np.array([0, 50]), max_q=64)
    c.check()
    # one row for every token: stride 0
    c = Cache(8, heads, 16, seed=24)
    c.append(k[:1].expand(T, heads, ref.D), v[:1].expand(T, heads, ref.D), _tables([60], 16, 8, 23), [60],
             np.array([0, 50]), max_q=64)
    c.check()


def test_append_skips_bad_blocks_and_clamps_counts():
    B = pa._native
    c = Cache(6, 2, 16, seed=25)
    k, v = _rows(8, 2, torch.float16, seed=26)
    c.append(k[:3], v[:3], np.array([[0, 9], [2, -1], [4, 1]], dtype=np.int32), [20, 17, 18])
    c.check()
    assert pa.read_device_status(clear=True) == B.DEV_BAD_BLOCK_ID
    # more tokens than max_q, than the context, than rows; a span outside the rows; a length beyond the table
    c.append(k, v, np.array([[0], [2], [3], [5], [1]], dtype=np.int32), [10, 2, 4, 3, 40], np.array([0, 5, 8, 12, 9, 3]),
             max_q=3)
    c.check()
    assert pa.read_device_status(clear=True) == B.DEV_BAD_CONTEXT


def test_append_query_start_behind_the_first_rows():
    """query_start[0] > 0: the rows before it belong to no sequence."""
    c = Cache(12, 1, 16, seed=27)
    k, v = _rows(90, 1, torch.float16, seed=28)
    c.append(k, v, _tables([30, 33], 16, 12, 29), [30, 33], np.array([70, 75, 90]), max_q=16)
    c.check()
    assert pa.read_device_status(clear=True) == 0


def test_append_in_a_graph_and_on_a_stream():
    c = Cache(12, 2, 16, seed=31)
    k, v = _rows(4, 2, torch.float16, seed=32)
    tables = np.arange(12, dtype=np.int32).reshape(4, 3)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.append(k, v, tables, [17, 5, 32, 1], stream=side)
    torch.cuda.current_stream().wait_stream(side)
    c.check()
    lens = torch.tensor([18, 6, 33, 2], dtype=torch.int32, device=DEV)
    t = torch.from_numpy(tables).to(DEV)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        pa.cache_append_q8(k, v, *c.dev, t, lens)
    for step in range(3):
        g.replay()
        ref.append(ref.f64(k), ref.f64(v), c.k, c.v, c.ke, c.ve, tables, lens.cpu().numpy())
        c.check()
        lens.add_(1)
        k.mul_(1.5)


def test_every_way_to_call_gives_the_same():
    """By way of the binding's C part, and of its Python code (a stream, a tensor of another class)."""
    k, v = _rows(4, 2, torch.float16, seed=36)
    tables, lens = np.arange(12, dtype=np.int32).reshape(4, 3), [17, 5, 32, 1]
    c = Cache(12, 2, 16, seed=37)
    start = [x.clone() for x in c.dev]
    c.append(k, v, tables, lens)
    c.check()
    for how in (dict(stream=torch.cuda.current_stream()), dict(q=torch.arange(5, dtype=torch.int32, device=DEV)),
                dict(k=torch.nn.Parameter(k, requires_grad=False))):
        again = [x.clone() for x in start]
        pa.cache_append_q8(how.get("k", k), v, *again, *c.args[:2], query_start=how.get("q"), max_q=2,
                           stream=how.get("stream"))
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(again, c.dev))
    ids = torch.arange(12, dtype=torch.int32, device=DEV)
    outs = [[torch.empty((12, 2, 16, ref.D), dtype=torch.bfloat16, device=DEV) for _ in range(2)] for _ in range(2)]
    pa.read_blocks_q8(*c.dev, *outs[0], ids, ids)
    pa.read_blocks_q8(*c.dev, *outs[1], ids, ids, stream=torch.cuda.current_stream())
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(*outs))


# ---- read-back -----------------------------------------------------------------------------

@pytest.mark.parametrize("block,heads", [(16, 1), (32, 3), (64, 2), (128, 5)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_read_blocks(block, heads, dtype):
    """Every code under exponents from the smallest to the largest, beyond fp16's range too."""
    c = Cache(9, heads, block, seed=41, exps=(-128, 128))
    c.ke[:3], c.ve[:3] = np.int8(-16), np.int8(8)          # fp16's subnormals and its largest values
    c.dev[2].copy_(torch.from_numpy(c.ke))
    c.dev[3].copy_(torch.from_numpy(c.ve))
    src, dst = np.array([4, 0, 8, 2, 1, 3, 4], dtype=np.int32), np.array([1, 0, 6, 7, 5, 2, 4], dtype=np.int32)
    out = [torch.full((8, heads, block, ref.D), 7.0, dtype=dtype, device=DEV) for _ in range(2)]
    pa.read_blocks_q8(*c.dev, *out, torch.from_numpy(src).to(DEV), torch.from_numpy(dst).to(DEV))
    torch.cuda.synchronize()
    for got, code, exp in ((out[0], c.k, c.ke), (out[1], c.v, c.ve)):
        want = torch.full((8, heads, block, ref.D), 7.0, dtype=torch.float64)
        top = torch.finfo(dtype).max
        want[torch.from_numpy(dst).long()] = torch.from_numpy(ref.values(code, exp)[src]).clamp(-top, top)
        assert torch.equal(got.cpu().nan_to_num(nan=9.0), want.to(dtype).nan_to_num(nan=9.0))
    assert pa.read_device_status(clear=True) == 0


def test_read_skips_bad_ids():
    c = Cache(4, 2, 16, seed=43)
    out = [torch.full((3, 2, 16, ref.D), 7.0, dtype=torch.float16, device=DEV) for _ in range(2)]
    ids = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    pa.read_blocks_q8(*c.dev, *out, ids(-1, 4, 1, 0, 2), ids(0, 1, 3, -1, 2))
    torch.cuda.synchronize()
    assert pa.read_device_status(clear=True) == pa._native.DEV_BAD_BLOCK_ID
    assert (out[0][:2] == 7.0).all() and (out[1][:2] == 7.0).all()
    want = torch.from_numpy(ref.values(c.k, c.ke)[2]).to(torch.float16)
    assert torch.equal(out[0][2].cpu().nan_to_num(9.0), want.nan_to_num(9.0))
    pa.read_blocks_q8(*c.dev, *out, ids(), ids())
    assert pa.read_device_status(clear=True) == 0


def test_read_what_was_appended():
    """Quantise and read back: within half an e4m3 step of the rows under the block's exponent."""
    T, heads, block = 200, 2, 32
    k, v = _rows(T, heads, torch.bfloat16, seed=45)
    c = Cache(8, heads, block, seed=46)
    table = _tables([T], block, 8, 47)
    c.append(k, v, table, [T], np.array([0, T]), max_q=T)
    n = -(-T // block)
    out = [torch.empty((n, heads, block, ref.D), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    pa.read_blocks_q8(*c.dev, *out, torch.from_numpy(table[0, :n].copy()).to(DEV),
                      torch.arange(n, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    for got, x, exp in ((out[0], k, c.ke), (out[1], v, c.ve)):
        y = ref.f64(got).transpose(0, 2, 1, 3).reshape(n * block, heads, ref.D)[:T]
        e = np.repeat(exp[table[0, :n]].astype(np.float64), block, axis=0)[:T, :, None]
        x = ref.f64(x)
        half = np.maximum(np.abs(x) * 2.0 ** -4, 2.0 ** (e - 10))
        assert (np.abs(y - x) <= half).all()


def test_copy_blocks_serves_an_8_bit_pool():
    """Copy-on-write of 8-bit blocks: the pools seen as 16-bit elements, the exponents by index."""
    c = Cache(8, 2, 16, seed=49)
    as16 = [x.view(torch.float16) for x in c.dev[:2]]
    src, dst = torch.tensor([1, 5], device=DEV), torch.tensor([7, 0], device=DEV)
    pa.copy_blocks(*as16, *as16, src.int(), dst.int())
    for e in c.dev[2:]:
        e[dst] = e[src]
    for x in (c.k, c.v, c.ke, c.ve):
        x[[7, 0]] = x[[1, 5]]
    c.check()


def test_append_and_read_refuse():
    c = Cache(4, 2, 16, seed=51)
    k, v = _rows(2, 2, torch.float16, seed=52)
    t = torch.zeros((2, 2), dtype=torch.int32, device=DEV)
    lens = torch.ones(2, dtype=torch.int32, device=DEV)
    out = torch.empty((4, 2, 16, 128), dtype=torch.float16, device=DEV)
    kc, vc, ke, ve = c.dev
    for call, error in ((lambda: pa.cache_append_q8(k, v, kc.view(torch.uint8), vc, ke, ve, t, lens), TypeError),
                        (lambda: pa.cache_append_q8(k, v, kc, vc, ke.int(), ve, t, lens), TypeError),
                        (lambda: pa.cache_append_q8(k.float(), v, kc, vc, ke, ve, t, lens), TypeError),
                        (lambda: pa.cache_append_q8(k, v.bfloat16(), kc, vc, ke, ve, t, lens), TypeError),
                        (lambda: pa.cache_append_q8(k, v, kc, vc, ke, ve, t.long(), lens), TypeError),
                        (lambda: pa.cache_append_q8(k, v, kc, vc[:3], ke, ve, t, lens), ValueError),
                        (lambda: pa.cache_append_q8(k, v, kc, vc, ke[:3], ve, t, lens), ValueError),
                        (lambda: pa.cache_append_q8(k[:1], v[:1], kc, vc, ke, ve, t, lens), ValueError),
                        (lambda: pa.cache_append_q8(k, v[:1], kc, vc, ke, ve, t, lens), ValueError),
                        (lambda: pa.cache_append_q8(k, v, kc, vc, ke, ve, t[:1], lens), ValueError),
                        (lambda: pa.cache_append_q8(k, v, kc, vc, ke, ve, t, lens, query_start=lens), ValueError),
                        (lambda: pa.cache_append_q8(k, v, kc, vc, ke, ve, t, lens,
                                                    query_start=torch.zeros(3, dtype=torch.int32, device=DEV), max_q=0),
                         pa.PAError),
                        (lambda: pa.read_blocks_q8(*c.dev, out.float(), out, lens, lens), TypeError),
                        (lambda: pa.read_blocks_q8(*c.dev, out, out.bfloat16(), lens, lens), TypeError),
                        (lambda: pa.read_blocks_q8(*c.dev, out[:, :1], out[:, :1], lens, lens), ValueError),
                        (lambda: pa.read_blocks_q8(*c.dev, out, out, lens, lens[:1]), ValueError)):
        with pytest.raises(error):
            call()


def test_append_flags_a_query_start_that_decreases():
    """Not a batch the call takes: some of its rows may stay unwritten, but never without the status word."""
    for start in ([0, 50, 10, 60], [100, 0, 50], [0, 60, 60, 59, 60]):
        S = len(start) - 1
        c = Cache(6 * S, 2, 16, seed=41)
        k, v = _rows(max(start), 2, torch.float16, seed=42)
        tables = np.arange(6 * S, dtype=np.int32).reshape(S, 6)
        c.append(k, v, tables, [65] * S, np.array(start), max_q=64)
        torch.cuda.synchronize()
        assert pa.read_device_status(clear=True) == pa._native.DEV_BAD_CONTEXT, start
