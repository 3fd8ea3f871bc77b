"""Attention over the 8-bit cache against softmax(scale q K^T) V in 64 bits on the cached values, within
bounds derived per element (q8_reference.attention)."""
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_08_gb300 as pa
import q8_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")
SCALE = 1.0 / math.sqrt(ref.D)


@pytest.fixture(autouse=True)
def _clean_status():
    pa.read_device_status(clear=True)
    yield


class Problem:
    """A cache of values like keys and values, with rows, exponents and table entries no token owns
    holding what must not matter: NaN codes, extreme exponents, ids outside the pool."""

    def __init__(self, lens, Hq, Hkv, block, dtype, new=None, seed=0, spread=1.0, poison=True, extra_rows=0):
        rng = np.random.default_rng(seed)
        need = [-(-L // block) for L in lens]
        nb = sum(need) + 3
        self.lens, self.new = list(lens), None if new is None else list(new)
        self.Hq, self.Hkv, self.block = Hq, Hkv, block
        x = rng.standard_normal((2, nb, Hkv, block, ref.D)) * np.exp(spread * rng.standard_normal((2, nb, Hkv, 1, 1)))
        self.codes, self.exps = [], []
        for y in x:
            amax = np.abs(y).max((2, 3))
            e = np.ceil(np.log2(amax / 448)).astype(np.int64)
            self.codes.append(ref.to_code(y * np.exp2(-e.astype(np.float64))[:, :, None, None]))
            self.exps.append(e.astype(np.int8))
        ids = rng.permutation(nb)
        width = max([1] + need) + 2
        self.tables = np.full((len(lens), width), -1, dtype=np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = ids[at:at + n]
            if poison and n:
                last = ids[at + n - 1]
                for c in self.codes:
                    c[last, :, lens[s] - (n - 1) * block:] = 0x7F
                self.tables[s, n:] = [2**31 - 1, -5][:width - n] + [nb] * (width - n - 2)
            at += n
        if poison:
            for c, e in zip(self.codes, self.exps):
                c[ids[at:]], e[ids[at:]] = 0xFF, 127
        rows = (len(lens) if new is None else sum(new)) + extra_rows
        gen = torch.Generator().manual_seed(seed + 1)
        self.q = torch.randn((rows, Hq, ref.D), generator=gen).to(dtype)
        self.start = None if new is None else np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        self.max_q = 1 if new is None else max([1] + list(new))

    def upload(self):
        t = lambda x: torch.from_numpy(np.ascontiguousarray(x)).to(DEV)  # noqa: E731
        self.args = [self.q.to(DEV)] + [t(c).view(torch.float8_e4m3fn) for c in self.codes] + [t(e) for e in self.exps]
        self.args += [t(self.tables), torch.tensor(self.lens, dtype=torch.int32, device=DEV)]
        if self.start is not None:
            self.args.append(t(self.start))

    def call(self, scale=SCALE, **kw):
        if self.start is None:
            return pa.decode_q8(*self.args, scale, self.Hkv, **kw)
        return pa.multi_query_q8(*self.args, scale, self.Hkv, self.max_q, **kw)

    def reference(self, scale=SCALE):
        return ref.attention(ref.f64(self.q), *self.codes, *self.exps, self.tables, self.lens, scale, self.start,
                             self.max_q)

    def run(self, scale=SCALE, status=0, **kw):
        self.upload()
        out = self.call(scale, **kw)
        torch.cuda.synchronize()
        assert pa.read_device_status(clear=True) == status
        ref.check_attention(out, *self.reference(scale))
        return out


LENS = [1, 0, 2, 15, 16, 17, 31, 64, 65, 100, 128, 129, 300]


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (12, 2), (3, 3), (16, 1), (32, 1), (8, 4), (20, 2), (9, 1)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_decode(block, Hq, Hkv, dtype):
    Problem(LENS, Hq, Hkv, block, dtype, seed=block + Hq).run()


@pytest.mark.parametrize("lens,Hq,Hkv", [([4097], 6, 1), ([9000, 3], 4, 1), ([2500] * 3 + [1], 12, 2), ([20000], 1, 1)])
@pytest.mark.parametrize("block", [16, 64])
def test_decode_long(lens, Hq, Hkv, block):
    Problem(lens, Hq, Hkv, block, torch.bfloat16 if block == 64 else torch.float16, seed=7).run()


@pytest.mark.parametrize("S", [1, 300, 1100])
def test_decode_many_sequences(S):
    rng = np.random.default_rng(S)
    Problem(rng.integers(0, 40, S).tolist(), 2, 2, 16, torch.float16, seed=S).run()


@pytest.mark.parametrize("group,n", [(1, 2), (1, 32), (2, 16), (3, 5), (4, 8), (6, 5), (8, 4), (16, 2), (8, 1), (1, 9)])
@pytest.mark.parametrize("block", [16, 32, 128])
def test_several_tokens(group, n, block):
    lens = [n, 70, 129, 64 + n, 300, 40, 2 * block + 3, 17 + n]
    new = [n, n, 1, n, n, 0, n, max(1, n - 1)]
    Problem(lens, 2 * group, 2, block, torch.float16 if n % 2 else torch.bfloat16, new=new, seed=group * n).run()


def test_first_tokens_see_only_themselves():
    """Full prefill: row i of a sequence sees i + 1 tokens."""
    Problem([32, 5, 1, 20], 1, 1, 16, torch.bfloat16, new=[32, 5, 1, 20], seed=61).run()


@pytest.mark.parametrize("scale", [0.0, -0.3, 1.0, 4.0])
def test_scales(scale):
    """A large scale moves the softmax's base in the middle of a sequence."""
    Problem([700, 33, 1, 260], 12, 2, 16, torch.float16, seed=63).run(scale)
    Problem([700, 33, 1, 260], 4, 1, 64, torch.bfloat16, new=[5, 3, 1, 8], seed=64).run(scale)


@pytest.mark.parametrize("spread", [4.0, 9.0])
def test_blocks_of_very_different_scales(spread):
    """Exponents of neighbouring blocks 20 and more apart."""
    Problem([500, 64, 90], 6, 1, 16, torch.float16, seed=65, spread=spread).run(0.01)


def test_exponents_at_their_limits():
    p = Problem([100, 40], 4, 2, 16, torch.bfloat16, seed=66)
    p.exps[1][:] = np.random.default_rng(67).choice([-128, -60, -59, 0, 59, 60, 127], p.exps[1].shape)
    p.run()
    p.exps[0][:] = -60
    p.run()
    p.exps[0][:] = 60
    p.run(2.0 ** -60)


@pytest.mark.parametrize("scale", [0.3, 1.0, 3.0])
def test_values_of_extreme_blocks_far_apart_in_score(scale):
    """V blocks 2^120 apart whose tokens share the weight: the sum of weights keeps the small blocks' tokens,
    within a piece, when the base moves, and when pieces meet."""
    for lens, block, seed in (([900, 64, 33], 16, 0), ([6000, 700], 128, 1)):
        p = Problem(lens, 6, 1, block, torch.bfloat16, seed=166 + seed, spread=0.0)
        p.exps[1][:] = np.where(np.arange(p.exps[1].size).reshape(p.exps[1].shape) % 2, -60, 60)
        p.run(scale)
        p.exps[1][:] = 60
        p.exps[1][p.tables[0, 0]] = -60
        p.run(scale)


def test_nan_is_where_the_definition_has_it():
    """A NaN in V reaches its dimension in the rows that see its token; one in K every dimension of them."""
    p = Problem([40, 50, 33], 4, 2, 16, torch.float16, new=[6, 4, 8], seed=68)
    at = lambda s, t: (p.tables[s, t // 16], t % 16)  # noqa: E731
    b, o = at(0, 37)
    p.codes[1][b, 1, o, 7] = 0x7F             # seen by rows 3..5 of sequence 0
    b, o = at(1, 48)
    p.codes[0][b, 0, o, 90] = 0xFF            # seen by rows 2, 3 of sequence 1
    b, o = at(2, 3)
    p.codes[1][b, 0, o, 127] = 0xFF           # seen by every row of sequence 2
    b, o = at(2, 32)
    p.codes[1][b, 0, o, :3] = 0x7F            # the last row alone
    p.run()


def test_infinities_in_q():
    p = Problem([40, 50, 33], 2, 1, 16, torch.bfloat16, seed=69)
    p.q[1, 0, 5] = float("inf")
    p.q[2, 1] = float("nan")
    p.upload()
    out = p.call()
    torch.cuda.synchronize()
    assert torch.isnan(out[1, 0]).all() and torch.isnan(out[2, 1]).all()
    for row, h in ((0, 0), (0, 1), (1, 1), (2, 0)):
        assert torch.isfinite(out[row, h]).all()


@pytest.mark.parametrize("top", [3e38, 1e-38])
def test_queries_at_bf16s_limits(top):
    """bf16 queries far outside fp16's range, rows of one tile with very different sizes."""
    p = Problem([40, 17], 12, 1, 16, torch.bfloat16, seed=70)
    p.q[0, 3] *= top / p.q[0, 3].abs().max()
    p.q[1, 7] *= 2.0 ** -100
    p.q[1, 8] = 0
    p.exps[0][:] = -7
    if top > 1:
        p.q[0, 3] *= 2.0 ** -20
        p.run(2.0 ** -108)
    else:
        p.run(1.0)


@pytest.mark.parametrize("new", [None, [5, 1, 0, 3]])
def test_tables_much_wider_than_the_contexts(new):
    """The grid is sized by the table's width: most shares are then empty, or a unit or two."""
    for lens in ([5, 60, 7, 33], [5, 0, 7, 3]):
        n = None if new is None else [min(a, b) for a, b in zip(new, lens)]
        p = Problem(lens, 12, 2, 16, torch.float16, new=n, seed=96)
        p.tables = np.concatenate([p.tables, np.full((4, 3000), -1, dtype=np.int32)], axis=1)
        p.run()


@pytest.mark.parametrize("group,n", [(4, 4), (8, 3), (4, 8), (1, 32), (16, 2)])
def test_several_tokens_over_long_contexts(group, n):
    """Segments cut between warps and CTAs with 9 to 32 rows."""
    Problem([3000, 40, 777], group, 1, 32, torch.float16, new=[n, 2, n], seed=97).run()


def test_several_tokens_of_many_sequences():
    rng = np.random.default_rng(98)
    lens = rng.integers(0, 30, 1100)
    new = np.minimum(lens, rng.integers(0, 3, 1100))
    Problem(lens.tolist(), 2, 1, 16, torch.float16, new=new.tolist(), seed=98).run()


@pytest.mark.parametrize("new", [False, True])
def test_many_short_segments(new):
    """More than two segments begin in every warp's share: the grid of twelve warps a CTA."""
    rng = np.random.default_rng(100)
    lens = rng.integers(0, 70, 640)
    lens[100] = 5000                          # and one that is cut many times
    n = np.minimum(lens, rng.integers(0, 3, 640)).tolist() if new else None
    assert 640 * 4 >= 2 * 8 * 152
    Problem(lens.tolist(), 12, 4, 16, torch.float16, new=n, seed=100).run()


@pytest.mark.parametrize("seed", range(24))
def test_shares_cut_anywhere(seed):
    """Random batches of short and long contexts under tables of random width: the warps' shares begin and end at every
    place of a segment, and some are empty."""
    rng = np.random.default_rng(900 + seed)
    Hkv, group = int(rng.integers(1, 5)), int(rng.integers(1, 9))
    S = int(rng.integers(1, 60))
    top = int(rng.choice([40, 200, 1500]))
    lens = rng.integers(0, top, S)
    lens[rng.random(S) < 0.3] = rng.integers(0, 33)
    new = None if seed % 3 == 0 else [int(min(x, n)) for x, n in zip(lens, rng.integers(0, 32 // group + 1, S))]
    p = Problem([int(x) for x in lens], Hkv * group, Hkv, int(rng.choice([16, 32, 64, 128])),
                [torch.float16, torch.bfloat16][seed % 2], new=new, seed=seed)
    if seed % 4 == 1:
        p.tables = np.concatenate([p.tables, np.full((S, 400), -1, dtype=np.int32)], 1)
    p.run()


def test_no_sequences_and_no_rows():
    p = Problem([20, 33], 4, 1, 16, torch.float16, new=[0, 0], seed=99)
    p.upload()
    assert p.call().shape == (0, 4, 128)
    p.args[5], p.args[6], p.args[7] = p.args[5][:0], p.args[6][:0], p.args[7][:1]
    assert p.call().shape == (0, 4, 128)
    q, kc, vc, ke, ve, t, n, _ = p.args
    assert pa.decode_q8(q, kc, vc, ke, ve, t, n, SCALE, 1).shape == (0, 4, 128)


def test_bad_blocks_are_left_out():
    p = Problem([40, 50, 16, 33], 4, 1, 16, torch.float16, seed=71)
    nb = p.codes[0].shape[0]
    p.tables[0, 1] = nb
    p.tables[1, 3] = -1
    p.tables[2, 0] = -2**31                  # no token left: a zero row
    p.tables[3, 0], p.tables[3, 2] = 2**31 - 1, -7
    out = p.run(status=pa._native.DEV_BAD_BLOCK_ID)
    assert (out[2] == 0).all()
    p = Problem([40, 50, 33], 4, 1, 16, torch.float16, new=[3, 8, 1], seed=72)
    p.tables[0, 2] = -1
    p.tables[1, 0] = nb + 9
    p.tables[2] = -1
    p.run(status=pa._native.DEV_BAD_BLOCK_ID)


def test_counts_and_lengths_outside_their_range():
    p = Problem([40, 20, 33], 4, 1, 16, torch.float16, new=[4, 4, 4], seed=73)
    p.lens[1] = 3                             # fewer tokens than new rows
    p.lens[2] = 10**6                         # longer than the table
    p.tables[2, :] = p.tables[0, 0]
    p.codes[1][p.tables[0, 0]] &= 0x3F
    p.start = np.array([0, 4, 8, 30], dtype=np.int32)
    p.max_q = 5
    p.upload()
    out = torch.full_like(p.args[0], 3.0)
    p.call(out=out)
    torch.cuda.synchronize()
    assert pa.read_device_status(clear=True) == pa._native.DEV_BAD_CONTEXT
    want, bound, owned = p.reference()
    ref.check_attention(out, want, bound, owned)
    assert (out.cpu()[torch.from_numpy(~owned)] == 3.0).all()
    p = Problem([40, 20], 4, 1, 16, torch.float16, seed=74)
    p.lens[0] = -3
    out = p.run(status=pa._native.DEV_BAD_CONTEXT)
    assert (out[0] == 0).all()


def test_rows_behind_the_last_sequence_stay():
    p = Problem([40, 20, 9], 6, 1, 16, torch.float16, new=[2, 0, 5], seed=75, extra_rows=4)
    p.q[7:] = float("nan")
    p.upload()
    out = torch.full_like(p.args[0], -1.5)
    got = p.call(out=out)
    torch.cuda.synchronize()
    assert got is out and (out[7:] == -1.5).all()
    ref.check_attention(out, *p.reference())


def test_the_call_repeats_bit_for_bit():
    p = Problem([2048, 3, 900, 64, 1], 12, 2, 16, torch.float16, seed=76)
    first = p.run()
    for _ in range(5):
        assert torch.equal(p.call(), first)


def test_one_token_each_is_decode():
    p = Problem([500, 33, 1, 260], 12, 2, 16, torch.float16, seed=77)
    a = p.run()
    p.start = np.arange(5, dtype=np.int32)
    b = p.run()
    assert torch.equal(a, b)


def test_streams_do_not_share_scratch():
    """Calls on two streams at once, and two captured graphs replayed at once, keep their own results."""
    ps = [Problem([3000 + 500 * i, 77], 6, 1, 16, torch.float16, seed=80 + i) for i in range(2)]
    want = [p.run() for p in ps]
    streams = [torch.cuda.Stream() for _ in ps]
    got = [[] for _ in ps]
    torch.cuda.synchronize()
    for _ in range(20):
        for p, s, g in zip(ps, streams, got):
            g.append(p.call(stream=s))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
    graphs, outs = [], []
    for p in ps:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(p.call())
        graphs.append(g)
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(w, o) for w, o in zip(want, outs))


def test_two_host_threads_on_one_stream():
    import threading
    ps = [Problem([2500 + 700 * i, 90], 6, 1, 16, torch.float16, seed=88 + i) for i in range(3)]
    want = [p.run() for p in ps]
    got = [[] for _ in ps]

    def work(i):
        for _ in range(60):
            got[i].append(ps[i].call())

    threads = [threading.Thread(target=work, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert len(g) == 60 and all(torch.equal(w, x) for x in g)


def test_every_way_to_call_gives_the_same():
    """The C part of the binding takes plain tensors on the current stream; a stream, a workspace, or a tensor of
    another class goes by way of Python."""
    for new in (None, [3, 1]):
        p = Problem([400, 33], 12, 2, 16, torch.float16, new=new, seed=92)
        want = p.run()
        ws = torch.empty(pa.decode_q8_workspace_size(2, 12, 2, 128, 16, p.tables.shape[1], p.max_q) + 16,
                         dtype=torch.uint8, device=DEV)
        out = torch.empty_like(want)
        assert torch.equal(p.call(stream=torch.cuda.current_stream()), want)
        assert torch.equal(p.call(workspace=ws), want)
        assert torch.equal(p.call(workspace=ws, out=out, stream=torch.cuda.current_stream()), want)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            assert torch.equal(p.call(), want)
        torch.cuda.synchronize()
        p.args[0] = torch.nn.Parameter(p.args[0], requires_grad=False)
        assert torch.equal(p.call(), want)


def test_a_captured_call_follows_lengths_and_tables():
    p = Problem([60, 33, 90], 12, 2, 16, torch.float16, seed=84, poison=False)
    p.upload()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = p.call()
    for lens in ([1, 0, 17], [60, 33, 90], [16, 5, 64]):
        p.lens = lens
        p.args[6].copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        ref.check_attention(out, *p.reference())


def test_workspace_contents_do_not_matter():
    p = Problem([2048, 3, 900], 12, 2, 16, torch.float16, seed=85)
    want = p.run()
    need = pa.decode_q8_workspace_size(3, 12, 2, 128, 16, p.tables.shape[1])
    for fill in (0, 255, 0x7F):
        ws = torch.full((max(need, 16) + 16,), fill, dtype=torch.uint8, device=DEV)
        assert torch.equal(p.call(workspace=ws), want)


def test_a_pool_beyond_32_bit_offsets():
    """The last blocks of a pool of more than 4 GiB of codes."""
    nb, block = (1 << 32) // (128 * 128) + 500, 128
    p = Problem([300, 130], 8, 1, block, torch.float16, seed=86)
    small = p.codes[0].shape[0]
    p.upload()
    want = p.call()
    big = [torch.zeros((nb, 1, block, ref.D), dtype=torch.uint8, device=DEV) for _ in range(2)]
    exps = [torch.zeros((nb, 1), dtype=torch.int8, device=DEV) for _ in range(2)]
    for i in range(2):
        big[i][nb - small:] = p.args[1 + i].view(torch.uint8)
        exps[i][nb - small:] = p.args[3 + i]
    table = p.args[5].clone()
    owned = (table >= 0) & (table < small)
    table[owned] += nb - small
    table[~owned] = -1
    got = pa.decode_q8(p.args[0], *[x.view(torch.float8_e4m3fn) for x in big], *exps, table, p.args[6], SCALE, 1)
    torch.cuda.synchronize()
    assert torch.equal(got, want) and pa.read_device_status(clear=True) == 0


def test_attention_refuses():
    p = Problem([40, 20], 12, 2, 16, torch.float16, seed=87)
    p.upload()
    q, kc, vc, ke, ve, t, n = p.args
    start = torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV)
    cases = ((lambda: pa.decode_q8(q.float(), kc, vc, ke, ve, t, n, SCALE, 2), TypeError),
             (lambda: pa.decode_q8(q, kc.view(torch.uint8), vc, ke, ve, t, n, SCALE, 2), TypeError),
             (lambda: pa.decode_q8(q, kc, vc, ke.int(), ve, t, n, SCALE, 2), TypeError),
             (lambda: pa.decode_q8(q, kc, vc, ke, ve, t.long(), n, SCALE, 2), TypeError),
             (lambda: pa.decode_q8(q, kc, vc, ke, ve, t, n, SCALE, 1), ValueError),
             (lambda: pa.decode_q8(q[:1], kc, vc, ke, ve, t, n, SCALE, 2), ValueError),
             (lambda: pa.decode_q8(q[:, :, :64].contiguous(), kc, vc, ke, ve, t, n, SCALE, 2), ValueError),
             (lambda: pa.decode_q8(q.transpose(0, 1), kc, vc, ke, ve, t, n, SCALE, 2), ValueError),
             (lambda: pa.decode_q8(q, kc, vc, ke, ve, t[:1], n, SCALE, 2), ValueError),
             (lambda: pa.decode_q8(q, kc, vc, ke, ve, t, n, SCALE, 2, out=q[:1]), ValueError),
             (lambda: pa.decode_q8(q, kc, vc, ke, ve, t, n, SCALE, 2, out=q.float()), TypeError),
             (lambda: pa.decode_q8(q[:, :7].contiguous(), kc, vc, ke, ve, t, n, SCALE, 2), pa.PAError),
             (lambda: pa.multi_query_q8(q, kc, vc, ke, ve, t, n, start[:2], SCALE, 2, 1), ValueError),
             (lambda: pa.multi_query_q8(q, kc, vc, ke, ve, t, n, start, SCALE, 2, 6), pa.PAError),
             (lambda: pa.multi_query_q8(q, kc, vc, ke, ve, t, n, start, SCALE, 2, 0), pa.PAError),
             (lambda: pa.multi_query_q8(q, kc, vc, ke, ve, t, n, None, SCALE, 2, 1), TypeError))
    for call, error in cases:
        with pytest.raises(error):
            call()


def test_a_step_through_all_of_it():
    """Prefill in a chunk, decode steps and a draft's verification on one 8-bit cache: rotate, append,
    attend, compared at each step with the reference's cache and attention; then the whole context read
    back to 16 bits serves multi_query's tiles."""
    Hq, Hkv, block, dtype = 12, 2, 16, torch.float16
    nb, seqs = 40, 3
    rng = np.random.default_rng(90)
    tables = rng.permutation(nb)[:36].reshape(seqs, 12).astype(np.int32)
    t = torch.from_numpy(tables).to(DEV)
    f, m = pa.rope_frequencies(ref.D, scaling="yarn", factor=4.0, original_context=64)
    code = [np.zeros((nb, Hkv, block, ref.D), dtype=np.uint8) for _ in range(2)]
    exp = [np.zeros((nb, Hkv), dtype=np.int8) for _ in range(2)]
    dev = [torch.from_numpy(c.copy()).to(DEV).view(torch.float8_e4m3fn) for c in code]
    dev += [torch.from_numpy(e.copy()).to(DEV) for e in exp]
    lens = np.zeros(seqs, dtype=np.int32)
    gen = torch.Generator().manual_seed(91)
    steps = [[70, 9, 33], [1, 1, 1], [1, 1, 1], [5, 3, 1], [1, 1, 1]]
    for step, new in enumerate(steps):
        lens = lens + np.array(new, dtype=np.int32)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        x = torch.randn((int(start[-1]), Hq + 2 * Hkv, ref.D), generator=gen).to(dtype).to(DEV)
        q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
        pos = torch.from_numpy(np.concatenate([np.arange(L - n, L) for L, n in zip(lens, new)])).to(DEV)
        q, k = pa.rope(q, k, pos, f, magnitude=m)
        n_t, s_t = torch.from_numpy(lens).to(DEV), torch.from_numpy(start).to(DEV)
        pa.cache_append_q8(k, v, *dev, t, n_t, query_start=s_t, max_q=max(new))
        ref.append(ref.f64(k), ref.f64(v), *code, *exp, tables, lens, start, max(new))
        torch.cuda.synchronize()
        assert all(np.array_equal(ref.codes(a), b) for a, b in zip(dev[:2], code))
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(dev[2:], exp))
        if max(new) * Hq // Hkv <= 32:
            out = pa.multi_query_q8(q, *dev, t, n_t, s_t, SCALE, Hkv, max(new))
        else:          # a long chunk: the blocks read back, then the 16-bit tiles
            back = [torch.empty((nb, Hkv, block, ref.D), dtype=dtype, device=DEV) for _ in range(2)]
            ids = t.reshape(-1).contiguous()
            pa.read_blocks_q8(*dev, *back, ids, ids)
            out = pa.multi_query(q, *back, t, n_t, s_t, SCALE, Hkv, max(new))
        torch.cuda.synchronize()
        want, bound, owned = ref.attention(ref.f64(q), *code, *exp, tables, lens, SCALE, start, max(new))
        ref.check_attention(out, want, bound, owned)
        if step == 3:
            lens = lens - np.array([4, 1, 0], dtype=np.int32)      # drafts rejected: their slots are taken again
    assert pa.read_device_status(clear=True) == 0
