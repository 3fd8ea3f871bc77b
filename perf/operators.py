"""The 8-bit paged cache's operators as they are measured: rotary positions, the quantising append,
reading blocks back to 16 bits, and attention over the 8-bit cache (one or several query tokens).

An 8-bit cache holds e4m3 codes [NB, Hkv, B, 128] and one int8 exponent per (block, kv head); the
value of a code c is c * 2^e, with -60 <= e <= 60.

``run`` computes an operator in its plain form (elementary torch operations in 32 bits), or with
``own`` calls the library.  ``exact`` gives the same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

D = 128                      # head size of the cache
E_MIN, E_MAX = -60, 60       # range of a block's exponent
TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
F8 = torch.float8_e4m3fn


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------

def listed():
    return [
        # a decode step's rotation: one new token of each of 64 sequences, 12 query / 2 kv heads
        dict(name="rope_step_64", op="rope", tokens=64, q_heads=12, kv_heads=2, type="f16", rotary=128,
             interleaved=False, scaling="none", factor=1.0, far=2048),
        # a prefill chunk of a long-context model: 8192 tokens, half of each head rotated, frequencies
        # stretched to 32 times the trained context
        dict(name="rope_chunk_8192", op="rope", tokens=8192, q_heads=32, kv_heads=8, type="bf16", rotary=64,
             interleaved=True, scaling="yarn", factor=32.0, far=131072),
        # the decode step's cache write: 64 sequences, one token each, most blocks partly filled
        dict(name="append_step_64", op="append", seqs=64, kv_heads=2, block=16, type="f16", lens="uniform",
             ctx_min=16, ctx_max=2048, new_min=1, new_max=1, draw=2),
        # ragged continuous batch: none to a few dozen new tokens per sequence, large blocks
        dict(name="append_ragged_128", op="append", seqs=128, kv_heads=8, block=128, type="bf16", lens="uniform",
             ctx_min=65, ctx_max=1536, new_min=0, new_max=65, draw=3),
        # chunked prefill: 512 new tokens of 16 sequences of 4096
        dict(name="append_chunk_512", op="append", seqs=16, kv_heads=32, block=32, type="f16", lens="uniform",
             ctx_min=4096, ctx_max=4096, new_min=512, new_max=512, draw=4),
        # one sequence's blocks read back before a chunk is prefilled over them
        dict(name="read_one_2048", op="read", blocks=128, pool=160, kv_heads=2, block=16, type="f16"),
        # the contexts of a whole prefill batch: 16 x 4096 tokens of 32 heads
        dict(name="read_batch_65536", op="read", blocks=2048, pool=2458, kv_heads=32, block=32, type="bf16"),
        # the smallest decode: 4 sequences of 7 to 64 tokens
        dict(name="decode_tiny_4", op="decode", seqs=4, q_heads=12, kv_heads=2, block=16, type="f16", lens="uniform",
             ctx_min=7, ctx_max=64, new_min=1, new_max=1, draw=8),
        # the decode step: 64 sequences of 16 to 2048 tokens
        dict(name="decode_step_64", op="decode", seqs=64, q_heads=12, kv_heads=2, block=16, type="f16",
             lens="uniform", ctx_min=16, ctx_max=2048, new_min=1, new_max=1, draw=9),
        # many short chats without shared heads
        dict(name="decode_short_256", op="decode", seqs=256, q_heads=32, kv_heads=32, block=32, type="f16",
             lens="lognormal", ctx_min=1, ctx_max=2048, new_min=1, new_max=1, draw=10),
        # few long contexts
        dict(name="decode_long_16", op="decode", seqs=16, q_heads=32, kv_heads=8, block=64, type="bf16",
             lens="uniform", ctx_min=16384, ctx_max=16384, new_min=1, new_max=1, draw=11),
        # speculative verification: up to five new tokens per sequence, causal among themselves
        dict(name="verify_64", op="decode", seqs=64, q_heads=12, kv_heads=2, block=16, type="f16", lens="uniform",
             ctx_min=16, ctx_max=2048, new_min=1, new_max=5, draw=12),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rope", "append", "read", "decode", "decode"])
    kind = rng.choice(["f16", "bf16"])
    block = rng.choice([16, 32, 64, 128])
    if op == "rope":
        kv = rng.choice([1, 2, 4, 8])
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return dict(op="rope", tokens=_log_int(rng, 1, 8192), q_heads=kv * rng.choice([1, 3, 4]), kv_heads=kv,
                    type=kind, rotary=rng.choice([16, 32, 64, 96, 128]), interleaved=rng.random() < 0.5,
                    scaling=scaling, factor=1.0 if scaling == "none" else float(rng.choice([2, 8, 32])),
                    far=_log_int(rng, 64, 1 << 20))
    if op == "append":
        new = _log_int(rng, 1, 512)
        ctx = new + _log_int(rng, 1, 2048)
        seqs = _log_int(rng, 1, max(2, min(256, 8192 // new)))
        kv = rng.choice([1, 2, 8, 32]) if seqs * ctx <= 65536 else rng.choice([1, 2])
        return dict(op="append", seqs=seqs, kv_heads=kv, block=block, type=kind, lens="uniform",
                    ctx_min=new, ctx_max=ctx, new_min=rng.choice([0, new]), new_max=new, draw=rng.randrange(1 << 30))
    if op == "read":
        kv = rng.choice([1, 2, 8, 32])
        blocks = _log_int(rng, 1, max(2, 2048 * 1024 // (kv * block)))
        return dict(op="read", blocks=blocks, pool=blocks + _log_int(rng, 1, 64), kv_heads=kv, block=block,
                    type=kind)
    kv = rng.choice([1, 2, 8])
    group = rng.choice([1, 2, 3, 4, 6, 8, 16])
    new = rng.randint(1, max(1, 32 // group)) if rng.random() < 0.5 else 1
    ctx = max(new, _log_int(rng, 1, 32768))
    budget = 16 * 16384 // (1 if new * group <= 8 else 4)
    seqs = _log_int(rng, 1, max(1, min(256, budget // ctx)))
    return dict(op="decode", seqs=seqs, q_heads=kv * group, kv_heads=kv, block=block, type=kind,
                lens=rng.choice(["uniform", "lognormal"]), ctx_min=max(new, ctx // rng.choice([1, 4, 64])), ctx_max=ctx,
                new_min=rng.choice([1, new]), new_max=new, draw=rng.randrange(1 << 30))


def _lens(case):
    """Context lengths and new tokens of every sequence: part of the case, not of the values."""
    rng = random.Random(case["draw"])
    lo, hi = case["ctx_min"], case["ctx_max"]
    lens, new = [], []
    for _ in range(case["seqs"]):
        if case["lens"] == "lognormal":      # 90th percentile 287, as short chats have it
            x = int(round(math.exp(math.log(287.0) - 1.2815515655446004 * 0.75 + 0.75 * rng.gauss(0, 1))))
        else:
            x = rng.randint(lo, hi)
        lens.append(min(hi, max(lo, x)))
        new.append(min(lens[-1], rng.randint(case["new_min"], case["new_max"])))
    return lens, new


def work(case):
    if case["op"] == "rope":
        n = case["tokens"] * (case["q_heads"] + case["kv_heads"]) * D
        rot = n * case["rotary"] // D
        return {"bytes": 4.0 * n + 8 * case["tokens"], "flops": 3.0 * rot}
    if case["op"] == "read":
        n = 2.0 * case["blocks"] * case["kv_heads"] * case["block"] * D
        return {"bytes": 3 * n + 2 * case["blocks"] * (case["kv_heads"] + 4), "flops": n}
    lens, new = _lens(case)
    table = sum(4 * -(-x // case["block"]) for x in lens)
    if case["op"] == "append":
        n = 2.0 * sum(new) * case["kv_heads"] * D
        return {"bytes": 3 * n + 4 * sum(-(-x // case["block"]) + 1 for x in new) + 8 * case["seqs"], "flops": 3 * n}
    seen = [sum(x - n + i + 1 for i in range(n)) for x, n in zip(lens, new)]
    kv = 2.0 * sum(lens) * case["kv_heads"] * D + table / 4 * 2 * case["kv_heads"]
    io = 2.0 * 2 * sum(new) * case["q_heads"] * D
    return {"bytes": kv + io + table + 8 * case["seqs"], "flops": 4.0 * sum(seen) * case["q_heads"] * D}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------

def _quantised(shape, gen, dev):
    """A filled cache: rows with a few strong channels, as keys and values have them, quantised block by block."""
    nb, heads, block, d = shape
    codes = torch.empty(shape, dtype=F8, device=dev)
    exps = torch.empty((nb, heads), dtype=torch.int8, device=dev)
    channel = torch.exp(0.5 * torch.randn((1, heads, 1, d), generator=gen, device=dev))
    slab = max(1, (1 << 26) // (heads * block * d))
    for i in range(0, nb, slab):
        x = torch.randn((min(slab, nb - i), heads, block, d), generator=gen, device=dev) * channel
        e = _exponent(x.abs().amax((2, 3)))
        codes[i:i + slab] = (x * torch.exp2(-e.float())[:, :, None, None]).clamp(-448, 448).to(F8)
        exps[i:i + slab] = e.to(torch.int8)
    return codes, exps


def _exponent(amax):
    """The least e with amax <= 448 * 2^e (448 = 0.875 * 2^9, the largest e4m3 value)."""
    m, e = torch.frexp(amax)
    e = e.to(torch.int32) - 9 + (m > 0.875).to(torch.int32)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN)).clamp(E_MIN, E_MAX)


def _tables(lens, block, gen, dev):
    need = [-(-x // block) for x in lens]
    nb = max(1, math.ceil(1.2 * sum(need)))
    ids = torch.randperm(nb, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(1, max(need))), -1, dtype=torch.int32)
    host, at = ids.cpu(), 0
    for s, n in enumerate(need):
        table[s, :n] = host[at:at + n]
        at += n
    return table.to(dev), nb


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    s = {"case": dict(case)}
    kind = TYPES[case["type"]]

    def rows(n, heads):
        return torch.randn((n, heads, D), generator=gen, device=dev).to(kind)

    if case["op"] == "rope":
        t = case["tokens"]
        s.update(q=rows(t, case["q_heads"]), k=rows(t, case["kv_heads"]))
        s["positions"] = torch.randint(0, case["far"], (t,), generator=gen, device=dev)
        f, s["magnitude"] = _frequencies(case)
        s["inv_freq"] = torch.tensor(f, dtype=torch.float64, device=dev)     # a model keeps it with its weights
        return s
    if case["op"] == "read":
        shape = (case["pool"], case["kv_heads"], case["block"], D)
        s["k_cache"], s["k_exp"] = _quantised(shape, gen, dev)
        s["v_cache"], s["v_exp"] = _quantised(shape, gen, dev)
        s["src"] = torch.randperm(case["pool"], generator=gen, device=dev)[:case["blocks"]].to(torch.int32)
        s["dst"] = torch.randperm(case["blocks"], generator=gen, device=dev).to(torch.int32)
        s["k_out"] = torch.empty((case["blocks"],) + shape[1:], dtype=kind, device=dev)
        s["v_out"] = torch.empty_like(s["k_out"])
        return s
    lens, new = _lens(case)
    s["max_len"], s["max_q"] = max(lens), max(1, max(new))
    s["one_each"] = all(n == 1 for n in new)
    s["tables"], nb = _tables(lens, case["block"], gen, dev)
    s["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    start = [0]
    for n in new:
        start.append(start[-1] + n)
    s["start"] = torch.tensor(start, dtype=torch.int32, device=dev)
    shape = (nb, case["kv_heads"], case["block"], D)
    s["k_cache"], s["k_exp"] = _quantised(shape, gen, dev)
    s["v_cache"], s["v_exp"] = _quantised(shape, gen, dev)
    if case["op"] == "append":
        s["k"], s["v"] = rows(start[-1], case["kv_heads"]), rows(start[-1], case["kv_heads"])
    else:
        s["q"] = rows(start[-1], case["q_heads"])
        s["scale"] = 1.0 / math.sqrt(D)
    return s


# ---------------------------------------------------------------------------------------------
# rotary frequencies: theta_i = base^(-2 i / R), and their scaled forms
# ---------------------------------------------------------------------------------------------

BASE, TRAINED = 10000.0, 4096


def _frequencies(case):
    rot, factor, scaling = case["rotary"], case["factor"], case["scaling"]
    base = BASE
    if scaling == "ntk":         # the base moves so that the slowest pair turns `factor` times slower
        base = BASE * factor ** (rot / (rot - 2.0))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if scaling == "linear":
        return [x / factor for x in f], 1.0
    if scaling != "yarn":
        return f, 1.0

    # yarn: pairs that turn more than 32 times within the trained context stay, those that turn less
    # than once are slowed by `factor`, a ramp in the pair's index between; weights sharpened by a magnitude
    def pair_of(turns):
        return rot * math.log(TRAINED / (turns * 2 * math.pi)) / (2 * math.log(BASE))

    lo, hi = max(0, math.floor(pair_of(32.0))), min(rot - 1, math.ceil(pair_of(1.0)))
    hi = hi if hi > lo else lo + 0.001
    ramp = [min(1.0, max(0.0, (i - lo) / (hi - lo))) for i in range(rot // 2)]
    return [x * (1 - r) + x / factor * r for x, r in zip(f, ramp)], 0.1 * math.log(factor) + 1.0


# ---------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------

def run(s):
    return (_own if own else _plain)[s["case"]["op"]](s)


def _own_rope(s):
    import paged_kv_cache_08_gb300 as pa
    return pa.rope(s["q"], s["k"], s["positions"], s["inv_freq"], magnitude=s["magnitude"],
                   interleaved=s["case"]["interleaved"])


def _own_append(s):
    import paged_kv_cache_08_gb300 as pa
    if s["one_each"]:
        pa.cache_append_q8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], s["tables"], s["lens"])
    else:
        pa.cache_append_q8(s["k"], s["v"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], s["tables"], s["lens"],
                           query_start=s["start"], max_q=s["max_q"])
    return s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"]


def _own_read(s):
    import paged_kv_cache_08_gb300 as pa
    pa.read_blocks_q8(s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], s["k_out"], s["v_out"], s["src"], s["dst"])
    return s["k_out"], s["v_out"]


def _own_decode(s):
    import paged_kv_cache_08_gb300 as pa
    if s["one_each"]:
        return pa.decode_q8(s["q"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], s["tables"], s["lens"],
                            s["scale"], s["case"]["kv_heads"])
    return pa.multi_query_q8(s["q"], s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"], s["tables"], s["lens"],
                             s["start"], s["scale"], s["case"]["kv_heads"], s["max_q"])


def _plain_rope(s):
    rot, inter = s["case"]["rotary"], s["case"]["interleaved"]
    # far positions: the angle in 64 bits, its cosine and sine rounded to 32
    angle = s["positions"].double()[:, None] * s["inv_freq"][None, :]
    cos, sin = torch.cos(angle).float()[:, None, :], torch.sin(angle).float()[:, None, :]

    def turned(x):
        f = x.float()
        y = f.clone()
        a, b = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
        y[..., a] = (f[..., a] * cos - f[..., b] * sin) * s["magnitude"]
        y[..., b] = (f[..., b] * cos + f[..., a] * sin) * s["magnitude"]
        return y.to(x.dtype)

    return turned(s["q"]), turned(s["k"])


def _rows(s, n):
    """Sequence and position of each of the n new rows."""
    start = s["start"].long()
    row = torch.arange(n, device=start.device)
    seq = torch.searchsorted(start[1:].contiguous(), row, right=True)
    pos = s["lens"].long()[seq] - (start[seq + 1] - row)
    return seq, pos


def _plain_append(s):
    block = s["case"]["block"]
    seq, pos = _rows(s, s["k"].shape[0])
    blk, off = s["tables"].long()[seq, pos // block], pos % block
    touched = torch.zeros(s["k_cache"].shape[0], dtype=torch.bool, device=blk.device)
    touched[blk] = True
    first = torch.full_like(touched, block, dtype=torch.int64).scatter_reduce(0, blk, off, "amin")
    slots = torch.arange(block, device=blk.device)
    for x, codes, exps in ((s["k"], s["k_cache"], s["k_exp"]), (s["v"], s["v_cache"], s["v_exp"])):
        f = x.float()
        need = _exponent(f.abs().amax(-1))
        e = torch.full(exps.shape, E_MIN, dtype=torch.int32, device=f.device)
        e = e.scatter_reduce(0, blk[:, None].expand_as(need), need, "amax")
        old = exps.int()
        e = torch.where((first == 0)[:, None], e, torch.maximum(e, old))
        # rows before the first new one move to the grown exponent
        b = torch.nonzero(touched & (first > 0)).squeeze(1)
        kept = (codes[b].float() * torch.exp2((old[b] - e[b]).float())[:, :, None, None]).clamp(-448, 448).to(F8)
        keep = (slots[None] < first[b][:, None])[:, None, :, None]
        codes[b] = torch.where(keep, kept.view(torch.uint8), codes[b].view(torch.uint8)).view(F8)
        scale = torch.exp2(-e[blk].float())[:, :, None]
        codes.view(torch.uint8)[blk, :, off] = (f * scale).clamp(-448, 448).to(F8).view(torch.uint8)
        exps.copy_(torch.where(touched[:, None], e, old).to(torch.int8))
    return s["k_cache"], s["v_cache"], s["k_exp"], s["v_exp"]


def _plain_read(s):
    src, dst = s["src"].long(), s["dst"].long()
    for codes, exps, out in ((s["k_cache"], s["k_exp"], s["k_out"]), (s["v_cache"], s["v_exp"], s["v_out"])):
        c = codes.view(torch.uint8)[src].view(F8).float()
        out[dst] = (c * torch.exp2(exps[src].float())[:, :, None, None]).to(out.dtype)
    return s["k_out"], s["v_out"]


def _plain_decode(s):
    case = s["case"]
    hkv, group = case["kv_heads"], case["q_heads"] // case["kv_heads"]
    block, kind = case["block"], s["q"].dtype
    nblk = -(-s["max_len"] // block)
    table = s["tables"].long()[:, :nblk].clamp(min=0)
    lens, start = s["lens"].long(), s["start"].long()
    n = start[1:] - start[:-1]
    seqs, t = lens.numel(), nblk * block
    at = torch.arange(t, device=lens.device)
    there = (at[None] < lens[:, None])[:, None, :, None]

    def values(codes, exps):
        c = codes.view(torch.uint8)[table].view(F8).float()                        # [S, nblk, Hkv, B, D]
        c = c * torch.exp2(exps[table].float())[..., None, None]
        c = c.permute(0, 2, 1, 3, 4).reshape(seqs, hkv, t, D)
        return torch.where(there, c, torch.zeros((), device=c.device))

    row = (start[:-1, None] + torch.arange(s["max_q"], device=lens.device)[None]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float()                                                        # [S, max_q, Hq, D]
    q = q.reshape(seqs, s["max_q"], hkv, group, D).permute(0, 2, 1, 3, 4).reshape(seqs, hkv, s["max_q"] * group, D)
    score = torch.matmul(q, values(s["k_cache"], s["k_exp"]).transpose(2, 3)) * s["scale"]
    own_pos = (lens - n)[:, None] + torch.arange(s["max_q"], device=lens.device)[None]
    seen = (at[None, None] <= own_pos[:, :, None])[:, None, :, None, :]            # [S, 1, max_q, 1, T]
    score = score.reshape(seqs, hkv, s["max_q"], group, t).masked_fill(~seen, -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).reshape(seqs, hkv, s["max_q"] * group, t)
    out = torch.matmul(p, values(s["v_cache"], s["v_exp"])).to(kind)
    out = out.reshape(seqs, hkv, s["max_q"], group, D).permute(0, 2, 1, 3, 4).reshape(seqs, s["max_q"], hkv * group, D)
    r = torch.arange(s["q"].shape[0], device=lens.device)
    seq = torch.searchsorted(start[1:].contiguous(), r, right=True)
    return out[seq, r - start[seq]]


_plain = {"rope": _plain_rope, "append": _plain_append, "read": _plain_read, "decode": _plain_decode}
_own = {"rope": _own_rope, "append": _own_append, "read": _own_read, "decode": _own_decode}


# ---------------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------------

def exact(case, seed):
    return _exact[case["op"]](case, prepare(case, seed))


def _exact_rope(case, s):
    rot = case["rotary"]
    f, m = _frequencies(case)
    turn = torch.exp(1j * s["positions"].double()[:, None].cpu() * torch.tensor(f, dtype=torch.float64)[None]) * m
    turn = turn.to(s["q"].device)[:, None]
    done = []
    for x in (s["q"], s["k"]):
        y = x.double().clone()
        r = y[..., :rot]
        r = r.unflatten(-1, (rot // 2, 2)) if case["interleaved"] else r.unflatten(-1, (2, rot // 2)).transpose(-1, -2)
        z = torch.complex(r[..., 0].contiguous(), r[..., 1].contiguous()) * turn
        z = torch.view_as_real(z)
        y[..., :rot] = (z if case["interleaved"] else z.transpose(-1, -2)).flatten(-2)
        done.append(y)
    return tuple(done)


def _e4m3(x):
    """Nearest e4m3 value of each x, ties to even: steps of 2^(exponent - 3), the exponent at least -6."""
    _, e = torch.frexp(x)
    step = torch.exp2((e.double() - 1).clamp(min=-6) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_append(case, s):
    """Sequence by sequence and block by block: every (block, head)'s exponent, then its codes.
    The exponents are whole numbers, which have no 64-bit form of their own."""
    block = case["block"]
    lens, new = _lens(case)
    table = s["tables"].cpu()
    jobs = [(int(table[i, j]), max(0, x - n - j * block), min(block, x - j * block), j * block - (x - n), i)
            for i, (x, n) in enumerate(zip(lens, new)) if n for j in range((x - n) // block, (x - 1) // block + 1)]
    start = s["start"].cpu().tolist()
    done = []
    for x, codes, exps in ((s["k"], s["k_cache"], s["k_exp"]), (s["v"], s["v_cache"], s["v_exp"])):
        out = codes.float()                     # codes are e4m3 values: a float holds them exactly
        for b, lo, hi, shift, i in jobs:
            r = x[start[i] + shift + lo:start[i] + shift + hi].double().transpose(0, 1)      # [Hkv, rows, D]
            e = torch.ceil(torch.log2(r.abs().amax((1, 2)) / 448)).clamp(E_MIN, E_MAX)
            if lo:
                e = torch.maximum(e, exps[b].double())
                out[b, :, :lo] = _e4m3(out[b, :, :lo].double() * torch.exp2(exps[b].double() - e)[:, None, None]).float()
            out[b, :, lo:hi] = _e4m3(r * torch.exp2(-e)[:, None, None]).float()
        done.append(out)
    return done[0], done[1], None, None


def _exact_read(case, s):
    done = []
    for codes, exps in ((s["k_cache"], s["k_exp"]), (s["v_cache"], s["v_exp"])):
        v = codes.double() * torch.pow(2.0, exps.double())[:, :, None, None]
        out = torch.empty((case["blocks"],) + tuple(v.shape[1:]), dtype=torch.float64, device=v.device)
        out[s["dst"].long()] = v[s["src"].long()]
        done.append(out)
    return tuple(done)


def _exact_decode(case, s):
    lens, new = _lens(case)
    hkv, group, block = case["kv_heads"], case["q_heads"] // case["kv_heads"], case["block"]
    out = torch.empty(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    at = 0
    for i, (x, n) in enumerate(zip(lens, new)):
        ids = s["tables"][i, :-(-x // block)].long()

        def rows(codes, exps):
            c = codes.view(torch.uint8)[ids].view(F8).to(torch.float64) * torch.exp2(exps[ids].double())[:, :, None, None]
            return c.transpose(0, 1).reshape(hkv, -1, D)[:, :x]

        k, v = rows(s["k_cache"], s["k_exp"]), rows(s["v_cache"], s["v_exp"])
        for j in range(n):
            q = s["q"][at + j].double().reshape(hkv, group, D)
            upto = x - n + j + 1
            p = torch.softmax(q @ k[:, :upto].transpose(1, 2) * s["scale"], -1)
            out[at + j] = (p @ v[:, :upto]).reshape(hkv * group, D)
        at += n
    return out


_exact = {"rope": _exact_rope, "append": _exact_append, "read": _exact_read, "decode": _exact_decode}
