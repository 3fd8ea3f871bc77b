"""Plain 64-bit forms of the rotary positions and the 8-bit cache's operators (CPU, numpy), written
from their definitions, and the error bounds that the GPU tests hold the kernels to."""
import math
from fractions import Fraction

import numpy as np
import torch

D = 128
E_MIN, E_MAX = -60, 60
# 2 pi to 60 digits
TWO_PI = 2 * Fraction("3.14159265358979323846264338327950288419716939937510582097494")


# ---- e4m3 ----------------------------------------------------------------------------------

def _code_value(c: int) -> float:
    sign, e, m = c >> 7, (c >> 3) & 15, c & 7
    if e == 15 and m == 7:
        return math.nan
    v = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
    return -v if sign else v


CODE_VALUES = np.array([_code_value(c) for c in range(256)])
_POSITIVE = CODE_VALUES[:127]                      # ascending: 0 .. 448


def to_code(x: np.ndarray) -> np.ndarray:
    """Nearest code of each x, ties to the even code, beyond 448 to +-448, NaN to 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    a = np.minimum(np.abs(x), 448.0)
    hi = np.clip(np.searchsorted(_POSITIVE, np.nan_to_num(a), side="left"), 0, 126)
    lo = np.maximum(hi - 1, 0)
    d_lo, d_hi = np.nan_to_num(a) - _POSITIVE[lo], _POSITIVE[hi] - np.nan_to_num(a)
    code = np.where((d_lo < d_hi) | ((d_lo == d_hi) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(x), code | 0x80, code)
    return np.where(np.isnan(x), 0x7F, code).astype(np.uint8)


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().to(torch.float64).numpy()


def codes(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().view(torch.uint8).numpy().copy()


def values(code: np.ndarray, exp: np.ndarray) -> np.ndarray:
    """Values of codes [NB, H, B, D] under exponents [NB, H]."""
    e = np.clip(exp.astype(np.int64), E_MIN, E_MAX)
    return CODE_VALUES[code] * np.exp2(e.astype(np.float64))[:, :, None, None]


# ---- append --------------------------------------------------------------------------------

def exponent_for(x: np.ndarray) -> int:
    """Least e in range with amax <= 448 * 2^e over the finite |x|."""
    a = np.abs(x[np.isfinite(x)])
    amax = a.max() if a.size else 0.0
    e = E_MIN
    while e < E_MAX and amax > 448.0 * 2.0 ** e:
        e += 1
    return e


def append(k, v, k_code, v_code, k_exp, v_exp, tables, lens, query_start=None, max_q=1):
    """In place on numpy arrays: the caches' codes and exponents after the append."""
    nb, heads, block, _ = k_code.shape
    for s, L in enumerate(lens):
        L = max(0, min(int(L), tables.shape[1] * block))
        if query_start is None:
            row0, n = s, min(1, L)
        else:
            row0 = max(0, min(int(query_start[s]), k.shape[0]))
            n = max(0, min(int(query_start[s + 1]) - int(query_start[s]), k.shape[0] - row0, L, max_q))
        if n == 0:
            continue
        p0 = L - n
        for j in range(p0 // block, (L - 1) // block + 1):
            b = int(tables[s, j])
            if not 0 <= b < nb:
                continue
            lo, hi = max(0, p0 - j * block), min(block, L - j * block)
            rows = slice(row0 + j * block + lo - p0, row0 + j * block + hi - p0)
            for x, code, exp in ((k, k_code, k_exp), (v, v_code, v_exp)):
                for h in range(heads):
                    new = x[rows, h]
                    e, old = exponent_for(new), int(np.clip(exp[b, h], E_MIN, E_MAX))
                    if lo:
                        e = max(e, old)
                        if e > old:
                            code[b, h, :lo] = to_code(CODE_VALUES[code[b, h, :lo]] * 2.0 ** (old - e))
                    code[b, h, lo:hi] = to_code(new * 2.0 ** -e)
                    exp[b, h] = e


# ---- attention -----------------------------------------------------------------------------

def attention(q, k_code, v_code, k_exp, v_exp, tables, lens, scale, query_start=None, max_q=1):
    """(out, bound): the outputs in 64 bits and how far a kernel may be from them before it rounds.

    The bound counts, for a row with weights w_t: the weights' rounding to fp16, half a step 2^-11 of
    each, 2^-25 under fp16's normal range (relative to the largest w_t 2^ve_t); the score's fp32 sum of
    128 products and its scaling, (128 + 4) 2^-24 sum |q k| scale, which moves a weight and the sum of
    weights by that factor each; the exponential, 2^-21; and the fp32 sums over L tokens, 16 a product and
    then pieces, where a tensor-core product may cut its sum off two bits early: (L / 16 + 64) 2^-22.
    NaN where the definition gives NaN."""
    nb, heads, block, _ = k_code.shape
    rows, hq, _ = q.shape
    group = hq // heads
    out = np.full(q.shape, np.nan)
    bound = np.zeros(q.shape)
    owned = np.zeros(rows, dtype=bool)
    for s, L in enumerate(lens):
        L = max(0, min(int(L), tables.shape[1] * block))
        if query_start is None:
            row0, n, p0 = s, 1, L - 1
        else:
            row0 = max(0, min(int(query_start[s]), rows))
            n = max(0, min(int(query_start[s + 1]) - int(query_start[s]), rows - row0, L, max_q))
            p0 = L - n
        ids = tables[s, :-(-L // block)].astype(np.int64)
        good = (ids >= 0) & (ids < nb)
        there = np.repeat(good, block)[:L]
        safe = np.where(good, ids, 0)

        def gathered(code, exp):
            e = np.clip(exp[safe].astype(np.float64), E_MIN, E_MAX)
            c = CODE_VALUES[code[safe]].transpose(1, 0, 2, 3).reshape(heads, -1, D)[:, :L]
            return c, np.repeat(np.exp2(e).T, block, axis=1)[:, :L]

        kc, ks = gathered(k_code, k_exp)
        vc, vs = gathered(v_code, v_exp)
        for i in range(n):
            owned[row0 + i] = True
            t = np.nonzero(there[:max(0, p0 + i + 1)])[0]
            if t.size == 0:
                out[row0 + i] = 0.0
                continue
            for h in range(hq):
                g = h // group
                qk = q[row0 + i, h] * kc[g, t]
                score = qk.sum(-1) * ks[g, t] * scale
                w = np.exp(score - score.max())
                w /= w.sum()
                cv, sv = vc[g, t], vs[g, t][:, None]
                out[row0 + i, h] = (w[:, None] * cv * sv).sum(0)
                ds = 132 * 2.0 ** -24 * (np.abs(qk).sum(-1) * ks[g, t] * abs(scale)).max()
                rel = 2.0 ** -11 + 2 * ds + 2.0 ** -20 + (t.size / 16 + 64) * 2.0 ** -22
                bound[row0 + i, h] = (rel * (w[:, None] * np.abs(cv) * sv).sum(0) +
                                      2.0 ** -25 * np.abs(cv).sum(0) * (w * vs[g, t]).max())
    return out, bound, owned


def half_step(ref: np.ndarray, dtype: torch.dtype) -> np.ndarray:
    """Half a step of `dtype` at ref's values (half the smallest step below the normal range)."""
    info = torch.finfo(dtype)
    return np.maximum(np.abs(ref) * info.eps / 2, info.smallest_normal * info.eps / 2)


def check_attention(got: torch.Tensor, ref, bound, owned):
    y = f64(got)
    r, b = ref[owned], bound[owned]
    y = y[owned]
    assert np.array_equal(np.isnan(y), np.isnan(r)), "NaN in other places than the definition's"
    # a value of (1 + eps / 4) max and more rounds to infinity in the output's type
    top = torch.finfo(got.dtype).max * (1 + torch.finfo(got.dtype).eps / 4)
    overflow = np.isinf(y) & (np.sign(y) == np.sign(r)) & (np.abs(r) + b >= top)
    fine = ~np.isnan(r) & ~overflow
    # the rounding at the end acts on a value that is `bound` away
    excess = np.abs(y - r)[fine] - (b + half_step(np.abs(r) + b, got.dtype))[fine]
    assert excess.size == 0 or excess.max() <= 0, f"beyond the bound by {excess.max():.3e}"


# ---- rotary positions ----------------------------------------------------------------------

def rope_angles(positions, inv_freq) -> np.ndarray:
    """Angles reduced to [0, 2 pi) in exact arithmetic, then in 64 bits: [T, R/2]."""
    f = [Fraction(float(x)) for x in inv_freq]
    return np.array([[float((int(p) * x) % TWO_PI) for x in f] for p in positions]).reshape(len(positions), len(f))


def rope(x, positions, inv_freq, magnitude, interleaved):
    """(values in 64 bits, bound before the final rounding).

    The angle: its phase rounded to 24 bits of a half turn, pi 2^-25, and |p f| 2^-52; sine and
    cosine 2 ulp, 2^-23; four fp32 roundings 2^-24.  Together below 2^-20 + |p f| 2^-52 of |a| + |b|."""
    angle = rope_angles(positions, inv_freq)
    R = 2 * len(inv_freq)
    y, bound = x.copy(), np.zeros_like(x)
    a, b = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    c, s = np.cos(angle)[:, None], np.sin(angle)[:, None]
    y[..., a] = magnitude * (x[..., a] * c - x[..., b] * s)
    y[..., b] = magnitude * (x[..., b] * c + x[..., a] * s)
    far = np.abs(np.asarray(positions, dtype=np.float64)[:, None] * np.asarray(inv_freq)[None])[:, None]
    off = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(magnitude) * (2.0 ** -20 + far * 2.0 ** -52)
    bound[..., a] = off
    bound[..., b] = off
    return y, bound
