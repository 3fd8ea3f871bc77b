"""Rotary positions whose angles are small: slow pairs near position 0 of a model with a large base and stretched
frequencies.  The turned element that starts at zero is then the angle itself, and keeps the type's precision."""
import numpy as np
import pytest
import torch

import paged_kv_cache_08_gb300 as pa
import q8_reference as ref

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda")


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_small_angles_keep_their_precision(dtype, interleaved):
    """(a, 0) turns to a (cos, sin).  The sine's bound, relative to the angle t = p f with |t| < 1: the phase
    |p| (|f| 2^-52 + 2^-62) and its rounding t 2^-23; sincospi 2 ulp, 2^-22; the product and the sum 2^-23; below 2^-21 t +
    |p| 2^-61 together.  Then the rounding to the type."""
    f = torch.tensor([2.0 ** -4, 1e-4, 1e-6, 4e-8, 3e-9, -1e-9, 2e-10, -1e-12], dtype=torch.float64)
    pos = torch.tensor([0, 1, -1, 2, 3, 7, -12, 15])
    a = 1024.0 if dtype is torch.float16 else 1.5    # fp16: the smallest angles' sines fall into its subnormals
    q = torch.zeros((len(pos), 3, 128), dtype=dtype)
    at_a, at_b = (slice(0, 16, 2), slice(1, 16, 2)) if interleaved else (slice(0, 8), slice(8, 16))
    q[:, :, at_a] = a
    out, _ = pa.rope(q.to(DEV), None, pos.to(DEV), f.to(DEV), interleaved=interleaved)
    torch.cuda.synchronize()
    got, angle = ref.f64(out), pos.double().numpy()[:, None] * f.numpy()[None]
    for part, want in ((at_a, a * np.cos(angle)), (at_b, a * np.sin(angle))):
        bound = a * (2.0 ** -21 * np.maximum(np.abs(angle), np.abs(want) / a) + np.abs(pos.numpy())[:, None] * 2.0 ** -61)
        y = got[:, :, part]
        excess = np.abs(y - want[:, None]) - (bound + ref.half_step(np.abs(want) + bound, dtype))[:, None]
        assert excess.max() <= 0, f"beyond the bound by {excess.max():.3e}"
    assert (got[:, :, 16:] == 0).all()


def test_a_half_turn_and_a_whole_one():
    """Phases at the ends of the reduced range: half a turn, and just below it."""
    f = torch.tensor([np.pi, np.pi * (1 - 2.0 ** -40), -np.pi, 2 * np.pi, np.pi / 2, 1.5 * np.pi, 0.0, 3 * np.pi],
                     dtype=torch.float64)
    pos = torch.tensor([1, 2, 3, -1, 2**31 - 1])
    gen = torch.Generator().manual_seed(1)
    q = torch.randn((len(pos), 2, 32), generator=gen).to(torch.float16)
    out, _ = pa.rope(q.to(DEV), None, pos.to(DEV), f.to(DEV))
    torch.cuda.synchronize()
    want, bound = ref.rope(ref.f64(q), pos.tolist(), f.tolist(), 1.0, False)
    got = ref.f64(out)
    excess = np.abs(got - want) - (bound + ref.half_step(np.abs(want) + bound, torch.float16))
    assert excess.max() <= 0
