"""Attention over the 8-bit cache in the grid of twelve warps a CTA, which calls with many segments (a sequence's kv head
each) of up to eight rows take: its ring, its joins and its cuts differ from those of eight warps."""
import numpy as np
import pytest
import torch

import paged_kv_cache_08_gb300 as pa
from test_gpu_decode_q8 import Problem

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _clean_status():
    pa.read_device_status(clear=True)
    yield


def _enough(S, Hkv, rows):
    """Two segments and more for each of eight warps of every SM, of eight rows at most: the rule for twelve."""
    assert rows <= 8 and S * Hkv >= 2 * 8 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("group,n,block", [(1, 1, 64), (3, 1, 16), (8, 1, 64), (8, 1, 16), (1, 8, 16), (3, 2, 64)])
@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_many_segments(dtype, group, n, block):
    rng = np.random.default_rng(10 * group + n)
    lens = rng.integers(0, 50, 640)
    lens[[3, 500]] = 700, 2900               # two that are cut many times
    new = None if n == 1 else np.minimum(lens, rng.integers(0, n + 1, 640))
    if new is not None:
        new[500] = n
    _enough(640, 4, group * n)
    Problem(lens.tolist(), 4 * group, 4, block, dtype, new=None if new is None else new.tolist(), seed=200 + group).run()


@pytest.mark.parametrize("dtype,new", [(torch.float16, False), (torch.bfloat16, False), (torch.bfloat16, True)])
def test_more_sequences_than_a_launch_takes(dtype, new):
    rng = np.random.default_rng(31)
    lens = rng.integers(0, 50, 1400)
    lens[[0, 1023, 1024, 1399]] = 700, 300, 33, 900
    n = np.minimum(lens, rng.integers(0, 3, 1400)).tolist() if new else None
    _enough(1400, 2, 4)
    Problem(lens.tolist(), 4, 2, 16, dtype, new=n, seed=31).run()


@pytest.mark.parametrize("seed", range(6))
def test_shares_cut_anywhere(seed):
    """Batches and tables of random sizes, so that shares begin and end at every place of a segment."""
    rng = np.random.default_rng(700 + seed)
    Hkv, group = int(rng.choice([4, 6, 8])), int(rng.integers(1, 9))
    S = -(-2 * 8 * torch.cuda.get_device_properties(0).multi_processor_count // Hkv) + int(rng.integers(0, 40))
    lens = rng.integers(0, int(rng.choice([20, 60, 100])), S)
    lens[rng.random(S) < 0.3] = rng.integers(0, 33)
    lens[int(rng.integers(0, S))] = int(rng.integers(300, 2500))
    new = None if seed % 2 else np.minimum(lens, rng.integers(0, 8 // group + 1, S)).tolist()
    p = Problem(lens.tolist(), Hkv * group, Hkv, int(rng.choice([16, 32, 64, 128])), [torch.float16, torch.bfloat16][seed // 2 % 2],
                new=new, seed=seed)
    if seed % 4 == 1:
        p.tables = np.concatenate([p.tables, np.full((S, 400), -1, dtype=np.int32)], 1)
    _enough(S, Hkv, group * p.max_q)
    p.run()


def test_the_call_repeats_bit_for_bit():
    rng = np.random.default_rng(44)
    p = Problem(rng.integers(0, 90, 620).tolist(), 12, 4, 32, torch.float16, seed=44)
    _enough(620, 4, 3)
    first = p.run()
    for _ in range(5):
        assert torch.equal(p.call(), first)
