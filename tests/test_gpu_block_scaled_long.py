"""Attention over a block-scaled cache where one warp walks many tiles: pairs of them and the odd
one after, the ring of stages reused, the scales' window moved on (every 32 tiles of a warp),
against 64 bits.  Neighbouring blocks' scales lie up to six binary orders apart."""
import numpy as np
import pytest
import torch

from tests.test_gpu_block_scaled import DT, check, filled, pa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

# groups of one and two rows take the CUDA cores, 3 to 8 pairs of tiles, more single tiles
ROWS = [(1, 1), (1, 2), (1, 4), (1, 8), (2, 2), (3, 1), (4, 1), (4, 2), (1, 12), (5, 4)]


def queries(rng, n, q_len, heads, dtype):
    return torch.from_numpy(rng.standard_normal((n, q_len, heads, 128)) * 3).to(DT[dtype])


@pytest.mark.parametrize("bs,dtype", [(8, "bf16"), (16, "fp16"), (16, "bf16"), (32, "bf16")])
@pytest.mark.parametrize("q_len,group", ROWS)
def test_partitions(pa, bs, dtype, q_len, group):  # noqa: F811
    """A partition is one thread block of three or four warps: 60 to 110 tiles a warp in
    one part of two, odd and even numbers, the last row anywhere in a pair's tiles."""
    rng = np.random.default_rng(bs * 100 + q_len * 10 + group)
    h = 2
    lens = [5300 + int(rng.integers(0, 700)) for _ in range(2)] + [40, 0, 9001 + int(rng.integers(0, 64)), 1023]
    state = filled(rng, lens, h, bs, 9088 // bs, spread=6)
    check(pa, rng, state, queries(rng, len(lens), q_len, h * group, dtype), lens, 0.3, dtype, num_splits=2)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("bs,dtype", [(8, "fp16"), (16, "bf16"), (32, "fp16")])
@pytest.mark.parametrize("q_len,group", [(1, 1), (1, 4), (4, 1), (2, 2), (1, 12)])
def test_one_pass_of_many_units(pa, bs, dtype, q_len, group):  # noqa: F811
    """912 units: single thread blocks, of which a few walk long sequences alone (up to 75 tiles
    a warp)."""
    rng = np.random.default_rng(bs * 10 + group)
    n, h = 114, 8
    lens = [int(rng.integers(1, 60)) for _ in range(n)]
    for i, length in ((3, 4100), (50, 4790), (77, 2049), (113, 3333)):
        lens[i] = length + int(rng.integers(0, 33))
    state = filled(rng, lens, h, bs, 4832 // bs, spread=6)
    check(pa, rng, state, queries(rng, n, q_len, h * group, dtype), lens, 0.3, dtype)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("q_len,group", [(1, 1), (1, 4), (4, 2), (1, 16)])
def test_one_long_sequence(pa, bs, q_len, group):  # noqa: F811
    """One unit in a cluster of eight thread blocks: 24 warps, 33 to 43 tiles each."""
    rng = np.random.default_rng(bs + group)
    for length in (12800 + int(rng.integers(0, 200)), 16384 - int(rng.integers(0, 40))):
        state = filled(rng, [length], 1, bs, 16384 // bs, spread=6)
        check(pa, rng, state, queries(rng, 1, q_len, group, "bf16"), [length], 0.3, "bf16")
    assert pa.pa_device_error() == 0
