"""Many-row attention over a block-scaled cache where a thread block takes several units of odd
and even numbers of chunks, each with scales of its own."""
import numpy as np
import pytest
import torch

from tests.test_gpu_block_scaled import DT, check, filled, pa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs,dtype", [(8, "bf16"), (16, "fp16"), (16, "bf16"), (32, "fp16")])
@pytest.mark.parametrize("chunks", [(1,), (3,), (1, 2, 3), (5, 1, 3)])
def test_units_after_odd_numbers_of_chunks(pa, bs, dtype, chunks):  # noqa: F811
    """44 sequences of 8 KV heads are 352 units of up to 128 rows, more than two a thread block
    of 152; a chunk is 128 positions."""
    rng = np.random.default_rng(bs + len(chunks) + chunks[0])
    n, h, q_len = 44, 8, 17
    lens = [128 * chunks[i % len(chunks)] - int(rng.integers(0, 100)) for i in range(n)]
    state = filled(rng, lens, h, bs, 640 // bs, spread=6)
    q = torch.from_numpy(rng.standard_normal((n, q_len, h, 128)) * 3).to(DT[dtype])
    check(pa, rng, state, q, lens, 0.5, dtype)
    assert pa.pa_device_error() == 0
