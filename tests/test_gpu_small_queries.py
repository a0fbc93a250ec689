"""Query rows of subnormal bf16 values over FP8 caches: their scores are nothing, their weights
equal."""
import numpy as np
import pytest
import torch

from tests import _pool_ref as ref
from tests.test_gpu_block_scaled import DEV, check, filled, on, pa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

LENS = (40, 1, 130, 0)


def rows(rng, q_len, heads):
    """Rows of magnitudes 2^-133 to 2^-120, one of ordinary values and one of zeros among them."""
    q = rng.standard_normal((len(LENS), q_len, heads, 128)).clip(-2, 2)
    q *= 2.0 ** rng.integers(-133, -119, (len(LENS), q_len, heads, 1))
    q[2, -1, 1], q[2, -1, 2] = rng.standard_normal(128), 0
    return torch.from_numpy(q).to(torch.bfloat16)


@pytest.mark.parametrize("q_len,group", [(1, 1), (1, 4), (1, 12), (3, 4), (40, 2)])
def test_block_scaled(pa, q_len, group):  # noqa: F811
    rng = np.random.default_rng(group)
    state = filled(rng, LENS, 3, 16, 9)
    for splits in (1, 2):
        check(pa, rng, state, rows(rng, q_len, 3 * group), LENS, 0.09, "bf16", num_splits=splits)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("q_len,group", [(1, 4), (1, 12), (40, 2)])
def test_scales_a_head(pa, q_len, group):  # noqa: F811
    """The same over a cache of one scale a head; fp32 sums of up to 130 rows of 448 s at most,
    weights of 16 bits (2^-11 of sum w |v| each and in sum), half a step of bf16."""
    rng = np.random.default_rng(group)
    kc, vc, _, tables = filled(rng, LENS, 3, 16, 9)
    scale = np.full(3, 2.0 ** -9, np.float32)
    every = np.tile(scale[:, None], (len(kc), 1, 2))
    q = rows(rng, q_len, 3 * group).to(DEV)
    out = torch.full_like(q, float("nan"))
    pa.pa_decode_fp8(out, q, on(kc), on(vc), on(scale), on(scale), on(tables), on(np.asarray(LENS, np.int32)), 0.09,
                     q_len=q_len)
    want, wv, _ = ref.attend(q.cpu().double().numpy(), kc, vc, every, tables, LENS, 0.09)
    got = out.cpu().double().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= wv * 2.0 ** -9 + np.abs(want) * 2.0 ** -8 + 2.0 ** -20).all()
    assert pa.pa_device_error() == 0
