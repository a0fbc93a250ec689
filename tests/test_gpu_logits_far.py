"""Probabilities of logits and temperatures near fp32's ends against 64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import _pool_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_20_gb300 as pa
    pa.load()
    assert pa.pa_device_error() == 0
    return pa


TEMPS = (1e-44, 1e-30, 0.7, 1.0, 1.5, 1e36, 7e37, 3.3e38, math.inf)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("v", [11, 3001, 70000])
def test_differences_past_the_largest_number(pa, v, dtype):
    """Logits of both signs near the type's ends (a mask of its lowest value among them), where
    x - max overflows and x / temperature does not.  Tolerance: exp2's argument is a difference, a
    factor (one rounding) and a product, each half a step of itself: below 2^-22 of |z|
    together; exp2 and the sum of a row 2^-17 (up to 86 chained terms).  Within the latter also what
    a subnormal factor adds: 2^-22.6 of |z| < 3 at 3.3e38, and the least subnormal where 0 is
    meant (temperature inf) moves an argument by 6.8e38 * 1.4e-45 = 2^-20."""
    rng = np.random.default_rng(v)
    x = torch.from_numpy(rng.standard_normal((len(TEMPS), 1, v))).to(dtype)
    low = torch.finfo(dtype).min
    for i, at in enumerate((0.3, 0.9, 1.0)):
        x[:, 0, i::7] = low * at
        x[:, 0, i + 3::9] = -low * at * 0.95
    listed = np.array([[0, 1, 3, 4, v - 1]] * len(TEMPS), np.int32)  # (counted, and nothing taken off)
    for counted in (False, True):
        kw = dict(history=torch.from_numpy(listed).to(DEV), presence=torch.zeros(len(TEMPS), device=DEV),
                  history_lens=torch.full((len(TEMPS),), 5, dtype=torch.int32, device=DEV)) if counted else {}
        got = pa.pa_adjust_logits(None, x.to(DEV), temperature=torch.tensor(TEMPS, device=DEV), probs=True, **kw)
        got = got.cpu().double().numpy()
        for i, t in enumerate(TEMPS):
            want = ref.probabilities(x[i, 0].float().numpy(), np.float32(t))
            with np.errstate(divide="ignore"):
                z = np.abs(np.log2(np.maximum(want, 1e-40)))
            over = np.abs(got[i, 0] - want) - want * (2.0 ** -17 + z * 2.0 ** -22) - 2.0 ** -126
            assert over.max() <= 0, (t, int(over.argmax()), got[i, 0, over.argmax()], want[over.argmax()])
    assert pa.pa_device_error() == 0
