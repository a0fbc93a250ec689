"""pa_evict where a table names blocks outside the pool: whole moves are left out, so that
a row and what the ledgers say of it stay together (needs a GPU)."""
import numpy as np
import pytest
import torch

from tests import _ops_ref as ref
from tests.test_gpu_evict import make, pa, run  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


def expected(c, budget, sinks, recent):
    """The moves of the definition, by following each kept row's place through a pool and
    ledgers of row numbers; then those whose two blocks exist, done on the real ones."""
    n, hkv, rows = c["scores"].shape
    bs, blocks = c["bs"], c["k"].shape[0]
    numbers = np.broadcast_to(np.arange(rows), (n, hkv, rows)).copy()
    k, v, s, p = (c[x].numpy().copy() for x in ("k", "v", "scores", "pos"))
    # (a table and a pool of its own for the choice: block ids play no part in it)
    width = c["table"].shape[1]
    own = np.arange(n * width).reshape(n, width)
    dummy = np.zeros((n * width, hkv, bs, 1))
    for i in range(n):
        for t in range(rows):
            dummy[own[i, t // bs], :, t % bs, 0] = t
    moved = ref.evict(dummy, dummy, c["scores"].numpy(), c["pos"].numpy(), own, np.array(c["lens"]),
                      np.array(c["sl"]), budget, sinks, recent)
    done = skipped = 0
    table = c["table"].numpy()
    for i in range(n):
        for h in range(hkv):
            for to in range(min(budget, c["lens"][i])):
                frm = int(moved[0][own[i, to // bs], h, to % bs, 0])
                assert numbers[i, h, to] == to
                if frm == to:
                    continue
                bt, bf = int(table[i, to // bs]), int(table[i, frm // bs])
                if not (0 <= bt < blocks and 0 <= bf < blocks):
                    skipped += 1
                    continue
                done += 1
                k[bt, h, to % bs] = c["k"].numpy()[bf, h, frm % bs]
                v[bt, h, to % bs] = c["v"].numpy()[bf, h, frm % bs]
                s[i, h, to], p[i, h, to] = c["scores"].numpy()[i, h, frm], c["pos"].numpy()[i, h, frm]
    return k, v, s, p, np.minimum(c["lens"], budget), done, skipped


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("lens,budget,bs", [
    ([100, 64], 30, 16),      # the radix select
    ([37, 34], 30, 8),        # a few rows over
    ([6000], 3000, 32),       # a cluster of thread blocks
    ([5002], 4995, 8),        # the same, a few rows over
])
def test_whole_moves_are_left_out(pa, lens, budget, bs, apart):  # noqa: F811
    c = make(40 + budget, lens, 2, 64, bs)
    c["scores"][..., :budget] *= 0.01  # (rows from behind the budget win)
    n, width = c["table"].shape
    c["table"][0, 0] = 10 ** 6                             # holes
    c["table"][0, (lens[0] - 1) // bs] = -1                # sources
    if n > 1:
        c["table"][1, 1] = c["k"].shape[0]
    want = expected(c, budget, 1, 2)
    assert want[5] > 0 and want[6] > 0
    k, v, so, po, new = run(pa, c, budget, 1, 2, apart)[:5]
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert np.array_equal(new.cpu().numpy(), want[4])
    assert np.array_equal(k.cpu().view(torch.int16).numpy(), want[0])
    assert np.array_equal(v.cpu().view(torch.int16).numpy(), want[1])
    for i, L in enumerate(want[4]):
        assert np.array_equal(so[i, :, :L].cpu().view(torch.int32).numpy(), want[2].view(np.int32)[i, :, :L])
        assert np.array_equal(po[i, :, :L].cpu().numpy(), want[3][i, :, :L])
