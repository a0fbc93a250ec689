"""Arguments that overlap: refused before a launch where a kernel would read what another
thread block has written (no GPU needed)."""
import pytest
import torch

from tests.test_abi import FAKE, lib  # noqa: F401  (fixture)
from tests.test_operators_abi import EVICT, INVALID, SCORED, _call

AT = 0x1000000  # never used: the calls are refused, or (without a GPU) fail at their first step

accepted = pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would use its pointers")

MANY = {"u": 17, "wsb": 1 << 30, "q": AT}
Q_BYTES = 2 * 17 * 8 * 128 * 2   # of that call


@pytest.mark.parametrize("out", [AT, AT + 16, AT + Q_BYTES - 16, AT - Q_BYTES + 16])
def test_scored_output_over_many_query_rows(lib, out):  # noqa: F811
    assert _call(lib, "pa_decode_scored", SCORED, {**MANY, "out": out}) == INVALID


@accepted
@pytest.mark.parametrize("kw", [{**MANY, "out": AT + Q_BYTES}, {**MANY, "out": AT - Q_BYTES},
                                {**MANY, "u": 16, "out": AT}])
def test_scored_output_beside_its_queries(lib, kw):  # noqa: F811
    assert _call(lib, "pa_decode_scored", SCORED, kw) != INVALID


ROOM = 2 * 2 * 32 * 8
LENS, LEDGER = 2 * 4, 2 * 2 * 4 * 16 * 4
EVICT_AT = {**{k: AT + i * 0x10000 for i, k in enumerate(EVICT) if EVICT[k] and EVICT[k] >= FAKE},
            "wsb": ROOM}


def beside(**kw):
    """The eviction call with arguments moved to so many bytes behind others."""
    a = dict(EVICT_AT)
    for k, (other, by) in kw.items():
        a[k] = EVICT_AT[other] + by
    return a


@pytest.mark.parametrize("kw", [
    beside(nl=("cl", 0)), beside(nl=("cl", 4)), beside(nl=("cl", 4 - LENS)), beside(nl=("sl", 4)),
    beside(nl=("sl", 4 - LENS)), beside(so=("sc", 64)), beside(so=("sc", 16 - LEDGER)),
    beside(po=("rp", LEDGER - 16)), beside(so=("rp", 0)), beside(po=("sc", 0)),
])
def test_evict(lib, kw):  # noqa: F811
    assert _call(lib, "pa_evict", EVICT, kw) == INVALID


@accepted
@pytest.mark.parametrize("kw", [beside(), beside(nl=("cl", LENS)), beside(nl=("sl", -LENS)),
                                beside(so=("sc", LEDGER), po=("rp", -LEDGER)),
                                beside(so=("sc", 0), po=("rp", 0))])
def test_evict_beside(lib, kw):  # noqa: F811
    assert _call(lib, "pa_evict", EVICT, kw) != INVALID
