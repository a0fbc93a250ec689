"""Arguments that overlap: refused before a launch where a kernel would read what another
thread block has written (no GPU needed)."""
import pytest
import torch

from tests.test_abi import FAKE, lib  # noqa: F401  (fixture)
from tests.test_operators_abi import EVICT, INVALID, SCORED, VERIFY, _call

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


SEQS, DRAFTS = 2, 3   # of VERIFY
VERIFY_AT = {**{k: AT + i * 0x10000 for i, k in enumerate(VERIFY) if VERIFY[k] == FAKE}, "dl": AT - 0x10000}


def verify(**kw):
    a = dict(VERIFY_AT)
    for k, (other, by) in kw.items():
        a[k] = VERIFY_AT[other] + by
    return a


@pytest.mark.parametrize("kw", [
    verify(nl=("cl", 4)), verify(nl=("cl", -4)), verify(nl=("dl", 4)), verify(acc=("dl", -4)), verify(acc=("cl", 0)),
    verify(out=("x", 0)), verify(out=("x", 4 * SEQS * DRAFTS - 4)), verify(out=("x", 4 - 4 * SEQS * (DRAFTS + 1))),
    verify(out=("dl", 0)), verify(out=("cl", 0)), verify(acc=("x", 8)), verify(nl=("x", 0)),
    verify(acc=("out", 16)), verify(nl=("out", 0)), verify(nl=("acc", 0)),
    {**verify(out=("x", 4)), "n": 1},
])
def test_verify_drafts(lib, kw):  # noqa: F811
    assert _call(lib, "pa_verify_drafts", VERIFY, kw) == INVALID


@accepted
@pytest.mark.parametrize("kw", [
    verify(), verify(nl=("cl", 0)), verify(nl=("dl", 0)), verify(acc=("dl", 0)), verify(out=("x", 4 * SEQS * DRAFTS)),
    {**verify(out=("x", 0)), "n": 1}, {**verify(acc=("cl", 0)), "nl": None}, {**verify(), "nl": None, "cl": None, "dl": None},
])
def test_verify_drafts_beside(lib, kw):  # noqa: F811
    assert _call(lib, "pa_verify_drafts", VERIFY, kw) != INVALID
