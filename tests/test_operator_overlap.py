"""Arguments that overlap: refused before a launch where a kernel would read what another
thread block has written (no GPU needed)."""
import pytest
import torch

from tests.test_abi import lib  # noqa: F401  (fixture)
from tests.test_operators_abi import INVALID, SCORED, _call

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
