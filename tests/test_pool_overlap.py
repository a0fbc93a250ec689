"""Arguments of the block-scaled append and of the pages' copy that overlap: refused before a
launch (no GPU needed)."""
import pytest
import torch

from tests.test_abi import lib  # noqa: F401  (fixture)
from tests.test_pool_abi import APPEND, COPY, INVALID, _call

AT = 0x1000000  # never used: the calls are refused, or (without a GPU) fail at their first step

accepted = pytest.mark.skipif(torch.cuda.is_available(), reason="an accepted call would use its pointers")

SEQS, TOKENS, HEADS, BLOCKS, WIDTH, PAIRS = 2, 3, 2, 8, 4, 5
CACHE, SCALES = BLOCKS * HEADS * 16 * 128, BLOCKS * HEADS * 8
ROWS = SEQS * TOKENS * HEADS * 128 * 2
TABLE, LENS = SEQS * WIDTH * 4, SEQS * 4


def placed(base, names, **sizes):
    """A call's arguments, its arrays apart from one another; with others=(array, bytes behind it)."""
    at = {**base, **sizes, **{k: AT + i * 0x100000 for i, k in enumerate(names)}}

    def call(**kw):
        a = dict(at)
        for k, (other, by) in kw.items():
            a[k] = at[other] + by
        return a
    return call


append = placed(APPEND, ("kc", "vc", "sc", "k", "v", "bt", "cl"), n=SEQS, u=TOKENS, hkv=HEADS, nb=BLOCKS, maxb=WIDTH)
copy = placed(COPY, ("kc", "vc", "sc", "sb", "db", "cnt"), most=PAIRS, hkv=HEADS, nb=BLOCKS)


@pytest.mark.parametrize("kw", [
    append(vc=("kc", 0)), append(vc=("kc", CACHE - 16)), append(kc=("vc", CACHE - 16)), append(sc=("kc", CACHE - 16)),
    append(sc=("vc", 16 - SCALES)), append(k=("kc", 0)), append(k=("vc", CACHE - 16)), append(v=("kc", 16 - ROWS)),
    append(v=("sc", 0)), append(k=("sc", 16 - ROWS)), append(bt=("kc", 0)), append(bt=("vc", 4 - TABLE)),
    append(bt=("sc", SCALES - 4)), append(cl=("vc", CACHE - 4)), append(cl=("sc", 4 - LENS)),
    {**append(k=("kc", 16 - 2 * (5 * 264 + 256))), "ks": 264},        # the last of strided rows
    {**append(), "ks": 1 << 39, "n": 1 << 20, "u": 1},                # rows past every address
])
def test_append(lib, kw):  # noqa: F811
    assert _call(lib, "pa_append_kv_block_scaled", APPEND, kw) == INVALID


@accepted
@pytest.mark.parametrize("kw", [
    append(), append(vc=("kc", CACHE)), append(kc=("vc", CACHE)), append(sc=("kc", CACHE)), append(sc=("vc", -SCALES)),
    append(k=("kc", CACHE)), append(v=("kc", -ROWS)), append(v=("sc", SCALES)), append(k=("sc", -ROWS)),
    append(bt=("vc", -TABLE)), append(cl=("sc", -LENS)), append(v=("k", 0)), append(v=("k", 512)),
    append(cl=("bt", 4)),
])
def test_append_beside(lib, kw):  # noqa: F811
    assert _call(lib, "pa_append_kv_block_scaled", APPEND, kw) != INVALID


@pytest.mark.parametrize("kw", [
    copy(vc=("kc", 0)), copy(vc=("kc", CACHE - 16)), copy(kc=("vc", CACHE - 16)), copy(sc=("kc", CACHE - 4)),
    copy(sc=("vc", 4 - SCALES)), copy(sb=("kc", 0)), copy(sb=("vc", CACHE - 4)), copy(db=("kc", 4 - 4 * PAIRS)),
    copy(db=("sc", 0)), copy(sb=("sc", SCALES - 4)), copy(cnt=("kc", 16)), copy(cnt=("vc", -4)), copy(cnt=("sc", -4)),
    {**copy(vc=("kc", CACHE)), "sc": None, "eb": 2},                  # pages of 16 bits
])
def test_copy(lib, kw):  # noqa: F811
    assert _call(lib, "pa_copy_pages", COPY, kw) == INVALID


@accepted
@pytest.mark.parametrize("kw", [
    copy(), copy(vc=("kc", CACHE)), copy(kc=("vc", CACHE)), copy(sc=("kc", CACHE)), copy(sc=("vc", -SCALES)),
    copy(sb=("kc", CACHE)), copy(db=("kc", -4 * PAIRS)), copy(sb=("sc", SCALES)), copy(cnt=("vc", -8)),
    copy(sb=("db", 0)), copy(cnt=("sb", 4)), {**copy(vc=("kc", 2 * CACHE)), "sc": None, "eb": 2},
    {**copy(sb=("kc", 0)), "sc": None, "most": 0},                    # (nothing listed: a no-op)
])
def test_copy_beside(lib, kw):  # noqa: F811
    assert _call(lib, "pa_copy_pages", COPY, kw) != INVALID
