"""Refusals of the block-scaled cache, the pool's bookkeeping and the logits' adjustment:
every one returns before a launch (no GPU needed)."""
import pytest

from tests.test_abi import FAKE, lib  # noqa: F401  (fixture)

INVALID, UNSUPPORTED = -1, -2
MB = 1 << 20


def _call(lib, name, args, kw):
    a = dict(args)
    for k in kw:
        assert k in a, k
    a.update(kw)
    return getattr(lib, name)(*a.values())


APPEND = dict(kc=FAKE, vc=FAKE, sc=FAKE, k=FAKE, v=FAKE, bt=FAKE, cl=FAKE, n=0, hkv=2, d=128, bs=16, maxb=4, nb=8,
              u=1, dtype=0, ks=256, vs=256, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"ks": 1024, "vs": 264}, 0), ({"kc": None}, INVALID), ({"sc": None}, INVALID), ({"v": None}, INVALID),
    ({"bt": None}, INVALID), ({"cl": None}, INVALID), ({"n": -1}, INVALID), ({"hkv": 0}, INVALID), ({"u": 0}, INVALID),
    ({"nb": 0}, INVALID), ({"maxb": 0}, INVALID), ({"k": FAKE + 8}, INVALID), ({"sc": FAKE + 4}, INVALID),
    ({"bt": FAKE + 2}, INVALID), ({"ks": 248}, INVALID), ({"ks": 260}, INVALID), ({"vs": 1 << 40}, INVALID),
    ({"n": 1 << 20, "u": 4096}, INVALID), ({"nb": 1 << 30}, INVALID),
    ({"d": 64, "ks": 128, "vs": 128}, UNSUPPORTED), ({"bs": 24}, UNSUPPORTED), ({"u": 4097}, UNSUPPORTED),
    ({"dtype": 2}, UNSUPPORTED),
])
def test_append(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_append_kv_block_scaled", APPEND, kw) == status


ATTEND = dict(out=FAKE, q=FAKE, kc=FAKE, vc=FAKE, sc=FAKE, bt=FAKE, cl=FAKE, n=2, hq=8, hkv=2, d=128, bs=16, scale=0.1,
              maxb=4, nb=8, u=1, dtype=0, splits=1, ws=None, wsb=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"out": None}, INVALID), ({"sc": None}, INVALID), ({"sc": FAKE + 8}, INVALID), ({"q": None}, INVALID),
    ({"kc": FAKE + 4}, INVALID), ({"splits": 0}, INVALID), ({"splits": 1 << 20}, INVALID), ({"splits": 2}, INVALID),
    ({"splits": 2, "ws": FAKE + 16, "wsb": MB}, INVALID), ({"splits": 2, "ws": FAKE, "wsb": 100}, INVALID),
    ({"hq": 9}, INVALID), ({"u": 0}, INVALID), ({"n": 0}, INVALID), ({"scale": float("nan")}, INVALID),
    ({"d": 64}, UNSUPPORTED), ({"bs": 64}, UNSUPPORTED), ({"u": 4097}, UNSUPPORTED), ({"dtype": 2}, UNSUPPORTED),
])
def test_attend(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_decode_block_scaled", ATTEND, kw) == status


FREE = dict(bt=FAKE, rc=FAKE + MB, kl=FAKE + 2 * MB, n=2, maxb=4, nb=8, bs=16, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"bt": None}, INVALID), ({"rc": None}, INVALID), ({"kl": None}, INVALID), ({"n": 0}, INVALID),
    ({"maxb": 0}, INVALID), ({"nb": 0}, INVALID), ({"bs": 0}, INVALID), ({"bt": FAKE + 4}, INVALID),
    ({"rc": FAKE + MB + 8}, INVALID), ({"kl": FAKE + 2 * MB + 1}, INVALID), ({"rc": FAKE + 16}, INVALID),
    ({"kl": FAKE + 28}, INVALID), ({"kl": FAKE + MB + 4}, INVALID), ({"n": 1 << 20, "maxb": 1 << 10}, INVALID),
    ({"nb": 1 << 30}, INVALID), ({"bs": 4}, UNSUPPORTED),
])
def test_free(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_free_blocks", FREE, kw) == status


RESERVE = dict(bt=FAKE, rc=FAKE + MB, ln=FAKE + 2 * MB, ms=FAKE + 3 * MB, n=2, maxb=4, nb=8, bs=16, ws=FAKE + 4 * MB,
               wsb=1 << 16, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"ms": None}, INVALID), ({"ws": None}, INVALID), ({"wsb": 8}, INVALID), ({"ws": FAKE + 4 * MB + 4}, INVALID),
    ({"ms": FAKE + MB}, INVALID), ({"ms": FAKE + 2 * MB + 4}, INVALID), ({"ws": FAKE}, INVALID),
    ({"ln": FAKE + 4 * MB}, INVALID), ({"n": 0}, INVALID), ({"bs": 12}, UNSUPPORTED),
])
def test_reserve(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_reserve_blocks", RESERVE, kw) == status


FORK = dict(bt=FAKE, cl=FAKE + MB, rc=FAKE + 2 * MB, ss=FAKE + 3 * MB, ds=FAKE + 4 * MB, sb=FAKE + 5 * MB,
            db=FAKE + 6 * MB, cnt=FAKE + 7 * MB, f=2, n=4, maxb=4, nb=8, bs=16, ws=FAKE + 8 * MB, wsb=1 << 16, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"f": 5}, INVALID), ({"f": -1}, INVALID), ({"ss": None}, INVALID), ({"db": None}, INVALID), ({"cnt": None}, INVALID),
    ({"sb": FAKE + 6 * MB}, INVALID), ({"ss": FAKE + 5 * MB}, INVALID), ({"cl": FAKE + 4}, INVALID),
    ({"ds": FAKE + MB}, INVALID), ({"cnt": FAKE + 2 * MB}, INVALID), ({"wsb": 16}, INVALID), ({"bs": 7}, UNSUPPORTED),
])
def test_fork(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_fork_blocks", FORK, kw) == status


COMPACT = dict(to=FAKE, ro=FAKE + MB, bt=FAKE, rc=FAKE + MB, sb=FAKE + 2 * MB, db=FAKE + 3 * MB, cnt=FAKE + 4 * MB, n=2,
               maxb=4, nb=8, ws=FAKE + 5 * MB, wsb=1 << 16, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"to": None}, INVALID), ({"sb": None}, INVALID), ({"to": FAKE + 16}, INVALID), ({"ro": FAKE + MB + 16}, INVALID),
    ({"ro": FAKE}, INVALID), ({"db": FAKE + 2 * MB + 12}, INVALID), ({"cnt": FAKE + 5 * MB}, INVALID),
    ({"wsb": 20}, INVALID), ({"n": 0}, INVALID), ({"nb": 0}, INVALID), ({"bt": FAKE + 8}, INVALID),
])
def test_compact(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_compact_blocks", COMPACT, kw) == status


def test_pages_workspace(lib):  # noqa: F811
    size = lib.pa_pages_workspace_size
    assert size(0, 0) == 0 and size(8, -1) == 0
    assert size(100, 0) >= 4 * (100 + 50) and size(100, 300) >= 4 * (100 + 300)


COPY = dict(kc=FAKE, vc=FAKE, sc=None, sb=FAKE, db=FAKE, cnt=FAKE, most=0, hkv=2, d=128, bs=16, nb=8, eb=1, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"sc": FAKE}, 0), ({"eb": 2, "d": 64}, 0), ({"kc": None}, INVALID), ({"cnt": None}, INVALID),
    ({"most": -1}, INVALID), ({"kc": FAKE + 8}, INVALID), ({"sb": FAKE + 2}, INVALID), ({"eb": 2, "sc": FAKE}, INVALID),
    ({"hkv": 0}, INVALID), ({"nb": 1 << 30}, INVALID), ({"eb": 4}, UNSUPPORTED), ({"d": 64}, UNSUPPORTED),
    ({"bs": 64}, UNSUPPORTED), ({"d": 96, "eb": 2}, UNSUPPORTED),
])
def test_copy(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_copy_pages", COPY, kw) == status


LOGITS = dict(out=FAKE, x=FAKE + 64 * MB, h=None, hl=None, pl=None, dr=None, rep=None, pres=None, freq=None, bi=None,
              bv=None, mask=None, temp=None, n=0, r=2, v=1000, hist=0, nbias=0, dtype=1, probs=1, os=1000, xs=1000, ms=0,
              mr=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"dtype": 2}, 0), ({"out": None}, INVALID), ({"x": None}, INVALID), ({"h": FAKE}, INVALID),
    ({"hl": FAKE}, INVALID), ({"pl": FAKE}, INVALID), ({"bi": FAKE}, INVALID), ({"nbias": 1}, INVALID), ({"n": -1}, INVALID),
    ({"r": 0}, INVALID), ({"v": 0}, INVALID), ({"hist": -1}, INVALID), ({"os": 999}, INVALID), ({"xs": 999}, INVALID),
    ({"out": FAKE + 2}, INVALID), ({"x": FAKE + 1}, INVALID), ({"temp": FAKE + 2}, INVALID),
    ({"mask": FAKE, "ms": -1}, INVALID), ({"dtype": 3}, UNSUPPORTED), ({"v": 262145, "os": 262145, "xs": 262145}, UNSUPPORTED),
    ({"nbias": 1025, "bi": FAKE, "bv": FAKE}, UNSUPPORTED),
    # overlaps: out over logits of another type, stride or place, over an input
    ({"n": 1, "x": FAKE}, INVALID), ({"n": 1, "x": FAKE, "dtype": 2, "xs": 1004}, INVALID),
    ({"n": 1, "x": FAKE + 4, "dtype": 2}, INVALID), ({"n": 1, "temp": FAKE + 4000}, INVALID),
    ({"n": 1, "h": FAKE + 7996, "hl": FAKE + 32 * MB, "hist": 5}, INVALID), ({"n": 1, "mask": FAKE + 16}, INVALID),
])
def test_logits(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_adjust_logits", LOGITS, kw) == status
