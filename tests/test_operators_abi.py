"""Refusals of the rotary append, scored attention, eviction and draft verification:
every one returns before a launch (no GPU needed)."""
import pytest

from tests.test_abi import FAKE, lib  # noqa: F401  (fixture)

INVALID, UNSUPPORTED = -1, -2


def _call(lib, name, args, kw):
    a = dict(args)
    for k in kw:
        assert k in a, k
    a.update(kw)
    return getattr(lib, name)(*a.values())


ROPE = dict(q_out=FAKE, q=FAKE, k=FAKE, v=FAKE, kc=FAKE, vc=FAKE, pos=FAKE, slots=FAKE, turns=FAKE,
            axis=FAKE, n=0, hq=8, hkv=2, d=128, rot=128, axes=1, inter=0, so=1024, sq=1024, sk=256,
            sv=256, bs=16, nb=8, dtype=0, ks=None, vs=None, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({}, 0), ({"ks": FAKE, "vs": FAKE}, 0), ({"so": 1536, "sq": 1536, "sk": 1536, "sv": 1536}, 0),
    ({"q_out": None}, INVALID), ({"v": None}, INVALID), ({"pos": None}, INVALID),
    ({"slots": None}, INVALID), ({"turns": None}, INVALID), ({"axis": None}, INVALID),
    ({"ks": FAKE}, INVALID), ({"n": -1}, INVALID), ({"hq": 0}, INVALID), ({"hkv": 0}, INVALID),
    ({"axes": 0}, INVALID), ({"nb": 0}, INVALID), ({"q": FAKE + 2}, INVALID),
    ({"k": FAKE + 8}, INVALID), ({"vc": FAKE + 4}, INVALID), ({"so": 1016}, INVALID),
    ({"sk": 255}, INVALID), ({"sk": 260}, INVALID), ({"sv": -256}, INVALID),
    ({"rot": 144}, INVALID), ({"rot": 0}, INVALID), ({"rot": 24}, UNSUPPORTED), ({"axes": 33}, UNSUPPORTED),
    ({"d": 96, "rot": 96}, UNSUPPORTED), ({"bs": 24}, UNSUPPORTED), ({"dtype": 7}, UNSUPPORTED),
    ({"d": 64, "rot": 64, "ks": FAKE, "vs": FAKE}, UNSUPPORTED),
    ({"so": 1032}, INVALID),  # over its own input with another stride
    ({"so": 1032, "q_out": FAKE + 64}, 0),
])
def test_rope_append(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_rope_append", ROPE, kw) == status


SCORED = dict(out=FAKE, scores=FAKE, pos=FAKE, q=FAKE, k=FAKE, v=FAKE, ks=None, vs=None, bt=FAKE,
              cl=FAKE, sl=FAKE, n=2, hq=8, hkv=2, d=128, bs=16, scale=0.1, maxb=4, nb=8, u=1, dtype=0,
              splits=1, ws=FAKE, wsb=0, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({}, INVALID),  # no room in the workspace
    ({"ws": None}, INVALID), ({"ws": FAKE + 16}, INVALID), ({"out": None}, INVALID),
    ({"scores": None}, INVALID), ({"scores": FAKE + 4}, INVALID), ({"pos": None}, INVALID),
    ({"sl": None}, INVALID), ({"pos": FAKE + 8}, INVALID), ({"ks": FAKE}, INVALID),
    ({"splits": 0}, INVALID), ({"splits": 1 << 20}, INVALID), ({"hq": 9}, INVALID), ({"u": 0}, INVALID),
    ({"scale": float("inf")}, INVALID), ({"u": 4097}, UNSUPPORTED), ({"d": 80}, UNSUPPORTED),
    ({"bs": 64}, UNSUPPORTED), ({"dtype": 2}, UNSUPPORTED),
    ({"d": 64, "ks": FAKE, "vs": FAKE}, UNSUPPORTED),
])
def test_decode_scored(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_decode_scored", SCORED, kw) == status
    need = lib.pa_decode_scored_workspace_size(2, 8, 1, 128, 1, 4, 16)
    assert _call(lib, "pa_decode_scored", SCORED, {"wsb": need - 1}) == INVALID


def test_decode_scored_workspace(lib):  # noqa: F811
    size = lib.pa_decode_scored_workspace_size
    al = lambda x: (x + 255) // 256 * 256  # noqa: E731
    rows = 3 * 2 * 8
    assert size(3, 8, 2, 128, 1, 5, 8) == 2 * al(rows * 4) + al(rows * 48 * 4)  # 40 rows: 3 tiles
    assert size(3, 8, 2, 128, 4, 5, 8) == lib.pa_decode_workspace_size(3, 8, 2, 128, 4) + al(rows * 48 * 4)
    assert size(3, 8, 17, 128, 4, 5, 8) == al(3 * 17 * 8 * 4)  # many rows: a statistic each
    for bad in ((0, 8, 2, 128, 1, 5, 8), (3, 8, 2, 128, 0, 5, 8), (3, 8, 2, 128, 1, 0, 8)):
        assert size(*bad) == 0


EVICT = dict(k=FAKE, v=FAKE, so=FAKE, po=FAKE + 64, nl=FAKE, sc=FAKE, rp=FAKE + 64, bt=FAKE,
             cl=FAKE + 16, sl=FAKE + 48, n=2, hkv=2, d=128, bs=16, maxb=4, nb=8, budget=32, sinks=2,
             recent=8, eb=2, ws=FAKE, wsb=2 * 2 * 32 * 8, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"wsb": 2 * 2 * 32 * 8 - 1}, INVALID), ({"ws": None}, INVALID), ({"ws": FAKE + 8}, INVALID),
    ({"k": None}, INVALID), ({"so": None}, INVALID), ({"nl": None}, INVALID), ({"rp": None}, INVALID),
    ({"sl": None}, INVALID), ({"k": FAKE + 8}, INVALID), ({"nl": FAKE + 16}, INVALID),
    ({"nl": FAKE + 32, "sl": FAKE + 32}, INVALID),
    ({"sc": FAKE + 4, "so": FAKE + 4}, INVALID), ({"rp": FAKE + 8, "po": FAKE + 8}, INVALID),
    ({"so": FAKE + 256}, INVALID),  # one ledger in place, the other not
    ({"budget": 0}, INVALID), ({"sinks": -1}, INVALID), ({"recent": -1}, INVALID),
    ({"sinks": 30, "recent": 3}, INVALID), ({"n": 0}, INVALID), ({"nb": 0}, INVALID),
    ({"maxb": 1 << 27}, INVALID), ({"eb": 4}, UNSUPPORTED), ({"d": 96}, UNSUPPORTED),
    ({"d": 64, "eb": 1}, UNSUPPORTED), ({"bs": 12}, UNSUPPORTED),
])
def test_evict(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_evict", EVICT, kw) == status
    assert lib.pa_evict_workspace_size(2, 2, 32) == 2 * 2 * 32 * 8
    assert lib.pa_evict_workspace_size(2, 0, 32) == 0


VERIFY = dict(out=FAKE, acc=FAKE, nl=FAKE, cl=FAKE, p=FAKE, q=FAKE, x=FAKE, dl=None, au=FAKE, su=FAKE,
              n=2, k=3, v=100, ps=100, qs=100, stream=None)


@pytest.mark.parametrize("kw,status", [
    ({"out": None}, INVALID), ({"acc": None}, INVALID), ({"p": None}, INVALID), ({"x": None}, INVALID),
    ({"au": None}, INVALID), ({"su": None}, INVALID), ({"cl": None}, INVALID), ({"n": 0}, INVALID),
    ({"k": 0}, INVALID), ({"v": 0}, INVALID), ({"ps": 99}, INVALID), ({"qs": 99}, INVALID),
    ({"p": FAKE + 2}, INVALID), ({"k": 4096}, UNSUPPORTED), ({"v": 1 << 31 - 1, "n": 1 << 30}, INVALID),
])
def test_verify_drafts(lib, kw, status):  # noqa: F811
    assert _call(lib, "pa_verify_drafts", VERIFY, kw) == status


def test_rope_table_on_the_host():
    import math

    import paged_kv_cache_20_gb300 as pa
    turns, axis = pa.rope_table(64, 32, base=500.0, sections=(4, 5, 7), device="cpu")
    assert axis.tolist() == [0] * 4 + [1] * 5 + [2] * 7
    for i, t in enumerate(turns.tolist()):
        f = 500.0 ** (-2 * i / 32)
        assert abs((t % (1 << 64)) / 2.0 ** 64 - f / (2 * math.pi)) < 2.0 ** -53
    # more than a turn a position wraps
    turns, _ = pa.rope_table(64, 32, inv_freq=[2 * math.pi * 1.25] * 16, device="cpu")
    assert turns.tolist() == [1 << 62] * 16
    with pytest.raises(ValueError):
        pa.rope_table(64, sections=(3, 4), device="cpu")
