"""pa_rope_append against a 64-bit rotation (needs a GPU)."""
import numpy as np
import pytest
import torch

from tests import _ops_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_20_gb300 as pa
    pa.load()
    assert pa.pa_device_error() == 0
    return pa


def make(seed, tokens, hq, hkv, d, bs, dtype, axes, rot, inter, fp8, packed, far=1 << 20):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    dt = DTYPES[dtype]
    c = dict(inter=inter, bs=bs)
    if packed:
        qkv = rnd(tokens, hq + 2 * hkv, d).to(dt).to(DEV)
        c["q"], c["k"], c["v"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
    else:
        c["q"], c["k"], c["v"] = (rnd(tokens, h, d).to(dt).to(DEV) for h in (hq, hkv, hkv))
    blocks = tokens // bs + 4
    slots = torch.randperm(blocks * bs, generator=g)[:tokens]
    if tokens > 2:
        slots[1] = -1
    c["slots"] = slots.to(DEV)
    shape = (blocks, hkv, bs, d)
    if fp8:
        c["k_cache"], c["v_cache"] = (torch.randint(0, 120, shape, generator=g, dtype=torch.uint8).to(DEV)
                                      for _ in range(2))
        c["k_scale"], c["v_scale"] = (torch.rand(hkv, generator=g).mul(0.03).add(0.001).to(DEV)
                                      for _ in range(2))
    else:
        c["k_cache"], c["v_cache"] = (torch.full(shape, float("nan"), dtype=dt, device=DEV)
                                      for _ in range(2))
        c["k_scale"] = c["v_scale"] = None
    c["pos"] = torch.randint(-5, far, (axes, tokens), generator=g, dtype=torch.int32).to(DEV)
    half = rot // 2
    cut = sorted(torch.randint(0, half + 1, (axes - 1,), generator=g).tolist())
    c["sections"] = [b - a for a, b in zip([0] + cut, cut + [half])]
    c["inv_freq"] = [10000.0 ** (-i / half) for i in range(half)]
    c["rot"] = rot
    return c


def run(pa, c, q_out=None, stream=None):
    turns, axis = pa.rope_table(c["q"].shape[2], c["rot"], sections=c["sections"], device=DEV)
    out = torch.empty(c["q"].shape, dtype=c["q"].dtype, device=DEV) if q_out is None else q_out
    pa.pa_rope_append(out, c["q"], c["k"], c["v"], c["k_cache"], c["v_cache"], c["pos"], c["slots"],
                      turns, axis, interleaved=c["inter"], k_scale=c["k_scale"],
                      v_scale=c["v_scale"], stream=stream)
    return out


def close16(got, want, slack, dtype):
    """One rounding to the 16-bit type (half a step, relative eps/2; fp16's subnormal
    step is 2^-24) on a value that is off by `slack`."""
    eps = torch.finfo(dtype).eps / 2
    tiny = 2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134
    bad = np.abs(got - want) > eps * (np.abs(want) + slack) + slack + tiny
    assert not bad.any(), (int(bad.sum()), np.abs(got - want)[bad][:4], want[bad][:4])


def check(c, out, before):
    axis = np.repeat(np.arange(len(c["sections"])), c["sections"])
    pos = c["pos"].cpu().numpy()
    half = c["rot"] // 2
    q, k, v = (ref.f64(c[x]) for x in ("q", "k", "v"))
    rq = ref.rope(q, pos, c["inv_freq"], axis, c["inter"])
    rk = ref.rope(k, pos, c["inv_freq"], axis, c["inter"])
    close16(ref.f64(out), rq, ref.rope_slack(q, half, c["inter"]), out.dtype)
    slots = c["slots"].cpu().numpy()
    live = slots >= 0
    blk, off = slots[live] // c["bs"], slots[live] % c["bs"]
    sk = ref.rope_slack(k, half, c["inter"])[live]
    untouched = np.ones(tuple(c["k_cache"].shape[:3]), bool)
    untouched[blk, :, off] = False
    for name, want, slack in (("k_cache", rk[live], sk), ("v_cache", v[live], 0 * sk)):
        raw = c[name].cpu().view(torch.uint8).numpy().reshape(*untouched.shape, -1)
        old = before[name].cpu().view(torch.uint8).numpy().reshape(*untouched.shape, -1)
        assert np.array_equal(raw[untouched], old[untouched]), name
        if c["k_scale"] is None:
            close16(ref.f64(c[name])[blk, :, off], want, slack, c[name].dtype)
        else:
            # half a step of e4m3 (2^-4 of the value; 2^-10 among the subnormals), on a
            # quotient off by the slack and its own rounding
            sc = ref.f64(c[name[0] + "_scale"])[:, None]
            x = want / sc
            e = slack / sc + 2.0 ** -23 * np.abs(x)
            x = np.clip(x, -448, 448)
            got = ref.e4m3_values(c[name].cpu())[blk, :, off]
            bad = np.abs(got - x) > np.maximum(2.0 ** -4 * (np.abs(x) + e), 2.0 ** -10) + e
            assert not bad.any(), (name, got[bad][:4], x[bad][:4])


SHAPES = [
    # tokens, hq, hkv, d, bs, dtype, axes, rot, inter, fp8, packed
    (1, 1, 1, 64, 8, "fp16", 1, 64, False, False, False),
    (1, 32, 8, 128, 16, "bf16", 3, 128, False, False, True),
    (5, 4, 4, 64, 16, "bf16", 2, 32, True, False, True),
    (7, 3, 1, 128, 32, "fp16", 1, 96, False, False, False),
    (33, 8, 2, 128, 16, "fp16", 3, 16, True, False, False),
    (130, 40, 40, 128, 8, "bf16", 2, 128, True, False, True),
    (9, 32, 8, 128, 16, "bf16", 3, 128, False, True, True),
    (65, 5, 5, 128, 32, "fp16", 1, 64, True, True, False),
    (1030, 16, 2, 64, 16, "fp16", 2, 48, False, False, False),
    (3, 300, 20, 128, 16, "bf16", 1, 128, False, False, False),   # more items than a pass
    (77, 1, 1, 128, 8, "bf16", 2, 112, True, True, False),
    (9, 2, 50, 64, 16, "fp16", 1, 64, False, False, True),        # more KV heads than a launch
    (3000, 2, 1, 128, 32, "fp16", 3, 128, False, True, True),     # many tokens a CTA
]


@pytest.mark.parametrize("shape", SHAPES)
def test_rotation_and_slots(pa, shape):
    c = make(1, *shape)
    before = {n: c[n].clone() for n in ("k_cache", "v_cache")}
    out = run(pa, c)
    torch.cuda.synchronize()
    assert pa.pa_device_error() == 0
    check(c, out, before)


def test_far_positions_keep_their_fraction_of_a_turn(pa):
    c = make(2, 300, 4, 2, 128, 16, "fp16", 2, 128, False, False, False, far=(1 << 31) - 1)
    # positions near 2^31: float64 angles are off by 2^31 * 2^-53 = 2.4e-7, which the
    # reference adds to the bound
    before = {n: c[n].clone() for n in ("k_cache", "v_cache")}
    out = run(pa, c)
    axis = np.repeat(np.arange(2), c["sections"])
    q = ref.f64(c["q"])
    want = ref.rope(q, c["pos"].cpu().numpy(), c["inv_freq"], axis, False)
    slack = ref.rope_slack(q, 64, False) * (1 + 2.4e-7 * 2 / 5.5e-7)
    close16(ref.f64(out), want, slack, out.dtype)
    assert before["k_cache"].shape == c["k_cache"].shape


def test_in_place_on_a_fused_projection(pa):
    c = make(3, 50, 8, 2, 128, 16, "bf16", 3, 128, False, False, True)
    keep = c["q"].clone()
    want = run(pa, {**c, "k_cache": c["k_cache"].clone(), "v_cache": c["v_cache"].clone()})
    kv = torch.cat((c["k"], c["v"]), 1).clone()
    got = run(pa, c, q_out=c["q"])  # strided, over its own input
    assert torch.equal(got, want) and not torch.equal(got, keep)
    assert torch.equal(torch.cat((c["k"], c["v"]), 1), kv)  # the slices beside it


def test_zero_position_is_the_identity(pa):
    c = make(4, 20, 4, 4, 64, 16, "fp16", 1, 64, True, False, False)
    c["pos"].zero_()
    assert torch.equal(run(pa, c), c["q"])


@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_codes_are_those_of_the_plain_append(pa, dtype):
    """V rows of every 16-bit pattern under scales from tiny to huge: the codes of
    pa_append_kv_fp8, which divides."""
    bits = torch.arange(1 << 16, dtype=torch.int32).to(torch.int16).view(DTYPES[dtype])
    scales = [1.0, 0.037, 3.3e-3, 448.0, 2.0 ** -60, 2.0 ** -61, 1e-30, 7e-39, 1.7e18, 1.3e19, 3e38, 0.0,
              -0.25, float("inf"), float("nan"), 1.1754944e-38]
    hkv, tokens = len(scales), (1 << 16) // 128
    v = bits.view(tokens, 1, 128).expand(tokens, hkv, 128).contiguous().to(DEV)
    k = torch.zeros_like(v)
    sc = torch.tensor(scales, device=DEV)
    slots = torch.arange(tokens, device=DEV)
    shape = (tokens // 16, hkv, 16, 128)
    a = [torch.full(shape, 0x55, dtype=torch.uint8, device=DEV) for _ in range(4)]
    pa.pa_append_kv_fp8(a[0], a[1], k, v, slots, sc, sc)
    turns, axis = pa.rope_table(128, device=DEV)
    q = torch.zeros(tokens, 1, 128, dtype=v.dtype, device=DEV)
    pos = torch.zeros(1, tokens, dtype=torch.int32, device=DEV)
    pa.pa_rope_append(q, q, k, v, a[2], a[3], pos, slots, turns, axis, k_scale=sc, v_scale=sc)
    torch.cuda.synchronize()
    same = a[1] == a[3]
    # (0 / 0 and the like: a NaN code of either sign is a NaN)
    nan = (a[1] & 0x7F == 0x7F) & (a[3] & 0x7F == 0x7F)
    assert (same | nan).all(), [(scales[int(h)], int((~(same | nan))[:, h].sum())) for h in range(hkv)]
    assert torch.equal(a[0][:, :4], a[2][:, :4])


def test_bad_slots_and_axes_are_reported(pa):
    c = make(5, 6, 2, 2, 64, 8, "fp16", 1, 64, False, False, False)
    before = c["k_cache"].clone()
    c["slots"][:] = torch.tensor([0, 10 ** 9, -1, -7, 1 << 40, 3])
    out = run(pa, c)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    want = ref.rope(ref.f64(c["q"]), c["pos"].cpu().numpy(), c["inv_freq"], np.zeros(32, int), False)
    close16(ref.f64(out), want, ref.rope_slack(ref.f64(c["q"]), 32, False), out.dtype)
    a, b = ref.f64(c["k_cache"]), ref.f64(before)
    rows = np.ones(a.shape[:3], bool)
    rows[0, :, 0] = rows[0, :, 3] = False
    assert np.isnan(a[rows]).all() and not np.isnan(a[0, :, 0]).any() and np.isnan(b).all()
    turns, axis = pa.rope_table(64, device=DEV)
    axis[3] = 4
    pa.pa_rope_append(out, c["q"], c["k"], c["v"], c["k_cache"], c["v_cache"], c["pos"], c["slots"],
                      turns, axis)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert pa.pa_device_error() == 0


def test_side_stream_and_graph(pa):
    c = make(6, 40, 8, 2, 128, 16, "bf16", 3, 128, False, False, False)
    want = run(pa, {**c, "k_cache": c["k_cache"].clone(), "v_cache": c["v_cache"].clone()}).clone()
    torch.cuda.synchronize()
    turns, axis = pa.rope_table(128, 128, sections=c["sections"], device=DEV)
    out = torch.zeros_like(want)
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        pa.pa_rope_append(out, c["q"], c["k"], c["v"], c["k_cache"], c["v_cache"], c["pos"],
                          c["slots"], turns, axis)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_rope_append(out, c["q"], c["k"], c["v"], c["k_cache"], c["v_cache"], c["pos"],
                          c["slots"], turns, axis)
    out.zero_()
    c["pos"].zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, c["q"])


def test_nothing_to_do(pa):
    c = make(7, 4, 2, 2, 64, 8, "fp16", 1, 64, False, False, False)
    turns, axis = pa.rope_table(64, device=DEV)
    e = c["q"][:0]
    assert pa.pa_rope_append(e, e, c["k"][:0], c["v"][:0], c["k_cache"], c["v_cache"],
                             c["pos"][:, :0], c["slots"][:0], turns, axis) is e
