"""The block-scaled FP8 cache on the GPU: the append byte for byte against the definition,
attention against 64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import _pool_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"fp16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_20_gb300 as pa
    pa.load()
    assert pa.pa_device_error() == 0
    return pa


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def pool(rng, n, width, h, bs, extra=3, d=128):
    """Random codes (NaN ones among them) and scales, tables over a permutation."""
    nb = n * width + extra
    tables = rng.permutation(nb)[:n * width].reshape(n, width).astype(np.int32)
    kc, vc = (rng.integers(0, 256, (nb, h, bs, d)).astype(np.uint8) for _ in range(2))
    scales = (2.0 ** rng.integers(-9, 3, (nb, h, 2))).astype(np.float32)
    return kc, vc, scales, tables


def on(x):
    return torch.from_numpy(np.ascontiguousarray(x)).to(DEV)


def values(rng, shape, dtype, size=1.0):
    x = rng.standard_normal(shape) * size
    x = np.where(rng.random(shape[:2] + (1,)) < 0.1, 40 * x, x)
    return torch.from_numpy(x).to(DT[dtype])


def run_append(pa, state, k_new, v_new, lens, q_len):
    kc, vc, scales, tables = state
    g = [on(a) for a in state]
    pa.pa_append_kv_block_scaled(g[0], g[1], g[2], k_new.to(DEV), v_new.to(DEV), g[3],
                                 on(np.asarray(lens, np.int32)), q_len=q_len)
    torch.cuda.synchronize()
    ref.append(kc, vc, scales, f64(k_new), f64(v_new), tables, lens, q_len)
    assert np.array_equal(g[2].cpu().numpy(), scales, equal_nan=True)
    # (a NaN keeps no sign: 0x7f and 0xff are one value)
    for got, want in ((g[0], kc), (g[1], vc)):
        got = got.cpu().numpy()
        assert np.array_equal(np.where((got & 127) == 127, 127, got), np.where((want & 127) == 127, 127, want))


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
@pytest.mark.parametrize("q_len,lens", [(1, (1, 17, 0, 8, 33, 40)), (3, (2, 3, 16, 18, 64, 65)),
                                        (40, (40, 39, 71, 96, 7, 0)), (97, (97, 100, 128, 1, 96, 111))])
def test_append(pa, bs, dtype, q_len, lens):
    rng = np.random.default_rng(bs * 100 + q_len)
    n, h = len(lens), 3
    state = pool(rng, n, 128 // bs, h, bs)
    k, v = (values(rng, (n * q_len, h, 128), dtype, s) for s in (1.0, 0.02))
    run_append(pa, state, k, v, lens, q_len)
    assert pa.pa_device_error() == 0


def test_append_token_by_token_with_growing_rows(pa):
    """Every token larger than the last: the scale grows, older codes are rounded again."""
    rng = np.random.default_rng(5)
    state = pool(rng, 2, 3, 2, 16)
    for t in range(40):
        size = 2.0 ** (rng.integers(-12, 12))
        k, v = (values(rng, (2, 2, 128), "bf16", size) for _ in range(2))
        run_append(pa, state, k, v, (t + 1, max(1, t - 5)), 1)


@pytest.mark.parametrize("old", [0.0, math.nan, 0.3, 2.0 ** -60, 2.0 ** 60, math.inf, -1.0])
def test_append_over_foreign_scales(pa, old):
    """Scales that the append did not write: clamped, others kept where they suffice."""
    rng = np.random.default_rng(9)
    state = pool(rng, 2, 2, 2, 16)
    state[2][:] = old
    k, v = (values(rng, (2, 2, 128), "fp16", s) for s in (1.0, 100.0))
    run_append(pa, state, k, v, (7, 20), 1)


def test_append_of_special_values(pa):
    rng = np.random.default_rng(11)
    state = pool(rng, 4, 2, 1, 8)
    k = values(rng, (4 * 5, 1, 128), "bf16")
    v = k.clone()
    k[3, 0, 5], k[3, 0, 6], k[4, 0, 1] = math.inf, -math.inf, math.nan
    k[7] = math.inf        # a row with nothing finite
    k[10:15] = 0           # zeros, negative ones among them
    k[11, 0, ::2] = -0.0
    v[:5] = v[:5] * 1e30   # past the range of scales: saturates
    v[5:10] = v[5:10] * 1e-30
    v[15:] = math.nan
    run_append(pa, state, k, v, (5, 5, 11, 13), 5)


def test_append_of_strided_tokens(pa):
    rng = np.random.default_rng(12)
    h, n, u = 2, 3, 9
    kc, vc, scales, tables = state = pool(rng, n, 4, h, 16)
    qkv = values(rng, (n * u, 4 * h, 128), "fp16")
    dev = qkv.to(DEV)
    g = [on(a) for a in state]
    lens = (9, 30, 41)
    pa.pa_append_kv_block_scaled(g[0], g[1], g[2], dev[:, 2 * h:3 * h], dev[:, 3 * h:], g[3],
                                 on(np.asarray(lens, np.int32)), q_len=u)
    ref.append(kc, vc, scales, f64(qkv[:, 2 * h:3 * h]), f64(qkv[:, 3 * h:]), tables, lens, u)
    assert np.array_equal(g[0].cpu().numpy(), kc) and np.array_equal(g[1].cpu().numpy(), vc)
    assert np.array_equal(g[2].cpu().numpy(), scales)


def test_append_skips_and_reports_bad_blocks(pa):
    rng = np.random.default_rng(13)
    for bad, lens in ((10 ** 6, (20, 20)), (-1, (20, 20)), (None, (20, 70))):
        state = pool(rng, 2, 2, 2, 16)
        if bad is not None:
            state[3][1, 1] = bad
        k, v = (values(rng, (2 * 6, 2, 128), "fp16") for _ in range(2))
        run_append(pa, state, k, v, lens, 6)
        assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK


# ------------------------------------------------------------------- attention
def bound(wv, mags, T, out, dtype):
    """Error of an output element.  base-2 scores: fp32 sums of 128 products (2^-17 of
    sum |q k|, chains of at most 128), q brought to fp16 by a power of two (an element far
    below its row's largest: 2^-25 of that), the multiply-add and the exponential's argument
    (2^-23 of |s|; the running maximum carries log2 of V's scale, at most 40: 2^-18), exp2 2^-22:
    each moves a weight by ln 2 times that, and its sum once more.  Weight times V scale to fp16: half a
    step 2^-11, or below 2^-14 of the largest such product 2^-25 of it, for T rows times
    448 times the largest scale.  Output: half a step."""
    s_max, dot, sv, spread = (mags[..., i:i + 1] for i in range(4))
    delta = 0.694 * (dot * 2.0 ** -17 + spread * 2.0 ** -25 + s_max * 2.0 ** -23 + 2.0 ** -18 + 2.0 ** -22)
    step = {"fp16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
    tiny = 2.0 ** -25 if dtype == "fp16" else 0.0
    return wv * (2.0 ** -11 + 2 * delta) * 1.01 + T * 2.0 ** -25 * 448 * sv + np.abs(out) * step + tiny


def filled(rng, lens, h, bs, width, spread=4):
    """A pool whose rows stand for ordinary values under scales of any size; codes past the
    sequences' ends, and blocks of nobody's, are NaN."""
    n = len(lens)
    nb = n * width + 3
    tables = rng.permutation(nb)[:n * width].reshape(n, width).astype(np.int32)
    kc, vc = (np.full((nb, h, bs, 128), 127, np.uint8) for _ in range(2))
    scales = np.full((nb, h, 2), np.nan, np.float32)
    for i, L in enumerate(lens):
        for lb in range(-(-L // bs)):
            b, r = tables[i, lb], min(bs, L - lb * bs)
            scales[b] = 2.0 ** rng.integers(-8 - spread, -7, (h, 2))
            for cache in (kc, vc):
                cache[b, :, :r] = ref.e4m3(rng.standard_normal((h, r, 128)) * 100)
    return kc, vc, scales, tables


def check(pa, rng, state, q, lens, scale, dtype, **kw):
    kc, vc, scales, tables = state
    g = [on(a) for a in state]
    qd = q.to(DEV)
    out = torch.full_like(qd, math.nan)
    pa.pa_decode_block_scaled(out, qd, g[0], g[1], g[2], g[3], on(np.asarray(lens, np.int32)), scale,
                              q_len=q.shape[1], **kw)
    torch.cuda.synchronize()
    want, wv, mags = ref.attend(f64(q), kc, vc, scales, tables, lens, scale)
    got = f64(out)
    assert np.isfinite(got).all()
    over = np.abs(got - want) - bound(wv, mags, max(max(lens), 1), want, dtype)
    assert over.max() <= 0, (np.unravel_index(over.argmax(), over.shape), over.max())
    return out


LENS = (1, 16, 37, 0, 130, 5)


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("group", [1, 2, 3, 8, 12, 16, 20])
@pytest.mark.parametrize("dtype", ["fp16", "bf16"])
def test_decode(pa, bs, group, dtype):
    rng = np.random.default_rng(bs + group)
    h = 2
    state = filled(rng, LENS, h, bs, 160 // bs)
    q = torch.from_numpy(rng.standard_normal((len(LENS), 1, h * group, 128))).to(DT[dtype])
    for splits in (1, 3):
        check(pa, rng, state, q, LENS, 0.09, dtype, num_splits=splits)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("bs", [8, 16, 32])
@pytest.mark.parametrize("q_len,group,dtype", [(2, 1, "fp16"), (4, 4, "bf16"), (16, 2, "fp16"), (17, 1, "bf16"),
                                               (17, 3, "fp16"), (64, 4, "bf16"), (130, 1, "fp16"),
                                               (129, 8, "bf16")])
def test_many_query_rows(pa, bs, q_len, group, dtype):
    rng = np.random.default_rng(bs + q_len)
    lens = (q_len, 300, q_len + 1, 3, 0, 141)  # (3 and 0: rows that see nothing)
    h = 2
    state = filled(rng, lens, h, bs, 320 // bs)
    q = torch.from_numpy(rng.standard_normal((len(lens), q_len, h * group, 128))).to(DT[dtype])
    for splits in (1, 2):
        check(pa, rng, state, q, lens, 0.09, dtype, num_splits=splits)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("q_len,group", [(1, 1), (1, 4), (4, 4), (20, 4)])
@pytest.mark.parametrize("spread", [40, 70])
def test_scales_far_apart(pa, q_len, group, spread):
    """Blocks whose V scales lie up to 70 binary orders apart, blocks of zeros among them."""
    rng = np.random.default_rng(spread + q_len)
    lens, h, bs = (100, 64, 200), 2, 16
    kc, vc, scales, tables = state = filled(rng, lens, h, bs, 16)
    used = np.unique(tables[:, :13])
    scales[used, :, 1] = 2.0 ** rng.integers(-40, spread - 40 + 1, (len(used), h))
    scales[used, :, 0] = 2.0 ** -9
    zero = used[::5]
    vc[zero] &= 128           # (codes past the sequences' ends lose their NaN here)
    scales[zero, :, 1] = 0.0  # counts as the least scale
    q = torch.from_numpy(rng.standard_normal((len(lens), q_len, h * group, 128))).to(torch.bfloat16)
    check(pa, rng, state, q, lens, 0.09, "bf16")


@pytest.mark.parametrize("scale", [0.0, -0.09, 30.0])
@pytest.mark.parametrize("q_len", [1, 33])
def test_softmax_scales(pa, scale, q_len):
    """No scale (equal weights), a negative one, and one that leaves a single weight."""
    rng = np.random.default_rng(3)
    lens, h, bs = (50, 77), 2, 16
    state = filled(rng, lens, h, bs, 5)
    q = torch.from_numpy(rng.standard_normal((2, q_len, 4 * h, 128))).to(torch.float16)
    check(pa, rng, state, q, lens, scale, "fp16")


@pytest.mark.parametrize("q_len", [1, 40])
def test_bad_blocks_read_as_zeros(pa, q_len):
    rng = np.random.default_rng(4)
    lens, h, bs = (60, 90), 2, 16
    state = filled(rng, lens, h, bs, 6)
    state[3][0, 1], state[3][1, 2] = 10 ** 6, -7
    q = torch.from_numpy(rng.standard_normal((2, q_len, 8, 128))).to(torch.float16)
    check(pa, rng, state, q, lens, 0.09, "fp16")
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK


@pytest.mark.parametrize("q_len,dtype", [(1, "fp16"), (24, "bf16")])
def test_append_then_attend(pa, q_len, dtype):
    """Attention of this step's queries over what the step appended, against attention of
    the 16-bit rows: K and V differ from them by half a step of e4m3 (2^-4), or below the
    normal codes by 2^-10 of a block's scale."""
    rng = np.random.default_rng(q_len)
    n, h, bs, L = 3, 2, 16, 48
    kc, vc, scales, tables = pool(rng, n, 4, h, bs)
    g = [on(a) for a in (kc, vc, scales, tables)]
    rows = [values(rng, (n * L, h, 128), dtype) for _ in range(2)]
    for t0 in range(0, L, q_len):
        part = [r.view(n, L, h, 128)[:, t0:t0 + q_len].reshape(-1, h, 128).contiguous().to(DEV) for r in rows]
        lens = np.full(n, t0 + q_len, np.int32)
        pa.pa_append_kv_block_scaled(g[0], g[1], g[2], *part, g[3], on(lens), q_len=q_len)
    q = torch.from_numpy(rng.standard_normal((n, q_len, 2 * h, 128))).to(DT[dtype])
    back = [a.cpu().numpy() for a in g]
    for cache, which, r in ((back[0], 0, rows[0]), (back[1], 1, rows[1])):
        for i in range(n):
            ids = tables[i, :L // bs]
            got = (ref.E4M3[cache[ids]] * back[2][ids][:, :, which, None, None]).transpose(0, 2, 1, 3).reshape(L, h, 128)
            want = f64(r).reshape(n, L, h, 128)[i]
            s = np.repeat(back[2][ids][:, :, which], bs, axis=0)[:, :, None]
            # (a row rounded again after its block's scale grew: a second half step below
            # the normal codes)
            assert (np.abs(got - want) <= np.maximum(np.abs(want) * 2.0 ** -4, 2 * 2.0 ** -10 * s)).all()
    check(pa, rng, back, q, np.full(n, L), 0.05, dtype)
