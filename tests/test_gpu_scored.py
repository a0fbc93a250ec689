"""pa_decode_scored against 64-bit attention with its weights summed per cached row
(needs a GPU)."""
import math

import numpy as np
import pytest
import torch

from tests import _ops_ref as ref
from tests import _tol

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


def make(seed, lens, u, hq, hkv, d, bs, dtype, fp8, spare=1):
    """Caches whose slots past each context are NaN, ledgers whose rows there are marked."""
    g = torch.Generator().manual_seed(seed)
    n, dt = len(lens), DTYPES[dtype]
    per = [-(-x // bs) for x in lens]
    width = max(1, max(per)) + spare
    blocks = sum(per) + 3
    order = torch.randperm(blocks, generator=g, dtype=torch.int32)
    table = torch.full((n, width), int(order[-1]), dtype=torch.int32)
    k, v = (torch.full((blocks, hkv, bs, d), float("nan")) for _ in range(2))
    at = 0
    for i, m in enumerate(per):
        own = order[at:at + m]
        table[i, :m] = own
        at += m
        for j, b in enumerate(own.tolist()):
            rows = min(bs, lens[i] - j * bs)
            k[b, :, :rows] = torch.randn(hkv, rows, d, generator=g)
            v[b, :, :rows] = torch.randn(hkv, rows, d, generator=g)
    c = dict(lens=lens, u=u, scale=d ** -0.5, ks=None, vs=None, bs=bs)
    if fp8:
        sc = [torch.rand(hkv, generator=g).mul(0.03).add(0.02) for _ in range(2)]
        k, v = ((x / s[:, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                for x, s in zip((k, v), sc))
        c["ks"], c["vs"] = sc[0].to(DEV), sc[1].to(DEV)
    else:
        k, v = k.to(dt), v.to(dt)
    c["k"], c["v"], c["table"] = k.to(DEV), v.to(DEV), table.to(DEV)
    c["cl"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    c["sl"] = c["cl"] + 5
    c["q"] = torch.randn(n, u, hq, d, generator=g).to(dt).to(DEV)
    c["scores"] = torch.rand(n, hkv, width * bs, generator=g).mul(2).to(DEV)
    c["pos"] = torch.randint(0, 99, c["scores"].shape, generator=g, dtype=torch.int32).to(DEV)
    return c


def run(pa, c, splits=1, **kw):
    out = torch.full_like(c["q"], float("nan"))
    scores, pos = c["scores"].clone(), c["pos"].clone()
    n, u, hq, d = c["q"].shape
    nb = pa.pa_decode_scored_workspace_size(n, hq, u, d, splits, c["table"].shape[1], c["bs"])
    ws = torch.full((nb,), 0xFF, dtype=torch.uint8, device=DEV)  # NaN
    kw = {"row_pos": pos, "seq_lens": c["sl"], **kw}
    pa.pa_decode_scored(out, scores, c["q"], c["k"], c["v"], c["table"], c["cl"], c["scale"],
                        q_len=u, num_splits=splits, workspace=ws, k_scale=c["ks"], v_scale=c["vs"],
                        **kw)
    torch.cuda.synchronize()
    return out, scores, pos


def caches64(c):
    if c["ks"] is None:
        return ref.f64(c["k"]), ref.f64(c["v"])
    return tuple(ref.e4m3_values(c[x].cpu()) * ref.f64(c[s])[:, None, None]
                 for x, s in (("k", "ks"), ("v", "vs")))


def check(c, got, dtype, what=""):
    out, scores, pos = got
    k, v = caches64(c)
    q = ref.f64(c["q"])
    want, ledger, share, biggest = ref.scored(q, k, v, c["table"].cpu().numpy(), c["lens"],
                                              c["scale"], ref.f64(c["scores"]))
    _tol.check(ref.f64(out), want, dtype, what)
    # A score s is a sum of D fp32 products: off by at most (D + 2) 2^-24 sum |q k| scale
    # (biggest), and over an FP8 cache a q scaled into fp16 adds 2^-25 of its largest
    # element per product.  A weight e^(s - m) / l then carries that twice (its own and
    # l's), and about 8 more roundings of 2^-24; the row's sum over up to `rows` weights
    # and the old score adds rows + 2.
    d, rows = q.shape[3], q.shape[1] * q.shape[2] // k.shape[1]
    ds = (d + 2) * 2.0 ** -24 * biggest
    if c["ks"] is not None:
        ds += d * 2.0 ** -25 * np.abs(q).max() * np.nanmax(np.abs(k)) * c["scale"]
    rel = 2 * ds + (8 + rows + 2) * 2.0 ** -24
    err = np.abs(ref.f64(scores) - ledger)
    bad = err > rel * share + 2.0 ** -23 * np.abs(ledger) + 1e-30
    assert not bad.any(), (what, int(bad.sum()), float(err.max()), rel)
    exp = c["pos"].cpu().numpy().copy()
    for i, L in enumerate(c["lens"]):
        for t in range(max(0, L - c["u"]), L):
            exp[i, :, t] = int(c["sl"][i]) - L + t
    assert np.array_equal(pos.cpu().numpy(), exp), what
    # rows past the context: bit for bit what they were
    for i, L in enumerate(c["lens"]):
        assert torch.equal(scores[i, :, L:], c["scores"][i, :, L:]), what


SHAPES = [
    # lens, u, hq, hkv, d, bs, dtype, fp8
    ([1, 17, 37], 1, 4, 4, 64, 16, "fp16", False),
    ([1, 16, 0, 250], 1, 8, 8, 128, 16, "bf16", False),
    ([300, 33], 1, 4, 2, 128, 8, "fp16", False),
    ([129, 64, 1], 1, 12, 4, 128, 32, "bf16", False),
    ([500, 7], 1, 32, 8, 128, 16, "bf16", False),
    ([77], 1, 16, 2, 64, 8, "bf16", False),
    ([200, 15, 3], 1, 16, 1, 128, 16, "fp16", False),      # 16 rows
    ([100, 31], 1, 40, 1, 64, 16, "fp16", False),          # 40 rows: three row groups
    ([90, 2, 0, 3], 4, 8, 2, 128, 16, "bf16", False),      # shorter than q_len
    ([260, 40], 16, 8, 8, 128, 32, "fp16", False),
    ([50, 6], 3, 4, 4, 64, 8, "bf16", False),
    ([70, 20], 13, 10, 2, 128, 16, "fp16", False),         # 65 rows
    ([1, 17, 300], 1, 6, 6, 128, 16, "fp16", True),
    ([40, 129], 1, 4, 2, 128, 8, "bf16", True),
    ([333, 5], 1, 10, 2, 128, 16, "bf16", True),
    ([64, 100], 4, 12, 4, 128, 32, "fp16", True),
    ([90, 300], 7, 8, 4, 128, 16, "bf16", True),
]
MANY = [
    ([17, 300], 17, 4, 4, 64, 16, "fp16", False),
    ([100, 0, 30], 40, 8, 2, 128, 16, "bf16", False),      # one empty, one shorter than q_len
    ([513, 129], 100, 4, 2, 128, 8, "fp16", False),
    ([700], 300, 5, 1, 128, 32, "bf16", False),
    ([257, 64], 64, 3, 3, 64, 8, "bf16", False),
    ([300, 20], 17, 135, 1, 64, 16, "bf16", False),        # more heads than a block of rows
    ([600, 511], 150, 8, 8, 128, 16, "fp16", False),
    ([520, 256, 257], 90, 7, 1, 128, 16, "bf16", False),
    ([200, 50], 33, 6, 2, 128, 16, "fp16", True),
    ([150, 290], 129, 4, 1, 128, 32, "bf16", True),
]


@pytest.mark.parametrize("splits", [1, 3])
@pytest.mark.parametrize("shape", SHAPES)
def test_up_to_16_query_tokens(pa, shape, splits):
    c = make(11, *shape)
    check(c, run(pa, c, splits), shape[6], f"{shape} splits {splits}")
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("shape", MANY)
def test_many_query_tokens(pa, shape):
    c = make(12, *shape)
    check(c, run(pa, c), shape[6], str(shape))
    assert pa.pa_device_error() == 0


def test_many_sequences(pa):
    """More sequences than one launch of the many-row pass takes."""
    lens = [17 + i % 3 for i in range(4099)]
    c = make(22, lens, 17, 1, 1, 64, 32, "fp16", False, spare=0)
    check(c, run(pa, c), "fp16")


def test_agrees_with_the_plain_calls(pa):
    """The output is pa_decode's, bit for bit: the scores are only written besides."""
    for shape in (SHAPES[4], SHAPES[8], MANY[1]):
        c = make(13, *shape)
        plain = torch.empty_like(c["q"])
        pa.pa_decode(plain, c["q"], c["k"], c["v"], c["table"], c["cl"], c["scale"], c["u"])
        assert torch.equal(run(pa, c)[0], plain)


def test_weights_of_a_row_sum_to_one(pa):
    c = make(14, [1000, 3, 0, 64], 1, 32, 8, 128, 16, "bf16", False)
    c["scores"].zero_()
    scores = run(pa, c)[1]
    total = scores.double().sum(-1).cpu().numpy()
    # 4 heads' rows a KV head, each weight off by at most 1e-4 of itself
    assert np.allclose(total, np.array([4, 4, 0, 4])[:, None], atol=4e-4)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3.0])
@pytest.mark.parametrize("u", [1, 5, 40])
def test_scales(pa, scale, u):
    c = make(15, [150, 41], u, 4, 2, 128, 16, "fp16", False)
    c["scale"] = scale
    check(c, run(pa, c), "fp16", f"scale {scale}")


def test_peaked_rows(pa):
    c = make(16, [400, 90], 2, 8, 2, 128, 16, "bf16", False)
    c["q"] *= 20
    check(c, run(pa, c), "bf16")


@pytest.mark.parametrize("u", [1, 3, 64])
def test_no_positions(pa, u):
    c = make(17, [100, 9], u, 4, 4, 64, 16, "fp16", False)
    out, scores, pos = run(pa, c)
    other = run(pa, c, row_pos=None, seq_lens=None)
    assert torch.equal(out, other[0]) and torch.equal(scores, other[1])
    assert torch.equal(other[2], c["pos"])


@pytest.mark.parametrize("shape", [SHAPES[4], SHAPES[7], SHAPES[14], MANY[1], MANY[6]])
def test_runs_are_bit_equal_and_independent_of_block_order(pa, shape):
    c = make(18, *shape)
    a = run(pa, c)
    for x, y in zip(a, run(pa, c)):
        assert torch.equal(x, y)
    perm = torch.randperm(c["k"].shape[0], generator=torch.Generator().manual_seed(1))
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(len(perm))
    d = {**c, "k": c["k"][perm.to(DEV)].contiguous(), "v": c["v"][perm.to(DEV)].contiguous(),
         "table": inv.to(torch.int32).to(DEV)[c["table"].long()].contiguous()}
    for x, y in zip(a, run(pa, d)):
        assert torch.equal(x, y)


@pytest.mark.parametrize("u", [1, 4, 33])
def test_bad_blocks_read_as_zeros(pa, u):
    c = make(19, [100, 70], u, 4, 2, 128, 16, "fp16", False)
    bad = {**c, "table": c["table"].clone()}
    bad["table"][0, 2] = 10 ** 6
    bad["table"][1, 0] = -4
    got = run(pa, bad)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    zero = {**c, "k": c["k"].clone(), "v": c["v"].clone()}
    for i, j in ((0, 2), (1, 0)):
        zero["k"][c["table"][i, j].long()] = 0
        zero["v"][c["table"][i, j].long()] = 0
    check(zero, got, "fp16")


def test_context_longer_than_its_table(pa):
    c = make(20, [64, 30], 1, 4, 2, 128, 16, "fp16", False, spare=0)
    c["cl"][0] = 70  # the table covers 64 rows
    out, scores, _ = run(pa, c)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert torch.isfinite(out).all() and torch.isfinite(scores).all()


@pytest.mark.parametrize("u,splits", [(1, 1), (1, 4), (4, 1), (40, 1)])
def test_side_stream_and_graph(pa, u, splits):
    c = make(21, [300, 77], u, 8, 2, 128, 16, "bf16", False)
    want = run(pa, c, splits)
    out, scores, pos = torch.empty_like(c["q"]), c["scores"].clone(), c["pos"].clone()
    nb = pa.pa_decode_scored_workspace_size(2, 8, u, 128, splits, c["table"].shape[1], 16)
    ws = torch.empty(nb, dtype=torch.uint8, device=DEV)

    def call():
        pa.pa_decode_scored(out, scores, c["q"], c["k"], c["v"], c["table"], c["cl"], c["scale"],
                            q_len=u, num_splits=splits, workspace=ws, row_pos=pos, seq_lens=c["sl"])

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    for x, y in zip((out, scores, pos), want):
        assert torch.equal(x, y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    out.zero_()
    scores.copy_(c["scores"])
    pos.copy_(c["pos"])
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((out, scores, pos), want):
        assert torch.equal(x, y)


def test_two_streams_with_their_own_workspaces(pa):
    cs = [make(30 + i, [900, 500], 1, 8, 2, 128, 16, "bf16", False) for i in range(2)]
    want = [run(pa, c, 2) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    state = []
    for c in cs:
        nb = pa.pa_decode_scored_workspace_size(2, 8, 1, 128, 2, c["table"].shape[1], 16)
        state.append((torch.empty_like(c["q"]), c["scores"].clone(),
                      torch.empty(nb, dtype=torch.uint8, device=DEV)))
    torch.cuda.synchronize()
    for _ in range(10):
        for c, s, (out, scores, ws) in zip(cs, streams, state):
            with torch.cuda.stream(s):
                scores.copy_(c["scores"])
                pa.pa_decode_scored(out, scores, c["q"], c["k"], c["v"], c["table"], c["cl"],
                                    c["scale"], num_splits=2, workspace=ws)
    torch.cuda.synchronize()
    for (out, scores, _), w in zip(state, want):
        assert torch.equal(out, w[0]) and torch.equal(scores, w[1])


@pytest.mark.parametrize("seed", range(20))
def test_random_shapes(pa, seed):
    r = np.random.default_rng(500 + seed)
    fp8 = bool(r.random() < 0.3)
    hkv, grp = int(r.choice([1, 2, 3, 8])), int(r.choice([1, 2, 3, 4, 5, 8]))
    u = int(r.choice([1, 1, 2, 4, 9, 16, 17, 50]))
    lens = [int(x) for x in r.integers(0, 700, size=int(r.integers(1, 5)))]
    dtype = str(r.choice(["fp16", "bf16"]))
    shape = (lens, u, hkv * grp, hkv, 128 if fp8 else int(r.choice([64, 128])),
             int(r.choice([8, 16, 32])), dtype, fp8)
    c = make(seed, *shape)
    check(c, run(pa, c, int(r.choice([1, 2, 7]))), dtype, str(shape))
    assert pa.pa_device_error() == 0 and math.isfinite(c["scale"])
