"""Calls on a stream that is named, with buffers that the binding makes: the results are
those of the current stream whatever the current stream does meanwhile (needs a GPU)."""
import numpy as np
import pytest
import torch

from tests import test_gpu_evict as evicts
from tests import test_gpu_scored as scoreds
from tests import test_gpu_verify as verifies

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_20_gb300 as pa
    pa.load()
    assert pa.pa_device_error() == 0
    return pa


def meanwhile(setup, call):
    """call(stream, *setup()) on a stream that is still busy, the current stream taking and
    filling whatever memory it is given; then again by the stream's raw handle."""
    torch.cuda.empty_cache()
    got = []
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        state = setup()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms
        out = call(stream, *state)
        pools = {s["stream"] for s in torch.cuda.memory_snapshot()}
        assert side.cuda_stream in pools
        hogs = [torch.full((n,), 255, dtype=torch.uint8, device=DEV)
                for n in (512, 4096, 1 << 16, 1 << 18, 1 << 20, 1 << 22, 1 << 24) for _ in range(4)]
        torch.cuda.synchronize()
        assert all(bool((h == 255).all()) for h in hogs)
        got.append(out)
    return got


@pytest.mark.parametrize("few", [False, True])
def test_evict(pa, few):
    # more moves than one CTA lists itself, and a context of several CTAs
    lens = [5000, 2003] if not few else [2003, 2001]
    budget = 1500 if not few else 2000
    c = evicts.make(31, lens, 2, 64, 16)
    want = evicts.run(pa, c, budget, 4, 100, False)[:5]

    def setup():
        return (*(c[x].to(DEV).view(torch.bfloat16) for x in ("k", "v")), c["scores"].to(DEV), c["pos"].to(DEV),
                c["table"].to(DEV), *(torch.tensor(c[x], dtype=torch.int32, device=DEV) for x in ("lens", "sl")))

    def call(stream, k, v, scores, pos, table, cl, sl):
        new = pa.pa_evict(k, v, scores, pos, table, cl, sl, budget, 4, 100, stream=stream)
        return k, v, scores, pos, new, (table, cl, sl)

    for got in meanwhile(setup, call):
        for x, y in zip(got[:5], want):
            assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("u,splits", [(1, 4), (4, 1), (6, 3), (40, 1)])
def test_decode_scored(pa, u, splits):
    c = scoreds.make(32, [900, 500], u, 16, 2, 128, 16, "bf16", False)
    want = scoreds.run(pa, c, splits)

    def setup():
        return torch.empty_like(c["q"]), c["scores"].clone(), c["pos"].clone()

    def call(stream, out, scores, pos):
        pa.pa_decode_scored(out, scores, c["q"], c["k"], c["v"], c["table"], c["cl"], c["scale"], q_len=u,
                            num_splits=splits, row_pos=pos, seq_lens=c["sl"], stream=stream)
        return out, scores, pos

    for got in meanwhile(setup, call):
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert pa.pa_device_error() == 0


def test_verify_drafts(pa):
    c = verifies.make(33, 5, 3, 4001)
    lens = [10, 11, 12, 13, 14]
    want = verifies.both(pa, c, lens=lens)
    d = {a: b.to(DEV) for a, b in c.items()}
    cl = torch.tensor(lens, dtype=torch.int32, device=DEV)
    for got in meanwhile(tuple, lambda s: pa.pa_verify_drafts(d["p"], d["q"], d["x"], d["au"], d["su"],
                                                              context_lens=cl, stream=s)):
        for x, y in zip(got, want):
            assert torch.equal(x, y)


@pytest.mark.parametrize("how", ["append", "fp8", "cascade", "step", "step in partitions"])
def test_attention(pa, how):
    r = np.random.default_rng(5)
    n, hq, hkv, d, bs, width = 3, 8, 2, 128, 16, 20
    blocks = n * width + 1
    fp8 = how == "fp8"
    k, v = (torch.from_numpy(r.standard_normal((blocks, hkv, bs, d)).astype(np.float32)).to(DEV) for _ in range(2))
    to = (lambda x: (x / 0.03).to(torch.float8_e4m3fn).view(torch.uint8)) if fp8 else lambda x: x.bfloat16()
    k, v = to(k), to(v)
    tables = torch.arange(n * width, dtype=torch.int32, device=DEV).view(n, width).contiguous()
    tables[:, :4] = tables[0, :4].clone()  # (a shared prefix)
    lens = torch.tensor([300, 100, 211], dtype=torch.int32, device=DEV)
    q, kn, vn = (torch.from_numpy(r.standard_normal(s).astype(np.float32)).bfloat16().to(DEV)
                 for s in ((n, 1, hq, d), (n, hkv, d), (n, hkv, d)))
    sc = torch.full((hkv,), 0.03, device=DEV)

    def setup():
        return k.clone(), v.clone(), torch.empty_like(q)

    def call(stream, kc, vc, out):
        if fp8:
            pa.pa_decode_fp8(out, q, kc, vc, sc, sc, tables, lens, 0.09, num_splits=3, k_new=kn, v_new=vn,
                             stream=stream)
        elif how == "append":
            pa.pa_append_decode(out, q, kn, vn, kc, vc, tables, lens, 0.09, num_splits=3, stream=stream)
        elif how == "cascade":
            pa.pa_decode_cascade(out, q, kc, vc, tables, lens, 0.09, 4, k_new=kn, v_new=vn, stream=stream)
        else:
            out = pa.paged_decode_step(q, kn, vn, kc, vc, tables, lens, 0.09,
                                       num_splits=1 if how == "step" else 3, stream=stream)
        return out, kc, vc

    want = call(None, *setup())
    torch.cuda.synchronize()
    for got in meanwhile(setup, call):
        for x, y in zip(got, want):
            assert torch.equal(x, y)
    assert pa.pa_device_error() == 0
