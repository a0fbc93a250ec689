"""Sizes at which the loops of scored attention and draft verification run more than once
per thread block: several units a block with several blocks of query rows each, and
vocabularies whose search takes a second piece (needs a GPU)."""
import numpy as np
import pytest
import torch

from tests import _ops_ref as ref
from tests import _tol
from tests import test_gpu_scored as scoreds
from tests import test_gpu_verify as verifies
from tests.test_gpu_scored import pa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"


def attention64(c):
    """(out, share, biggest) of tests/_ops_ref.scored, head by head in 64-bit torch."""
    n, u, hq, d = c["q"].shape
    k, v = scoreds.caches64(c)
    k, v = torch.from_numpy(k).to(DEV), torch.from_numpy(v).to(DEV)
    h = k.shape[1]
    g = hq // h
    out = torch.zeros(n, u, hq, d, dtype=torch.float64, device=DEV)
    share = torch.zeros(c["scores"].shape, dtype=torch.float64, device=DEV)
    biggest = 0.0
    for i, L in enumerate(c["lens"]):
        if L == 0:
            continue
        blocks = c["table"][i, :-(-L // c["bs"])].long()
        rows = [x[blocks].transpose(0, 1).reshape(h, -1, d)[:, :L] for x in (k, v)]
        sees = torch.arange(L, device=DEV) <= (L - u + torch.arange(u, device=DEV))[:, None]
        for j in range(h):
            q = c["q"][i, :, j * g:(j + 1) * g].double()                      # [u, g, d]
            s = torch.einsum("ugd,td->gut", q, rows[0][j]) * c["scale"]
            biggest = max(biggest, torch.einsum("ugd,td->gut", q.abs(), rows[0][j].abs()).max().item() * c["scale"])
            w = torch.softmax(s.masked_fill(~sees, -np.inf), -1).nan_to_num(0.0)
            out[i, :, j * g:(j + 1) * g] = torch.einsum("gut,td->ugd", w, rows[1][j])
            share[i, j, :L] = w.sum((0, 1))
    return out.cpu().numpy(), share.cpu().numpy(), biggest


@pytest.mark.parametrize("u,hq,hkv,d,bs,dtype,fp8", [
    (300, 32, 8, 128, 16, "bf16", False),
    (257, 16, 8, 128, 32, "fp16", True),
    (330, 24, 8, 64, 8, "fp16", False),     # three heads a group: 126 of a block's 128 rows
    (19, 16, 16, 128, 16, "bf16", True),    # one block of query rows a unit
])
def test_several_units_a_thread_block(pa, u, hq, hkv, d, bs, dtype, fp8):  # noqa: F811
    r = np.random.default_rng(u)
    lens = [int(x) for x in r.integers(1500, 4000, size=8)] + [u // 2, 0]
    c = scoreds.make(50, lens, u, hq, hkv, d, bs, dtype, fp8)
    units = sum(-(-x // 256) for x in lens) * hkv
    assert units > 3 * torch.cuda.get_device_properties(0).multi_processor_count
    out, scores, pos = scoreds.run(pa, c)
    want, share, biggest = attention64(c)
    _tol.check(ref.f64(out), want, dtype)
    # the bound on a row's share that tests/test_gpu_scored.py derives
    rows = u * hq // hkv
    ds = (d + 2) * 2.0 ** -24 * biggest
    if fp8:
        ds += d * 2.0 ** -25 * np.abs(ref.f64(c["q"])).max() * np.nanmax(np.abs(scoreds.caches64(c)[0])) * c["scale"]
    rel = 2 * ds + (8 + rows + 2) * 2.0 ** -24
    old, now, exp = ref.f64(c["scores"]), ref.f64(scores), c["pos"].cpu().numpy().copy()
    for i, L in enumerate(lens):
        old[i, :, max(0, L - u):L] = 0.0
        for t in range(max(0, L - u), L):
            exp[i, :, t] = int(c["sl"][i]) - L + t
        assert torch.equal(scores[i, :, L:], c["scores"][i, :, L:])
    ledger = old + share
    err = np.abs(now - ledger)
    bad = err > rel * share + 2.0 ** -23 * np.abs(ledger) + 1e-30
    assert not bad.any(), (int(bad.sum()), float(err.max()), rel)
    assert np.array_equal(pos.cpu().numpy(), exp)
    for x, y in zip(scoreds.run(pa, c), (out, scores, pos)):
        assert torch.equal(x, y)
    assert pa.pa_device_error() == 0


def per_warp(vocab):
    """Entries that a warp of a sequence's 64 sums, and searches 2048 at a time."""
    return ((vocab + 63) // 64 + 31) // 32 * 32


@pytest.mark.parametrize("bare", [False, True])   # whether a range's first 2048 entries weigh nothing
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("vocab", [131072, 131073, 160001])
def test_second_piece_of_a_search(pa, vocab, residual, bare):  # noqa: F811
    w = per_warp(vocab)
    at = [0, 1, 2047, 2048, 2049, w - 1, w, 5 * w + 2047, 5 * w + 2048, 5 * w + 2060, 6 * w - 1, 6 * w, 40 * w + 2050,
          41 * w - 1, vocab - w, vocab - 2, vocab - 1]
    at = sorted({v for v in at if 0 <= v < vocab})
    n = len(at)
    c = verifies.make(vocab % 1000, n, 1, vocab, sharp=0.5, apart=0.3)
    if bare:
        for first in (5 * w, 40 * w):
            c["p"][:, :, first:first + 2048] = 0.0
            if w == 2048:
                c["p"][:, :, first + 2040:first + 2048] = 1e-6
    # the draft is rejected (its token has no target weight), or there is none
    c["x"][:] = 7
    c["p"][:, 0, 7] = 0.0
    given = [1 if residual else 0] * n
    weights = ref.f64(c["p"])[:, 0] - (ref.f64(c["q"])[:, 0] if residual else 0.0)
    weights = np.where(weights > 0, weights, 0.0)
    total = np.cumsum(weights, -1)
    want = []
    for i, v in enumerate(at):
        v = int(np.nonzero(weights[i, v:])[0][0]) + v if weights[i, v:].any() else int(np.nonzero(weights[i])[0][-1])
        # the middle of the entry's share of the sum: no rounding comes near its borders
        c["su"][i] = float((total[i, v] - weights[i, v] / 2) / total[i, -1])
        want.append(v)
    got = verifies.both(pa, c, given=given)
    assert got[1].tolist() == [0] * n and got[0][:, 0].tolist() == want
    if w > 2048:
        assert any(v % w >= 2048 for v in want)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("sure", [False, True])
def test_large_vocabulary(pa, sure):  # noqa: F811
    c = verifies.make(60, 24, 2, 160001, sharp=1.0)
    c["su"] = torch.arange(24) / 24.0 + 0.02
    got = verifies.both(pa, c, sure=sure)
    assert (got[0].max(1).values.cpu() % per_warp(160001) >= 2048).any() or sure
    assert pa.pa_device_error() == 0


def test_longest_step(pa):  # noqa: F811
    """The most query tokens a call takes, over contexts as long, longer and shorter."""
    u, lens = 4096, [4096, 5001, 300, 4352]
    c = scoreds.make(51, lens, u, 2, 1, 64, 16, "bf16", False)
    out, scores, pos = scoreds.run(pa, c)
    want, share, biggest = attention64(c)
    _tol.check(ref.f64(out), want, "bf16")
    rel = 2 * (64 + 2) * 2.0 ** -24 * biggest + (8 + 2 * u + 2) * 2.0 ** -24
    old, now = ref.f64(c["scores"]), ref.f64(scores)
    for i, L in enumerate(lens):
        old[i, :, max(0, L - u):L] = 0.0
        at = torch.arange(max(0, L - u), L, dtype=torch.int32)
        assert torch.equal(pos[i, 0, max(0, L - u):L].cpu(), at + int(c["sl"][i]) - L)
    err = np.abs(now - (old + share))
    assert not (err > rel * share + 2.0 ** -23 * np.abs(old + share) + 1e-30).any(), float(err.max())
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("fp8", [False, True])
def test_caches_past_four_gigabytes(pa, fp8):  # noqa: F811
    """Blocks whose bytes and elements lie past 2^32 give what the same blocks give in a
    small pool, bit for bit."""
    n, hq, hkv, d, bs, u, drafts = 3, 16, 8, 128, 16, 40, 3
    lens, width = [700, 333, 40], 50
    blocks = (1 << 32) // (hkv * bs * d * (1 if fp8 else 2)) + n * width + 8
    assert blocks * hkv * bs * d > 1 << 31
    g = torch.Generator().manual_seed(52)
    spread = torch.randperm(n * width, generator=g).view(n, width).to(torch.int32)
    small = torch.randint(0, 255 if fp8 else 30000, (2, n * width, hkv, bs, d), generator=g)
    if fp8:
        small = torch.where(small % 128 == 127, 0, small).to(torch.uint8)   # (no NaN codes)
        sc = dict(k_scale=torch.full((hkv,), 0.01, device=DEV), v_scale=torch.full((hkv,), 0.02, device=DEV))
    else:
        small, sc = (small / 15000.0 - 1.0).bfloat16(), {}
    rnd = lambda *s: torch.randn(*s, generator=g).bfloat16()  # noqa: E731
    steps = [[rnd(n * t, h, d).to(DEV) for h in (hq, hkv, hkv)] for t in (u, 1 + drafts, 1)]
    turns, axis = pa.rope_table(d, device=DEV)
    got = []
    for first in (0, blocks - n * width):
        pool = torch.empty(2, blocks if first else n * width, hkv, bs, d, dtype=small.dtype, device=DEV)
        pool[:, first:first + n * width] = small.to(DEV)
        k, v = pool[0], pool[1]
        tables = (spread + first).to(DEV).contiguous()
        scores = torch.ones(n, hkv, width * bs, device=DEV)
        pos = torch.arange(width * bs, dtype=torch.int32, device=DEV).repeat(n, hkv, 1)
        ctx = torch.tensor(lens, dtype=torch.int32, device=DEV)
        outs = []
        for q, kn, vn in steps:
            t = q.shape[0] // n
            place = (ctx[:, None] - t + torch.arange(t, device=DEV)).reshape(1, -1).to(torch.int32)
            slots = pa.pa_slot_mapping(tables, ctx, bs, t)
            qr = torch.empty_like(q)
            pa.pa_rope_append(qr, q, kn, vn, k, v, place, slots, turns, axis, **sc)
            out = torch.empty(n, t, hq, d, dtype=q.dtype, device=DEV)
            pa.pa_decode_scored(out, scores, qr.view(n, t, hq, d), k, v, tables, ctx, d ** -0.5, q_len=t,
                                row_pos=pos, seq_lens=ctx, **sc)
            outs.append(out)
        new = pa.pa_evict(k, v, scores, pos, tables, ctx, ctx, 200, 2, 30)
        torch.cuda.synchronize()
        assert pa.pa_device_error() == 0
        got.append([*outs, scores, pos, new, k[first:first + n * width].clone(), v[first:first + n * width].clone()])
        del pool, k, v
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert all(torch.isfinite(x.float()).all() for x in got[0][:4]) and got[0][5].tolist() == [200, 200, 40]
