"""pa_evict against the definition: every kept row, position, score and byte of the pool
(needs a GPU)."""
import numpy as np
import pytest
import torch

from tests import _ops_ref as ref

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


def make(seed, lens, hkv, d, bs, nbytes=2, spare=1, zeros=0.2):
    """Rows of random bits; scores with many ties; positions in a random order."""
    g = torch.Generator().manual_seed(seed)
    n = len(lens)
    per = [-(-x // bs) for x in lens]
    width, blocks = max(1, max(per)) + spare, sum(per) + 3
    order = torch.randperm(blocks, generator=g, dtype=torch.int32)
    table = torch.full((n, width), int(order[-1]), dtype=torch.int32)
    at = 0
    for i, m in enumerate(per):
        table[i, :m] = order[at:at + m]
        at += m
    dt = torch.int16 if nbytes == 2 else torch.uint8
    lo, hi = (-32768, 32768) if nbytes == 2 else (0, 256)
    k, v = (torch.randint(lo, hi, (blocks, hkv, bs, d), generator=g).to(dt) for _ in range(2))
    rows = width * bs
    scores = torch.rand(n, hkv, rows, generator=g)
    scores[torch.rand(n, hkv, rows, generator=g) < zeros] = 0.0
    scores[torch.rand(n, hkv, rows, generator=g) < 0.1] = 0.5
    pos = torch.zeros(n, hkv, rows, dtype=torch.int32)
    for i, L in enumerate(lens):
        for h in range(hkv):
            # the first and the last positions are there, in between some are gone
            p = torch.arange(L, dtype=torch.int32)
            p[L // 2:] += 9
            pos[i, h, :L] = p[torch.randperm(L, generator=g)]
    return dict(lens=lens, k=k, v=v, table=table, scores=scores, pos=pos, bs=bs,
                sl=[L + 9 if L else 0 for L in lens])


def run(pa, c, budget, sinks, recent, apart):
    cache = torch.bfloat16 if c["k"].dtype == torch.int16 else torch.uint8
    k, v = (c[x].to(DEV).view(cache) for x in ("k", "v"))
    scores, pos = c["scores"].to(DEV), c["pos"].to(DEV)
    cl = torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    sl = torch.tensor(c["sl"], dtype=torch.int32, device=DEV)
    kw = {}
    if apart:
        kw = dict(scores_out=torch.full_like(scores, -7.0), row_pos_out=torch.full_like(pos, -7))
    new = pa.pa_evict(k, v, scores, pos, c["table"].to(DEV), cl, sl, budget, sinks, recent, **kw)
    torch.cuda.synchronize()
    so, po = (kw["scores_out"], kw["row_pos_out"]) if apart else (scores, pos)
    if apart:
        assert torch.equal(scores.cpu().view(torch.int32), c["scores"].view(torch.int32))
        assert torch.equal(pos.cpu(), c["pos"])
    return k, v, so, po, new, (scores, pos, cl, sl, kw)


def check(c, got, budget, sinks, recent, apart):
    bits = c["scores"].view(torch.int32).numpy()
    want = ref.evict(c["k"].numpy(), c["v"].numpy(), c["scores"].numpy(), c["pos"].numpy(),
                     c["table"].numpy(), np.array(c["lens"]), np.array(c["sl"]), budget, sinks, recent)
    k, v, so, po, new = got[:5]
    raw = torch.int16 if c["k"].dtype == torch.int16 else torch.uint8
    assert np.array_equal(new.cpu().numpy(), want[4])
    assert np.array_equal(k.cpu().view(raw).numpy(), want[0])
    assert np.array_equal(v.cpu().view(raw).numpy(), want[1])
    s, p = so.cpu().view(torch.int32).numpy(), po.cpu().numpy()
    ws = want[2].view(np.int32)
    for i, L in enumerate(want[4]):
        assert np.array_equal(s[i, :, :L], ws[i, :, :L])
        assert np.array_equal(p[i, :, :L], want[3][i, :, :L])
        # rows from the new length on are left as they were
        if apart:
            assert (so[i, :, L:] == -7.0).all() and (po[i, :, L:] == -7).all()
        else:
            assert np.array_equal(s[i, :, L:], bits[i, :, L:])
            assert np.array_equal(p[i, :, L:], c["pos"].numpy()[i, :, L:])


CASES = [
    # lens, hkv, d, bs, bytes, budget, sinks, recent
    ([33, 17, 0, 1], 2, 64, 8, 2, 16, 1, 4),
    ([17], 1, 128, 16, 2, 16, 0, 0),          # one row over
    ([65, 64, 63], 3, 128, 16, 2, 64, 4, 16),
    ([300, 90, 1000], 4, 128, 32, 2, 100, 4, 50),
    ([300, 5], 2, 128, 16, 1, 37, 0, 37),     # only the recent
    ([100, 120], 2, 64, 8, 2, 1, 1, 0),       # one row left
    ([100, 120], 1, 64, 16, 2, 1, 0, 0),
    ([2000, 1999], 2, 128, 8, 1, 700, 3, 200),
    ([513], 8, 64, 16, 2, 512, 4, 256),
    ([4100, 700], 2, 64, 32, 2, 1024, 4, 256),
    ([9001, 8998, 8995, 3], 2, 128, 16, 1, 8994, 4, 30),  # 7, 4, 1 and no rows over
    ([9001, 5000], 1, 64, 8, 2, 8993, 0, 8000),           # 8 over
    ([9001], 1, 64, 8, 2, 8992, 2, 100),                  # 9 over
    ([30, 27, 24, 23, 22], 3, 128, 8, 2, 22, 1, 3),
    ([12000, 40], 1, 128, 32, 2, 6000, 4, 64),            # many moves in a cluster
]


@pytest.mark.parametrize("apart", [False, True])
@pytest.mark.parametrize("case", CASES)
def test_every_byte(pa, case, apart):
    lens, hkv, d, bs, nb, budget, sinks, recent = case
    c = make(len(lens) + budget, lens, hkv, d, bs, nb)
    check(c, run(pa, c, budget, sinks, recent, apart), budget, sinks, recent, apart)
    assert pa.pa_device_error() == 0


def test_all_scores_equal_keeps_the_lowest_rows(pa):
    c = make(1, [500, 64], 2, 64, 16, zeros=1.1)
    c["scores"].zero_()
    check(c, run(pa, c, 60, 2, 8, False), 60, 2, 8, False)


def test_signed_zeros_infinities_and_nan(pa):
    c = make(2, [200, 300], 2, 64, 16)
    g = torch.Generator().manual_seed(5)
    for x in (float("nan"), float("inf"), -float("inf"), -0.0, 0.0, -3.0, 1e-45, -1e-45):
        c["scores"][torch.rand(c["scores"].shape, generator=g) < 0.1] = x
    for budget in (20, 100, 180):
        check(c, run(pa, c, budget, 3, 10, True), budget, 3, 10, True)


def test_more_rows_protected_than_fit(pa):
    # positions that repeat: more than `budget` rows count as recent
    c = make(3, [100], 2, 64, 16)
    c["pos"][:] = 1000
    check(c, run(pa, c, 30, 2, 10, False), 30, 2, 10, False)


def test_nothing_over_budget(pa):
    c = make(4, [10, 64, 0], 2, 64, 16)
    for apart in (False, True):
        check(c, run(pa, c, 64, 4, 8, apart), 64, 4, 8, apart)


def test_long_context(pa):
    # more rows than fit in shared memory as keys
    c = make(5, [52000, 700], 1, 64, 32, zeros=0.5)
    check(c, run(pa, c, 5000, 4, 1000, True), 5000, 4, 1000, True)
    check(c, run(pa, c, 49999, 4, 1000, False), 49999, 4, 1000, False)


def test_more_rows_than_keys_held(pa):
    """So many units that each is one CTA, and a context longer than its shared memory."""
    c = make(10, [46000] + [40] * 159, 1, 64, 32, zeros=0.3)
    check(c, run(pa, c, 20000, 4, 1000, True), 20000, 4, 1000, True)
    check(c, run(pa, c, 45997, 4, 1000, False), 45997, 4, 1000, False)


def test_again_with_other_ledgers_gives_the_same(pa):
    c = make(6, [400, 333], 2, 128, 16)
    k, v, so, po, new, (scores, pos, cl, sl, kw) = run(pa, c, 100, 4, 20, True)
    keep = [x.clone() for x in (k, v, so, po, new)]
    pa.pa_evict(k, v, scores, pos, c["table"].to(DEV), cl, sl, 100, 4, 20, **kw)
    for x, y in zip((k, v, so, po), keep):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


def test_bad_blocks_are_skipped(pa):
    c = make(7, [100], 1, 64, 16)
    c["table"][0, 0] = 10 ** 6
    got = run(pa, c, 30, 0, 4, False)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert got[4].tolist() == [30]


def test_context_longer_than_its_table(pa):
    c = make(8, [64], 1, 64, 16, spare=0)
    c["lens"] = [80]
    got = run(pa, c, 30, 0, 4, False)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert got[4].tolist() == [30]


def test_side_stream_and_graph(pa):
    c = make(9, [400, 100], 2, 128, 16)
    want = run(pa, c, 90, 4, 20, True)
    k, v = (c[x].to(DEV).view(torch.bfloat16) for x in ("k", "v"))
    scores, pos, table = c["scores"].to(DEV), c["pos"].to(DEV), c["table"].to(DEV)
    cl = torch.tensor(c["lens"], dtype=torch.int32, device=DEV)
    sl = torch.tensor(c["sl"], dtype=torch.int32, device=DEV)
    so, po, nl = torch.full_like(scores, -7.0), torch.full_like(pos, -7), torch.zeros_like(cl)
    ws = torch.empty(pa.pa_evict_workspace_size(2, 2, 90), dtype=torch.uint8, device=DEV)

    def call():
        pa.pa_evict(k, v, scores, pos, table, cl, sl, 90, 4, 20, scores_out=so, row_pos_out=po,
                    new_lens=nl, workspace=ws)

    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    so.fill_(-7.0)
    nl.zero_()
    graph.replay()
    torch.cuda.synchronize()
    for x, y in zip((k, v, so, po, nl), want):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


@pytest.mark.parametrize("seed", range(12))
def test_random_shapes(pa, seed):
    r = np.random.default_rng(seed)
    nb = int(r.choice([1, 2]))
    lens = [int(x) for x in r.integers(0, 1500, size=int(r.integers(1, 5)))]
    budget = int(r.integers(1, 900))
    sinks = int(r.integers(0, min(5, budget) + 1))
    recent = int(r.integers(0, budget - sinks + 1))
    c = make(seed, lens, int(r.choice([1, 2, 5])), 128 if nb == 1 else int(r.choice([64, 128])),
             int(r.choice([8, 16, 32])), nb)
    apart = bool(r.random() < 0.5)
    check(c, run(pa, c, budget, sinks, recent, apart), budget, sinks, recent, apart)
    assert pa.pa_device_error() == 0
