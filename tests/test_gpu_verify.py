"""pa_verify_drafts against the definition in 64 bits: every token equal (needs a GPU)."""
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


def make(seed, n, k, vocab, sharp=2.0, apart=0.7):
    g = torch.Generator().manual_seed(seed)
    logits = sharp * torch.randn(n, k + 1, vocab, generator=g)
    p = torch.softmax(logits, -1)
    q = torch.softmax(logits[:, :k] + apart * torch.randn(n, k, vocab, generator=g), -1)
    race = -torch.rand(n, k, vocab, generator=g).clamp_min(1e-30).log()
    x = (q / race).argmax(-1).to(torch.int32)
    return dict(p=p, q=q, x=x, au=torch.rand(n, k, generator=g), su=torch.rand(n, generator=g))


def both(pa, c, sure=False, given=None, lens=None):
    d = {a: b.to(DEV) for a, b in c.items()}
    dl = None if given is None else torch.tensor(given, dtype=torch.int32, device=DEV)
    cl = None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)
    got = pa.pa_verify_drafts(d["p"], None if sure else d["q"], d["x"], d["au"], d["su"],
                              draft_lens=dl, context_lens=cl)
    torch.cuda.synchronize()
    n, k = c["x"].shape
    want = ref.verify(ref.f64(c["p"]), None if sure else ref.f64(c["q"]), c["x"].numpy(),
                      [k] * n if given is None else given, ref.f64(c["au"]), ref.f64(c["su"]))
    assert np.array_equal(got[1].cpu().numpy(), want[1])
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    return got


@pytest.mark.parametrize("sure", [False, True])
@pytest.mark.parametrize("n,k,vocab", [(1, 1, 1), (1, 1, 2), (3, 2, 31), (2, 5, 33), (5, 3, 257),
                                       (4, 40, 300), (7, 4, 4099), (33, 1, 5000), (2, 3, 50021)])
def test_tokens_equal(pa, n, k, vocab, sure):
    both(pa, make(n * 100 + k, n, k, vocab), sure)
    assert pa.pa_device_error() == 0


def test_many_draws_of_a_flat_distribution(pa):
    # 512 borders searched among 30000 nearly equal weights
    both(pa, make(9, 512, 1, 30000, sharp=0.01, apart=0.02))


def test_ragged_drafts_and_new_lengths(pa):
    given = [0, 1, 4, 3, 2, 4]
    lens = [10, 11, 5, 300, 2, 0]
    got = both(pa, make(3, 6, 4, 97, apart=0.1), given=given, lens=lens)
    acc = got[1].cpu().numpy()
    assert np.array_equal(got[2].cpu().numpy(), np.maximum(0, np.array(lens) - (4 - acc)))
    assert (acc <= given).all()


def test_borders_are_strict(pa):
    # exact in fp32: 8 equal weights; a uniform on a border takes the next token
    n, v = 8, 8
    p = torch.full((n, 2, v), 0.125)
    q = torch.full((n, 1, v), 0.25)  # u q < p: 0.5 * 0.25 == 0.125 is not accepted
    q[:, :, 4:] = 0.0
    c = dict(p=p, q=q, x=torch.zeros(n, 1, dtype=torch.int32), au=torch.full((n, 1), 0.5),
             su=torch.arange(n) / 8.0)
    got = both(pa, c)
    assert got[1].sum().item() == 0
    # residual: tokens 4..7, 0.125 each
    assert got[0][:, 0].tolist() == [4, 4, 5, 5, 6, 6, 7, 7]
    c["au"] = torch.full((n, 1), 0.49999997)
    got = both(pa, c)
    assert got[1].tolist() == [1] * n and got[0][:, 1].tolist() == list(range(8))


def test_equal_distributions_sample_the_target(pa):
    c = make(5, 4, 2, 500, apart=0.0)
    c["q"] = c["p"][:, :2].clone()
    c["au"] = torch.ones(4, 2)  # u = 1: never accepted, and no residual
    both(pa, c)


def test_odd_entries_count_as_zero(pa):
    c = make(6, 3, 2, 100)
    c["p"][0, :, 3] = float("nan")
    c["p"][1, :, 5] = -1.0
    c["p"][2, :, 7] = float("inf")
    c["q"][0, :, 9] = float("nan")
    c["x"][:] = 50
    both(pa, c)
    assert pa.pa_device_error() == 0


def test_bad_ids_lengths_and_empty_rows_are_reported(pa):
    c = make(7, 3, 2, 64)
    c["x"][0, 0], c["x"][1, 1] = 64, -1
    both(pa, c)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    both(pa, c, sure=True)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    c = make(8, 2, 2, 64)
    c["p"][1] = 0.0
    got = both(pa, c)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK and got[0][1].tolist() == [-1, -1, -1]
    c = make(8, 2, 2, 64)
    d = {a: b.to(DEV) for a, b in c.items()}
    lens = torch.tensor([-3, 9], dtype=torch.int32, device=DEV)
    got = pa.pa_verify_drafts(d["p"], d["q"], d["x"], d["au"], d["su"], draft_lens=lens)
    want = ref.verify(ref.f64(c["p"]), ref.f64(c["q"]), c["x"].numpy(), [0, 2], ref.f64(c["au"]),
                      ref.f64(c["su"]))
    assert np.array_equal(got[0].cpu().numpy(), want[0])
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK


def test_padded_vocabulary_rows(pa):
    c = make(10, 3, 3, 130)
    wide_p = torch.full((3, 4, 144), 9.0)
    wide_q = torch.full((3, 3, 136), 9.0)
    wide_p[:, :, :130], wide_q[:, :, :130] = c["p"], c["q"]
    want = both(pa, c)
    wp, wq = wide_p.to(DEV), wide_q.to(DEV)
    got = pa.pa_verify_drafts(wp[:, :, :130], wq[:, :, :130], c["x"].to(DEV), c["au"].to(DEV),
                              c["su"].to(DEV))
    assert torch.equal(got[0], want[0])


def test_distribution_of_the_output(pa):
    # the first output token follows the target's row: 20000 draws over 6 tokens.  A
    # frequency's standard error is at most sqrt(0.25 / 20000) = 0.0035; 5 of them.
    n, v = 20000, 6
    g = torch.Generator().manual_seed(0)
    p = torch.softmax(torch.randn(1, 2, v, generator=g), -1).expand(n, 2, v).contiguous()
    q = torch.softmax(torch.randn(1, 1, v, generator=g), -1).expand(n, 1, v).contiguous()
    x = torch.multinomial(q[:, 0], 1, generator=g).to(torch.int32)
    got = pa.pa_verify_drafts(p.to(DEV), q.to(DEV), x.to(DEV), torch.rand(n, 1, generator=g).to(DEV),
                              torch.rand(n, generator=g).to(DEV))
    freq = torch.bincount(got[0][:, 0].cpu().long(), minlength=v) / n
    assert (freq - p[0, 0]).abs().max() < 0.018


def test_graph_replay(pa):
    c = make(11, 4, 3, 1000)
    d = {a: b.to(DEV) for a, b in c.items()}
    got = pa.pa_verify_drafts(d["p"], d["q"], d["x"], d["au"], d["su"])
    out, acc = torch.zeros_like(got[0]), torch.zeros_like(got[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pa.pa_verify_drafts(d["p"], d["q"], d["x"], d["au"], d["su"], out_tokens=out, num_accepted=acc)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, got[0]) and torch.equal(acc, got[1])
