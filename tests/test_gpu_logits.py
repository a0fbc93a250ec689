"""Adjusted logits and their probabilities on the GPU against the definition: logits bit for
bit (each operation is rounded to fp32), probabilities against 64 bits."""
import math

import numpy as np
import pytest
import torch

from tests import _pool_ref as ref

pytestmark = pytest.mark.gpu
DEV = "cuda"
DT = {"fp16": torch.float16, "bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module")
def pa():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import paged_kv_cache_20_gb300 as pa
    pa.load()
    assert pa.pa_device_error() == 0
    return pa


def f32(x):
    return torch.as_tensor(np.asarray(x, np.float32)).to(DEV)


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(np.asarray(x, np.int32))).to(DEV)


def packed(allowed):
    """bool [.., v] -> int32 words."""
    v = allowed.shape[-1]
    pad = np.zeros(allowed.shape[:-1] + (-v % 32,), bool)
    bits = np.concatenate((allowed, pad), -1).reshape(allowed.shape[:-1] + (-1, 32))
    return (bits.astype(np.uint64) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32).view(np.int32)


class Case:
    def __init__(self, rng, n, r, v, dtype, hist, bias, masked):
        self.n, self.r, self.v, self.dtype = n, r, v, dtype
        self.x = torch.from_numpy(rng.standard_normal((n, r, v)) * 3).to(DT[dtype])
        self.hist = rng.integers(-1, v, (n, hist)) if hist else None
        if hist:
            self.hist[rng.random((n, hist)) < 0.5] = rng.integers(0, min(v, 5))
            self.hl = rng.integers(0, hist + 1, n)
            self.hl[0] = hist
            self.pl = (self.hl * rng.random(n)).astype(np.int64)
        self.drafts = rng.integers(-1, min(v, 40), (n, r - 1)) if r > 1 else None
        self.rep, self.pres = 1 + rng.random(n), rng.random(n) - 0.3
        self.freq, self.temp = rng.random(n), 0.2 + 2 * rng.random(n)
        self.bias = None
        if bias:
            ids = rng.integers(-1, v, (n, bias))
            ids[:, bias // 2:] = ids[:, :bias - bias // 2]  # one token several times
            self.bias = ids, rng.standard_normal((n, bias)) * 5
        self.allowed = rng.random((n, r, v)) < rng.random((n, r, 1)) if masked else None

    def args(self):
        a = dict(repetition=f32(self.rep), presence=f32(self.pres), frequency=f32(self.freq))
        if self.hist is not None:
            a.update(history=i32(self.hist), history_lens=i32(self.hl), prompt_lens=i32(self.pl))
        if self.drafts is not None:
            a["drafts"] = i32(self.drafts)
        if self.bias is not None:
            a.update(bias_ids=i32(self.bias[0]), bias_values=f32(self.bias[1]))
        if self.allowed is not None:
            a["mask"] = i32(packed(self.allowed))
        return a

    def adjusted(self, i, j):
        f = np.float32
        h = [] if self.hist is None else self.hist[i, :self.hl[i]]
        return ref.adjusted(self.x[i, j].to(torch.float32).numpy(), h, 0 if self.hist is None else int(self.pl[i]),
                            [] if self.drafts is None else self.drafts[i, :j], f(self.rep[i]), f(self.pres[i]),
                            f(self.freq[i]), [] if self.bias is None else list(zip(*(b[i] for b in self.bias))),
                            None if self.allowed is None else self.allowed[i, j])

    def check_probs(self, got, temp):
        """exp2's argument: a difference, its factor (two roundings) and the product, each
        half a step of fp32 of itself, 2^-22 of |z| together; exp2 twice and the sum of
        up to 72 + 5 + 4 + 5 chained terms: 2^-17 covers both."""
        got = got.cpu().double().numpy()
        for i in range(self.n):
            for j in range(self.r):
                y = self.adjusted(i, j)
                want = ref.probabilities(y, np.float32(temp[i]))
                with np.errstate(divide="ignore"):
                    z = np.abs(np.log2(np.maximum(want, 1e-40)))
                over = np.abs(got[i, j] - want) - want * (2.0 ** -17 + z * 2.0 ** -22) - 2.0 ** -126
                assert over.max() <= 0, (i, j, int(over.argmax()), over.max())
                if not temp[i] > 0:
                    assert np.array_equal(got[i, j], want)


CASES = [(1, 1, 1, "fp32", 1, 1, False), (3, 2, 7, "fp16", 5, 0, True), (2, 1, 32, "bf16", 0, 2, True),
         (2, 3, 33, "fp32", 9, 4, True), (4, 1, 1000, "bf16", 300, 0, False), (3, 4, 4097, "fp16", 100, 40, True),
         (1, 1, 32000, "fp16", 700, 4, False), (2, 9, 32001, "bf16", 5000, 300, True),
         (2, 2, 131071, "bf16", 4096, 1024, True), (1, 2, 131071, "fp32", 64, 3, True),
         (1, 1, 262144, "fp16", 10, 0, True), (1, 2, 262143, "fp32", 10, 7, False), (200, 2, 777, "fp16", 3, 1, True),
         (300, 1, 20000, "bf16", 50, 0, False), (3, 21, 40001, "bf16", 40, 6, True), (40, 19, 3001, "fp32", 30, 3, True),
         (70, 17, 131070, "fp16", 100, 5, False)]


@pytest.mark.parametrize("n,r,v,dtype,hist,bias,masked", CASES)
def test_logits(pa, n, r, v, dtype, hist, bias, masked):
    c = Case(np.random.default_rng(v + n), n, r, v, dtype, hist, bias, masked)
    x = c.x.to(DEV)
    out = torch.full_like(x, math.nan)
    assert pa.pa_adjust_logits(out, x, **c.args()) is out
    again = x.clone()
    pa.pa_adjust_logits(again, again, **c.args())  # in place
    got = out.cpu()
    for i in range(n):
        for j in range(r):
            want = torch.from_numpy(c.adjusted(i, j)).to(DT[dtype])
            assert torch.equal(got[i, j], want), (i, j)
    assert torch.equal(again, out)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("n,r,v,dtype,hist,bias,masked", CASES)
def test_probabilities(pa, n, r, v, dtype, hist, bias, masked):
    c = Case(np.random.default_rng(v + n + 1), n, r, v, dtype, hist, bias, masked)
    c.temp[::3] = 0
    out = pa.pa_adjust_logits(None, c.x.to(DEV), temperature=f32(c.temp), probs=True, **c.args())
    assert out.dtype == torch.float32
    c.check_probs(out, c.temp.astype(np.float32))
    if dtype == "fp32":
        x = c.x.to(DEV)
        pa.pa_adjust_logits(x, x, temperature=f32(c.temp), probs=True, **c.args())
        assert torch.equal(x, out)
    assert pa.pa_device_error() == 0


def test_nothing_given(pa):
    x = torch.randn(3, 2, 1001, device=DEV)
    assert torch.equal(pa.pa_adjust_logits(None, x), x)
    p = pa.pa_adjust_logits(None, x, probs=True)
    # (the bound of check_probs at |z| < 30)
    assert float((p.double() / x.double().softmax(-1) - 1).abs().max()) < 2.0 ** -16


@pytest.mark.parametrize("v", [5, 40000])
def test_rows_that_the_mask_leaves_empty(pa, v):
    x = torch.randn(4, 1, v, device=DEV)
    x[0] = math.nan
    x[1] = math.inf
    allowed = np.zeros((4, 1, v), bool)
    allowed[3, 0, v - 1] = True
    for temp in (1.0, 0.0):
        p = pa.pa_adjust_logits(None, x, mask=i32(packed(allowed)), temperature=f32([temp] * 4), probs=True)
        assert bool((p[:3] == 0).all()) and bool((p[3, 0, :v - 1] == 0).all()) and float(p[3, 0, v - 1]) == 1.0
    y = pa.pa_adjust_logits(None, x, mask=i32(packed(allowed)))
    assert bool((y[:3] == -math.inf).all()) and float(y[3, 0, v - 1]) == float(x[3, 0, v - 1])


@pytest.mark.parametrize("v", [9, 50001])
def test_special_logits(pa, v):
    """NaN counts as -inf, infinite entries share the whole; one at the lowest of equals."""
    x = torch.full((5, 1, v), -2.0, device=DEV)
    x[0, 0, 3], x[0, 0, 5] = math.nan, 1.0
    x[1, 0, 2], x[1, 0, v - 1] = math.inf, math.inf
    x[2] = -math.inf
    x[3, 0, v // 2], x[3, 0, v - 1] = 4.0, 4.0
    x[4] = torch.finfo(torch.float32).min
    p = pa.pa_adjust_logits(None, x, probs=True).cpu()
    assert float(p[0, 0, 3]) == 0 and bool(torch.isfinite(p).all())
    assert p[1, 0, 2] == 0.5 and p[1, 0, v - 1] == 0.5
    assert bool((p[2] == 0).all())
    assert bool(((p[4] * v - 1).abs() < 2.0 ** -17).all())
    # an infinite entry beside counted ones, in 16 bits too
    for dt in (torch.float16, torch.float32):
        q = pa.pa_adjust_logits(None, x.to(dt), history=i32([[2, 3, v - 1]] * 5), history_lens=i32([3] * 5),
                                frequency=f32([0.5] * 5), probs=True).cpu()
        assert q[1, 0, 2] == 0.5 and q[1, 0, v - 1] == 0.5 and float(q[1].sum()) == 1
    for t in (0.0, -1.0, math.nan):
        g = pa.pa_adjust_logits(None, x, temperature=f32([t] * 5), probs=True).cpu()
        assert [int(g[i, 0].argmax()) for i in (0, 1, 3, 4)] == [5, 2, v // 2, 0]
        assert [float(g[i].sum()) for i in range(5)] == [1, 1, 0, 1, 1]


@pytest.mark.parametrize("temp", [1e-42, 1e-30, 1e30, math.inf])
def test_far_temperatures(pa, temp):
    x = torch.randn(1, 1, 3000, device=DEV)
    x[0, 0, 7] = 9.0
    allowed = np.ones((1, 1, 3000), bool)
    allowed[0, 0, 100:200] = False
    p = pa.pa_adjust_logits(None, x, mask=i32(packed(allowed)), temperature=f32([temp]), probs=True).cpu()
    if temp < 1:
        assert p[0, 0, 7] == 1 and float(p.sum()) == 1
    else:
        assert bool(((p[0, 0, :100] * 2900 - 1).abs() < 2.0 ** -17).all()) and bool((p[0, 0, 100:200] == 0).all())


def test_rows_apart(pa):
    """Padded vocabularies, and masks shared by rows or by sequences."""
    rng = np.random.default_rng(0)
    n, r, v = 3, 4, 5003
    wide = torch.randn(n, r, v + 13, device=DEV)
    x = wide[:, :, :v]
    room = torch.full((n, r, v + 5), 7.0, device=DEV)
    allowed = rng.random((n, r, v)) < 0.5
    for shape in ((n, 1), (1, r), (1, 1)):
        m = i32(packed(allowed[:shape[0], :shape[1]])).expand(n, r, -1)
        pa.pa_adjust_logits(room[:, :, :v], x, mask=m)
        want = np.broadcast_to(allowed[:shape[0], :shape[1]], (n, r, v))
        assert torch.equal(room[:, :, :v].cpu(), x.cpu().masked_fill(torch.from_numpy(~want), -math.inf))
        assert bool((room[:, :, v:] == 7).all())
    for dt in (torch.float16, torch.bfloat16):  # 16-bit rows that start at odd elements
        p = pa.pa_adjust_logits(None, wide.to(dt)[:, :, 1:v + 1], probs=True)
        want = wide.to(dt)[:, :, 1:v + 1].double().softmax(-1)
        assert float((p.double() / want - 1).abs().max()) < 2.0 ** -16


@pytest.mark.parametrize("hist,v", [(16383, 40000), (16384, 40000), (40000, 9000), (70000, 262144)])
def test_long_histories(pa, hist, v):
    """Counts that pass 14 and 16 bits, every entry of a slice counted."""
    rng = np.random.default_rng(hist)
    c = Case(rng, 2, 3, v, "bf16", hist, 5, True)
    c.hist[0, :hist // 2] = 7
    c.hist[1] = np.arange(hist) % v
    c.hl[:], c.pl[:] = hist, (0, hist // 3)
    x = c.x.to(DEV)
    got = pa.pa_adjust_logits(None, x, **c.args()).cpu()
    for i in range(2):
        for j in range(3):
            assert torch.equal(got[i, j], torch.from_numpy(c.adjusted(i, j)).to(torch.bfloat16))
    c.check_probs(pa.pa_adjust_logits(None, x, temperature=f32(c.temp), probs=True, **c.args()), c.temp.astype(np.float32))
    assert pa.pa_device_error() == 0


def test_drafts_on_the_list_and_off_it(pa):
    """The same token drafted again and again, one of the history, one of the biases; more
    rows than are summed at once."""
    rng = np.random.default_rng(8)
    c = Case(rng, 3, 27, 33000, "fp16", 20, 4, False)
    c.drafts[0] = 32999
    c.drafts[1] = [c.hist[1, 0], 5, 5, -1, 5, c.bias[0][1, 0], 0, 5, 32998, 32998, 7, 32998, 32999] * 2
    c.drafts[2] = [0, 1, 2, 3, 31, 32, 33, 3, 2, 1, 0, 0, 16000] * 2
    out = pa.pa_adjust_logits(None, c.x.to(DEV), **c.args()).cpu()
    for i in range(3):
        for j in range(27):
            assert torch.equal(out[i, j], torch.from_numpy(c.adjusted(i, j)).to(torch.float16)), (i, j)
    # (a batch of its own for each sequence, and several sequences' rows in one thread block)
    for n in (3, 300):
        x = c.x.repeat(n // 3, 1, 1).to(DEV)
        args = {k: v.repeat(*([n // 3] + [1] * (v.dim() - 1))) for k, v in c.args().items()}
        p = pa.pa_adjust_logits(None, x, temperature=f32(np.tile(c.temp, n // 3)), probs=True, **args)
        c.check_probs(p[:3], c.temp.astype(np.float32))
        c.check_probs(p[n - 3:], c.temp.astype(np.float32))


def test_ids_outside_the_vocabulary(pa):
    x = torch.ones(1, 2, 10, device=DEV)
    clean = dict(history=i32([[3, -1, -7]]), history_lens=i32([3]), drafts=i32([[-1]]),
                 bias_ids=i32([[-1, 2]]), bias_values=f32([[5.0, 1.0]]), repetition=f32([2.0]))
    y = pa.pa_adjust_logits(None, x, **clean).cpu()
    assert pa.pa_device_error() == 0
    assert y[0, 0].tolist() == [1, 1, 2, 0.5] + [1] * 6
    for kw in (dict(history=i32([[3, 10, -7]])), dict(bias_ids=i32([[10, 2]])), dict(history_lens=i32([4])),
               dict(history_lens=i32([-1]), history=i32([[-1, -1, -1]]))):
        pa.pa_adjust_logits(None, x, **{**clean, **kw})
        assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK, kw


@pytest.mark.parametrize("probs", [False, True])
@pytest.mark.parametrize("n", [1, 700])   # rows of their own thread blocks, and all rows in one
@pytest.mark.parametrize("at", [0, 1, 3])
def test_drafts_outside_the_vocabulary(pa, n, probs, at):
    x = torch.ones(n, 5, 10, device=DEV)
    drafts = torch.full((n, 4), 9, dtype=torch.int32, device=DEV)
    pa.pa_adjust_logits(None, x, drafts=drafts, probs=probs)
    assert pa.pa_device_error() == 0
    drafts[n - 1, at] = 10
    pa.pa_adjust_logits(None, x, drafts=drafts, probs=probs)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
