"""Whole serving steps over a block-scaled pool, against a simulation in 64 bits: blocks
reserved, rows appended, attention, the logits' probabilities, drafts verified, rejected
rows' blocks freed, a sequence forked, the pool compacted; the same from a CUDA graph, on a
stream that the call names, and from two streams at once."""
import numpy as np
import pytest
import torch

from tests import _ops_ref, _pool_ref as ref
from tests.test_gpu_block_scaled import bound, f64, values
from tests.test_gpu_named_stream import meanwhile
from tests.test_gpu_pages import i32

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


class Server:
    """n rows of a batch, k drafts a step, one layer."""

    def __init__(self, pa, seed, n, k, bs, h, g, dtype, vocab=1000, width=24):
        self.pa, self.n, self.k, self.bs, self.h, self.g, self.dtype, self.vocab = pa, n, k, bs, h, g, dtype, vocab
        self.rng = np.random.default_rng(seed)
        self.nb = n * width // 2
        self.tables = np.full((n, width), -1, np.int32)
        self.refs = np.zeros(self.nb, np.int32)
        self.kc, self.vc = (np.full((self.nb, h, bs, 128), 127, np.uint8) for _ in range(2))
        self.scales = np.full((self.nb, h, 2), np.nan, np.float32)
        self.lens = np.zeros(n, np.int32)
        self.said = [[] for _ in range(n)]
        self.t, self.r, self.l = i32(self.tables), i32(self.refs), i32(self.lens)
        self.ck, self.cv, self.cs = (torch.from_numpy(x.copy()).to(DEV) for x in (self.kc, self.vc, self.scales))

    def same(self):
        assert np.array_equal(self.t.cpu().numpy(), self.tables)
        assert np.array_equal(self.r.cpu().numpy(), self.refs)
        assert np.array_equal(self.l.cpu().numpy(), self.lens)
        assert np.array_equal(self.cs.cpu().numpy(), self.scales, equal_nan=True)
        assert np.array_equal(self.ck.cpu().numpy(), self.kc) and np.array_equal(self.cv.cpu().numpy(), self.vc)

    def append_and_attend(self, u):
        pa, rng = self.pa, self.rng
        want = self.lens + u
        assert int(pa.pa_reserve_blocks(self.t, self.r, i32(want), self.bs)) == 0
        assert ref.reserve(self.tables, self.refs, want, self.bs) == 0
        self.lens, self.l = want.astype(np.int32), i32(want)
        k_new, v_new = (values(rng, (self.n * u, self.h, 128), self.dtype, 2.0 ** rng.integers(-3, 3)) for _ in range(2))
        pa.pa_append_kv_block_scaled(self.ck, self.cv, self.cs, k_new.to(DEV), v_new.to(DEV), self.t, self.l, q_len=u)
        ref.append(self.kc, self.vc, self.scales, f64(k_new), f64(v_new), self.tables, self.lens, u)
        q = values(rng, (self.n, u, self.h * self.g * 128), self.dtype, 0.1).view(self.n, u, -1, 128)
        out = torch.empty_like(q, device=DEV)
        pa.pa_decode_block_scaled(out, q.to(DEV), self.ck, self.cv, self.cs, self.t, self.l, 0.09, q_len=u)
        o, wv, mags = ref.attend(f64(q), self.kc, self.vc, self.scales, self.tables, self.lens, 0.09)
        assert (np.abs(f64(out) - o) <= bound(wv, mags, int(self.lens.max()), o, self.dtype)).all()
        self.same()

    def decode(self):
        pa, rng, n, k, v = self.pa, self.rng, self.n, self.k, self.vocab
        self.append_and_attend(1 + k)
        logits = torch.from_numpy(rng.standard_normal((n, k + 1, v)) * 3).to(torch.bfloat16)
        drafts = rng.integers(0, v, (n, k))
        longest = max(1, max(map(len, self.said)))
        hist = np.full((n, longest), -1)
        for i, s in enumerate(self.said):
            hist[i, :len(s)] = s
        hl = [len(s) for s in self.said]
        rep, pres = 1 + 0.3 * rng.random(n, np.float32), 0.5 * rng.random(n, np.float32)
        freq, temp = 0.5 * rng.random(n, np.float32), 0.5 + rng.random(n, np.float32)
        fl = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
        p = pa.pa_adjust_logits(None, logits.to(DEV), history=i32(hist), history_lens=i32(hl), drafts=i32(drafts),
                                repetition=fl(rep), presence=fl(pres), frequency=fl(freq), temperature=fl(temp), probs=True)
        for i in range(n):
            for j in range(k + 1):
                y = ref.adjusted(logits[i, j].float().numpy(), np.array(self.said[i]), 0, drafts[i, :j], rep[i], pres[i],
                                 freq[i], [], None)
                w = ref.probabilities(y, temp[i])
                # (the bound of test_gpu_logits, where |log2 p| < 128)
                assert (np.abs(p[i, j].cpu().double().numpy() - w) <= w * 2.0 ** -14 + 2.0 ** -126).all()
        # the drafter is sure of its tokens; the middle ones are certain to stand
        u = rng.random((n, k)).astype(np.float32)
        u[:, :k // 2] = 0
        su = rng.random(n).astype(np.float32)
        tok, acc, new = pa.pa_verify_drafts(p, None, i32(drafts), fl(u), fl(su), context_lens=self.l)
        wt, wa = _ops_ref.verify(p.cpu().double().numpy(), None, drafts, [k] * n, u.astype(np.float64), su.astype(np.float64))
        assert np.array_equal(acc.cpu().numpy(), wa) and np.array_equal(tok.cpu().numpy(), wt)
        pa.pa_free_blocks(self.t, self.r, new, self.bs)
        self.lens = (self.lens - (k - wa)).astype(np.int32)
        ref.free(self.tables, self.refs, self.lens, self.bs)
        self.l = new
        for i in range(n):
            self.said[i] += wt[i, :wa[i] + 1].tolist()
        self.same()

    def fork(self, src, dst):
        pa = self.pa
        keep = self.lens.copy()
        keep[dst] = 0
        pa.pa_free_blocks(self.t, self.r, i32(keep), self.bs)
        ref.free(self.tables, self.refs, keep, self.bs)
        sb, db, counts = pa.pa_fork_blocks(self.t, self.l, self.r, i32(src), i32(dst), self.bs)
        pa.pa_copy_pages(self.ck, self.cv, sb, db, counts, kv_scales=self.cs)
        pairs, missing = ref.fork(self.tables, self.lens, self.refs, src, dst, self.bs)
        assert counts.tolist() == [len(pairs), missing]
        self.move(pairs)
        for s, d in zip(src, dst):
            self.said[d] = list(self.said[s])
        self.same()

    def move(self, pairs):
        for a, b in pairs:
            self.kc[b], self.vc[b], self.scales[b] = self.kc[a], self.vc[a], self.scales[a]

    def compact(self):
        sb, db, counts = self.pa.pa_compact_blocks(self.t, self.r)
        self.pa.pa_copy_pages(self.ck, self.cv, sb, db, counts, kv_scales=self.cs)
        self.tables, self.refs, pairs, live = ref.compact(self.tables, self.refs)
        assert counts.tolist() == [len(pairs), live]
        self.move(pairs)
        self.same()


@pytest.mark.parametrize("bs,h,g,k,dtype", [(16, 2, 4, 3, "bf16"), (8, 1, 1, 2, "fp16"), (32, 2, 8, 1, "bf16")])
def test_serving_steps(pa, bs, h, g, k, dtype):
    s = Server(pa, bs, 5, k, bs, h, g, dtype)
    s.append_and_attend(37)
    for _ in range(3):
        s.decode()
    s.fork([0, 2], [3, 1])
    s.decode()
    s.compact()
    for _ in range(2):
        s.decode()
    assert pa.pa_device_error() == 0


def made(seed, n=4, h=2, g=4, bs=16, u=1, vocab=5000, width=12):
    """A batch in the middle of its sequences, everything preallocated."""
    rng = np.random.default_rng(seed)
    nb = n * width
    d = dict(tables=np.full((n, width), -1), refs=np.zeros(nb), lens=rng.integers(u, width * bs // 2, n))
    d = {a: np.asarray(b, np.int32) for a, b in d.items()}
    ref.reserve(d["tables"], d["refs"], d["lens"] - 1, bs)
    d = {a: i32(b) for a, b in d.items()}
    t = lambda x: torch.from_numpy(x).to(DEV)  # noqa: E731
    d.update(k=t(rng.integers(0, 127, (nb, h, bs, 128)).astype(np.uint8)),
             v=t(rng.integers(0, 127, (nb, h, bs, 128)).astype(np.uint8)),
             s=t((2.0 ** rng.integers(-9, -5, (nb, h, 2))).astype(np.float32)),
             kn=values(rng, (n * u, h, 128), "bf16").to(DEV), vn=values(rng, (n * u, h, 128), "bf16").to(DEV),
             q=values(rng, (n, u, h * g * 128), "bf16", 0.1).view(n, u, -1, 128).to(DEV),
             out=torch.zeros(n, u, h * g, 128, dtype=torch.bfloat16, device=DEV),
             x=torch.from_numpy(rng.standard_normal((n, u, vocab)).astype(np.float32)).to(DEV),
             p=torch.zeros(n, u, vocab, device=DEV), hist=i32(rng.integers(0, vocab, (n, 50))), hl=i32([50] * n),
             rep=torch.full((n,), 1.2, device=DEV), miss=i32([0]), pairs=i32(np.zeros((2, nb // 2))), counts=i32([0, 0]),
             ws=torch.zeros(pa_ws(n, h * g, u, nb), dtype=torch.uint8, device=DEV))
    return d, bs, u


def pa_ws(n, hq, u, nb):
    import paged_kv_cache_20_gb300 as pa
    return max(pa.pa_decode_workspace_size(n, hq, u, 128, 3), pa.pa_pages_workspace_size(nb, n))


def step(pa, d, bs, u, **kw):
    own = {} if kw else dict(workspace=d["ws"])
    pa.pa_reserve_blocks(d["tables"], d["refs"], d["lens"], bs, missing=d["miss"], **own, **kw)
    pa.pa_append_kv_block_scaled(d["k"], d["v"], d["s"], d["kn"], d["vn"], d["tables"], d["lens"], q_len=u, **kw)
    pa.pa_decode_block_scaled(d["out"], d["q"], d["k"], d["v"], d["s"], d["tables"], d["lens"], 0.09, q_len=u,
                              num_splits=3, **own, **kw)
    pa.pa_adjust_logits(d["p"], d["x"], history=d["hist"], history_lens=d["hl"], repetition=d["rep"], probs=True, **kw)
    pa.pa_compact_blocks(d["tables"], d["refs"], src_blocks=d["pairs"][0], dst_blocks=d["pairs"][1], counts=d["counts"],
                         **own, **kw)
    pa.pa_copy_pages(d["k"], d["v"], d["pairs"][0], d["pairs"][1], d["counts"], kv_scales=d["s"], **kw)
    pa.pa_free_blocks(d["tables"], d["refs"], d["hl"], bs, **kw)


STATE = ("tables", "refs", "k", "v", "s", "out", "p", "miss", "counts")


@pytest.mark.parametrize("u", [1, 3, 24])
def test_a_captured_step(pa, u):
    want, bs, _ = made(u, u=u)
    step(pa, want, bs, u)
    got, _, _ = made(u, u=u)
    keep = {a: b.clone() for a, b in got.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(pa, got, bs, u)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(pa, got, bs, u)
    for _ in range(3):
        for a in keep:
            got[a].copy_(keep[a])
        graph.replay()
        torch.cuda.synchronize()
        for a in STATE:
            assert torch.equal(got[a], want[a]), a
    assert pa.pa_device_error() == 0


def test_two_captured_steps_at_once(pa):
    """Two graphs with workspaces of their own, replayed on two streams."""
    both = []
    for seed in (5, 6):
        want, bs, u = made(seed)
        step(pa, want, bs, u)
        got, _, _ = made(seed)
        keep = {a: b.clone() for a, b in got.items()}
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(pa, got, bs, u)
        both.append((want, got, keep, graph, torch.cuda.Stream()))
    for _ in range(5):
        for want, got, keep, graph, side in both:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for a in keep:
                    got[a].copy_(keep[a])
                graph.replay()
        torch.cuda.synchronize()
        for want, got, *_ in both:
            for a in STATE:
                assert torch.equal(got[a], want[a]), a
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("u", [1, 24])
def test_a_named_stream(pa, u):
    want, bs, _ = made(u, u=u)
    step(pa, want, bs, u)

    def setup():
        return (made(u, u=u)[0],)

    def call(stream, d):
        step(pa, d, bs, u, stream=stream)
        return d

    for got in meanwhile(setup, call):
        for a in STATE:
            assert torch.equal(got[a], want[a]), a
    assert pa.pa_device_error() == 0


def test_without_the_compiled_calls(pa):
    """The binding's own checks and calls, which take over where the compiled ones do not."""
    want, bs, u = made(9)
    step(pa, want, bs, u)
    got, _, _ = made(9)
    fast, pa._fast = pa._fast, None
    try:
        step(pa, got, bs, u)
    finally:
        pa._fast = fast
    for a in STATE:
        assert torch.equal(got[a], want[a]), a


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_rotated_heads_of_one_projection(pa, dtype):
    """q and k heads of a fused projection's output rotated in place, without cache rows, then
    k and v appended from their slices: as q, k and v apart."""
    g = torch.Generator(device=DEV).manual_seed(3)
    n, u, hq, h, bs = 3, 5, 8, 2, 16
    t = n * u
    qkv = torch.randn(t, hq + 2 * h, 128, generator=g, device=DEV).to(dtype)
    pos = torch.randint(0, 10000, (1, t), generator=g, device=DEV, dtype=torch.int32)
    turns, axis = pa.rope_table(128)
    nowhere = torch.full((t,), -1, dtype=torch.int64, device=DEV)
    ones = torch.ones(h, device=DEV)
    codes = [torch.zeros(12, h, bs, 128, dtype=torch.uint8, device=DEV) for _ in range(4)]
    scales = [torch.zeros(12, h, 2, device=DEV) for _ in range(2)]
    tables, lens = i32(np.arange(12).reshape(3, 4)), i32([5, 20, 37])
    apart = [x.contiguous() for x in (qkv[:, :hq], qkv[:, hq:hq + h], qkv[:, hq + h:])]
    for x in apart[:2]:
        pa.pa_rope_append(x, x, apart[1], apart[2], codes[0], codes[1], pos, nowhere, turns, axis, k_scale=ones,
                          v_scale=ones)
    pa.pa_append_kv_block_scaled(codes[0], codes[1], scales[0], apart[1], apart[2], tables, lens, q_len=u)
    qk, k, v = qkv[:, :hq + h], qkv[:, hq:hq + h], qkv[:, hq + h:]
    pa.pa_rope_append(qk, qk, k, v, codes[2], codes[3], pos, nowhere, turns, axis, k_scale=ones, v_scale=ones)
    pa.pa_append_kv_block_scaled(codes[2], codes[3], scales[1], k, v, tables, lens, q_len=u)
    assert torch.equal(qkv[:, :hq], apart[0])
    assert torch.equal(codes[0], codes[2]) and torch.equal(codes[1], codes[3]) and torch.equal(scales[0], scales[1])
    assert bool((codes[0] != 0).any()) and pa.pa_device_error() == 0
