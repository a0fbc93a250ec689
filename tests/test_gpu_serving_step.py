"""The operators as a serving loop uses them: rotary append, scored attention, draft
verification, rollback and eviction, step after step, against a 64-bit simulation that
follows the same choices (needs a GPU)."""
import numpy as np
import pytest
import torch

from tests import _ops_ref as ref
from tests import _tol

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


@pytest.mark.parametrize("fp8", [False, True])
def test_prompt_then_drafts_under_a_budget(pa, fp8):
    n, hq, hkv, d, bs, vocab, drafts = 3, 8, 2, 128, 16, 50, 3
    budget, sinks, recent = 48, 2, 16
    g = torch.Generator().manual_seed(4)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16)  # noqa: E731
    width = 10
    tables = torch.randperm(n * width + 2, generator=g)[:n * width].view(n, width).to(torch.int32).to(DEV)
    shape = (n * width + 2, hkv, bs, d)
    if fp8:
        k_cache, v_cache = (torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2))
        ks = torch.full((hkv,), 0.03, device=DEV)
        vs = torch.tensor([0.02, 0.04], device=DEV)
    else:
        k_cache, v_cache = (torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV)
                            for _ in range(2))
        ks = vs = None
    scores = torch.full((n, hkv, width * bs), 9.0, device=DEV)
    row_pos = torch.full((n, hkv, width * bs), -1, dtype=torch.int32, device=DEV)
    turns, axis = pa.rope_table(d, sections=(32, 16, 16), device=DEV)
    inv_freq = [10000.0 ** (-i / 64) for i in range(64)]
    ctx = torch.zeros(n, dtype=torch.int32, device=DEV)    # cached rows
    seen = torch.zeros(n, dtype=torch.int32, device=DEV)   # tokens of the sequence
    truth = [[] for _ in range(n)]  # the rotated K of every position, for the whole test
    for step in range(12):
        u = 37 if step == 0 else 1 + drafts
        ctx += u
        seen += u
        q, k, v = rnd(n * u, hq, d).to(DEV), rnd(n * u, hkv, d).to(DEV), rnd(n * u, hkv, d).to(DEV)
        # positions: the token's place in its sequence on each axis (not its cache row)
        place = (seen[:, None] - u + torch.arange(u, device=DEV)).reshape(-1).to(torch.int32)
        pos = torch.stack((place, place // 2, place % 7)).to(torch.int32)
        slots = pa.pa_slot_mapping(tables, ctx, bs, u)
        pa.pa_rope_append(q, q, k, v, k_cache, v_cache, pos, slots, turns, axis, k_scale=ks, v_scale=vs)
        qs = q.view(n, u, hq, d)
        out, before = torch.empty_like(qs), scores.clone()
        splits = 1 + step % 3
        pa.pa_decode_scored(out, scores, qs, k_cache, v_cache, tables, ctx, d ** -0.5, q_len=u,
                            num_splits=splits, row_pos=row_pos, seq_lens=seen, k_scale=ks, v_scale=vs)
        torch.cuda.synchronize()
        # attention and ledger against 64 bits on the cache as it is
        if fp8:
            kc, vc = (ref.e4m3_values(x.cpu()) * ref.f64(s)[:, None, None]
                      for x, s in ((k_cache, ks), (v_cache, vs)))
        else:
            kc, vc = ref.f64(k_cache), ref.f64(v_cache)
        want, ledger, _, _ = ref.scored(ref.f64(qs), kc, vc, tables.cpu().numpy(), ctx.tolist(),
                                        d ** -0.5, ref.f64(before))
        _tol.check(ref.f64(out), want, "bf16", f"step {step}")
        # a weight's bound as derived in the tests of pa_decode_scored is below 1.5e-4
        assert np.allclose(ref.f64(scores), ledger, rtol=2e-4, atol=1e-6), step
        # every cached row holds the rotated K of the position its ledger names
        rotated = ref.rope(ref.f64(k), pos.cpu().numpy(), inv_freq, axis.cpu().numpy(), False)
        rotated = rotated.reshape(n, u, hkv, d)
        for i in range(n):
            truth[i] = truth[i][:int(seen[i]) - u] + list(rotated[i])
            rows = ref.rows_of(kc, tables[i].cpu().numpy(), int(ctx[i]))
            for h in range(hkv):
                at = row_pos[i, h, :int(ctx[i])].tolist()
                assert len(set(at)) == len(at) and 0 <= min(at) and max(at) == int(seen[i]) - 1
                expect = np.array([truth[i][p][h] for p in at])
                # one rounding: bf16 2^-8 of the value, e4m3 2^-4 (2^-10 scaled among
                # its subnormals); rotation error below 2e-6
                lim = (2.0 ** -4 * np.abs(expect) + 2.0 ** -10 * 0.03 if fp8
                       else 2.0 ** -8 * np.abs(expect)) + 1e-5
                assert (np.abs(rows[h] - expect) <= lim).all()
        if step:
            p = torch.softmax(torch.randn(n, drafts + 1, vocab, generator=g), -1)
            dq = torch.softmax(torch.randn(n, drafts, vocab, generator=g), -1)
            x = torch.randint(0, vocab, (n, drafts), generator=g, dtype=torch.int32)
            au, su = torch.rand(n, drafts, generator=g), torch.rand(n, generator=g)
            toks, acc, new = pa.pa_verify_drafts(p.to(DEV), dq.to(DEV), x.to(DEV), au.to(DEV),
                                                 su.to(DEV), context_lens=ctx)
            w = ref.verify(ref.f64(p), ref.f64(dq), x.numpy(), [drafts] * n, ref.f64(au), ref.f64(su))
            assert np.array_equal(toks.cpu().numpy(), w[0]) and np.array_equal(acc.cpu().numpy(), w[1])
            assert torch.equal(new, ctx - (drafts - acc))
            seen -= drafts - acc
            ctx = new
        was = {"s": ref.f64(scores), "p": row_pos.cpu().numpy().copy(), "l": ctx.cpu().numpy(),
               "k": ref.f64(k_cache.view(torch.uint8)), "v": ref.f64(v_cache.view(torch.uint8))}
        ctx = pa.pa_evict(k_cache, v_cache, scores, row_pos, tables, ctx, seen, budget, sinks, recent)
        torch.cuda.synchronize()
        w = ref.evict(was["k"], was["v"], was["s"], was["p"], tables.cpu().numpy(), was["l"],
                      seen.cpu().numpy(), budget, sinks, recent)
        assert np.array_equal(ctx.cpu().numpy(), w[4])
        for i in range(n):
            L = int(ctx[i])
            assert np.array_equal(row_pos[i, :, :L].cpu().numpy(), w[3][i, :, :L])
            assert np.array_equal(ref.f64(scores)[i, :, :L], w[2][i, :, :L])
        assert np.array_equal(ref.f64(k_cache.view(torch.uint8)), w[0])
        assert np.array_equal(ref.f64(v_cache.view(torch.uint8)), w[1])
        assert pa.pa_device_error() == 0
    assert ctx.max().item() == budget and seen.min().item() > budget


def test_step_captured_in_a_graph(pa):
    """One whole step (append, scored attention, eviction, verification) replayed from a
    CUDA graph gives the eager step's bits."""
    n, hq, hkv, d, bs, u = 2, 8, 2, 64, 16, 2
    g = torch.Generator().manual_seed(8)
    rnd = lambda *s: torch.randn(*s, generator=g).to(torch.float16).to(DEV)  # noqa: E731
    tables = torch.randperm(14, generator=g)[:12].view(n, 6).to(torch.int32).to(DEV)
    q, k, v = rnd(n * u, hq, d), rnd(n * u, hkv, d), rnd(n * u, hkv, d)
    p = torch.softmax(torch.randn(n, u, 40, generator=g), -1).to(DEV)
    x = torch.randint(0, 40, (n, u - 1), generator=g, dtype=torch.int32).to(DEV)
    au, su = torch.rand(n, u - 1, generator=g).to(DEV), torch.rand(n, generator=g).to(DEV)
    turns, axis = pa.rope_table(d, device=DEV)
    ctx = torch.tensor([70, 51], dtype=torch.int32, device=DEV)
    seen = ctx + 30
    pos = (seen[:, None] - u + torch.arange(u, device=DEV)).reshape(1, -1).to(torch.int32)
    start = [rnd(14, hkv, bs, d), rnd(14, hkv, bs, d), torch.rand(n, hkv, 96, generator=g).to(DEV),
             torch.arange(96, dtype=torch.int32, device=DEV).repeat(n, hkv, 1) + 30]
    state = [t.clone() for t in start]
    slots = torch.empty(n * u, dtype=torch.int64, device=DEV)
    qr, out = torch.empty_like(q), torch.empty(n, u, hq, d, dtype=q.dtype, device=DEV)
    new = torch.empty_like(ctx)
    toks = torch.empty(n, u, dtype=torch.int32, device=DEV)
    acc = torch.empty_like(ctx)
    ws = torch.empty(pa.pa_decode_scored_workspace_size(n, hq, u, d, 1, 6, bs), dtype=torch.uint8, device=DEV)
    we = torch.empty(pa.pa_evict_workspace_size(n, hkv, 48), dtype=torch.uint8, device=DEV)

    def step():
        kc, vc, sc, rp = state
        pa.pa_slot_mapping(tables, ctx, bs, u, out=slots)
        pa.pa_rope_append(qr, q, k, v, kc, vc, pos, slots, turns, axis)
        pa.pa_decode_scored(out, sc, qr.view(n, u, hq, d), kc, vc, tables, ctx, d ** -0.5, q_len=u,
                            row_pos=rp, seq_lens=seen, workspace=ws)
        pa.pa_evict(kc, vc, sc, rp, tables, ctx, seen, 48, 2, 16, new_lens=new, workspace=we)
        pa.pa_verify_drafts(p, None, x, au, su, out_tokens=toks, num_accepted=acc)

    step()
    want = [t.clone() for t in (*state, out, new, toks, acc)]
    for t, s in zip(state, start):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        for t, s in zip(state, start):
            t.copy_(s)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for got, w in zip((*state, out, new, toks, acc), want):
            assert torch.equal(got, w)
    assert pa.pa_device_error() == 0
