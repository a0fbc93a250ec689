"""What the binding of the rotary append, scored decode, eviction and draft verification
refuses before a launch, and that a refused call leaves its outputs alone (needs a GPU)."""
import pytest
import torch

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


def z(*shape, dtype=torch.float16, device=DEV):
    return torch.zeros(*shape, dtype=dtype, device=device)


I32, I64, F32 = torch.int32, torch.int64, torch.float32


def rope_args():
    return dict(q_out=z(3, 4, 64), q=z(3, 4, 64), k=z(3, 2, 64), v=z(3, 2, 64), k_cache=z(2, 2, 16, 64),
                v_cache=z(2, 2, 16, 64), positions=z(1, 3, dtype=I32), slot_mapping=z(3, dtype=I64),
                turns=z(32, dtype=I64), pair_axis=z(32, dtype=I32))


@pytest.mark.parametrize("name,value,error", [
    ("q", "cpu", TypeError), ("q", None, TypeError), ("k", z, TypeError), ("q", "bf16", TypeError),
    ("q_out", "shape", ValueError), ("k", "heads", ValueError), ("v_cache", "heads", ValueError),
    ("positions", "short", ValueError), ("slot_mapping", "i32", TypeError), ("turns", "odd", ValueError),
    ("q", "strided heads", ValueError), ("k_scale", "one", ValueError), ("k_cache", "codes", TypeError),
    ("turns", "eight", RuntimeError),
])
def test_rope_append(pa, name, value, error):
    a = rope_args()
    a[name] = {
        "cpu": lambda: a["q"].cpu(), None: lambda: None, z: lambda: 3, "bf16": lambda: a["q"].bfloat16(),
        "shape": lambda: z(3, 4, 32), "heads": lambda: z(*[s + (i == 1) for i, s in enumerate(a[name].shape)]),
        "short": lambda: z(1, 2, dtype=I32), "i32": lambda: z(3, dtype=I32), "odd": lambda: z(32, 1, dtype=I64),
        "strided heads": lambda: z(3, 64, 4).transpose(1, 2), "one": lambda: z(2, dtype=F32),
        "codes": lambda: z(2, 2, 16, 64, dtype=torch.uint8), "eight": lambda: z(8, dtype=I64)[:4],
    }[value]()
    if value == "eight":
        a["pair_axis"] = z(4, dtype=I32)  # rotary_dim 8
    with pytest.raises(error):
        pa.pa_rope_append(**a)
    assert pa.pa_device_error() == 0


def scored_args():
    return dict(out=z(2, 1, 4, 64), scores=z(2, 2, 32, dtype=F32), q=z(2, 1, 4, 64), k_cache=z(4, 2, 16, 64),
                v_cache=z(4, 2, 16, 64), block_tables=z(2, 2, dtype=I32),
                context_lens=z(2, dtype=I32), scale=0.1)


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(q=z(2, 2, 4, 64)), ValueError), (lambda: dict(out=z(2, 1, 4, 32)), ValueError),
    (lambda: dict(scores=z(2, 2, 31, dtype=F32)), ValueError), (lambda: dict(scores=z(2, 2, 32)), TypeError),
    (lambda: dict(row_pos=z(2, 2, 32, dtype=I32)), ValueError), (lambda: dict(seq_lens=z(2, dtype=I32)), ValueError),
    (lambda: dict(context_lens=z(3, dtype=I32)), ValueError), (lambda: dict(block_tables=z(4, dtype=I32)), ValueError),
    (lambda: dict(k_cache=z(4, 2, 16, 64, dtype=torch.bfloat16)), TypeError), (lambda: dict(k_scale=z(2, dtype=F32)), ValueError),
    (lambda: dict(v_cache=z(4, 2, 16, 64).transpose(0, 1).contiguous().transpose(0, 1)), ValueError),
    (lambda: dict(q_len=2), ValueError), (lambda: dict(num_splits=0), RuntimeError),
    (lambda: dict(workspace=z(16, dtype=torch.uint8)), RuntimeError), (lambda: dict(scale=float("nan")), RuntimeError),
    (lambda: dict(out=z(2, 1, 4, 64, device="cpu")), TypeError),
])
def test_decode_scored(pa, kw, error):
    with pytest.raises(error):
        pa.pa_decode_scored(**{**scored_args(), **kw()})
    assert pa.pa_device_error() == 0


def test_decode_scored_takes_three_dimensions(pa):
    a = scored_args()
    a["q"], a["out"] = z(2, 4, 64), torch.ones(2, 4, 64, dtype=torch.float16, device=DEV)
    pa.pa_decode_scored(**a)
    assert (a["out"] == 0).all()  # empty contexts


def evict_args():
    return dict(k_cache=z(4, 2, 16, 64), v_cache=z(4, 2, 16, 64), scores=z(2, 2, 32, dtype=F32),
                row_pos=z(2, 2, 32, dtype=I32), block_tables=z(2, 2, dtype=I32),
                context_lens=z(2, dtype=I32), seq_lens=z(2, dtype=I32), budget=8)


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(scores=z(2, 2, 16, dtype=F32)), ValueError), (lambda: dict(row_pos=z(2, 2, 32, dtype=I64)), TypeError),
    (lambda: dict(scores_out=z(2, 2, 32, dtype=F32)), ValueError), (lambda: dict(seq_lens=z(1, dtype=I32)), ValueError),
    (lambda: dict(budget=0, workspace=z(256)), RuntimeError), (lambda: dict(sinks=5, recent=4), RuntimeError),
    (lambda: dict(k_cache=z(4, 2, 16, 64, dtype=F32), v_cache=z(4, 2, 16, 64, dtype=F32)), TypeError),
    (lambda: dict(new_lens=z(3, dtype=I32)), ValueError), (lambda: dict(workspace=z(16, dtype=torch.uint8)), RuntimeError),
])
def test_evict(pa, kw, error):
    with pytest.raises(error):
        pa.pa_evict(**{**evict_args(), **kw()})
    a = evict_args()
    with pytest.raises(RuntimeError):
        pa.pa_evict(**{**a, "new_lens": a["context_lens"]})
    assert pa.pa_device_error() == 0


def verify_args():
    return dict(target_probs=z(2, 4, 10, dtype=F32), draft_probs=z(2, 3, 10, dtype=F32),
                draft_tokens=z(2, 3, dtype=I32), accept_u=z(2, 3, dtype=F32), sample_u=z(2, dtype=F32))


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(target_probs=z(2, 3, 10, dtype=F32)), ValueError), (lambda: dict(draft_probs=z(2, 3, 9, dtype=F32)), ValueError),
    (lambda: dict(draft_probs=z(2, 3, 10)), TypeError), (lambda: dict(draft_tokens=z(2, 3, dtype=I64)), TypeError),
    (lambda: dict(accept_u=z(2, 2, dtype=F32)), ValueError), (lambda: dict(sample_u=z(3, dtype=F32)), ValueError),
    (lambda: dict(new_lens=z(2, dtype=I32)), ValueError), (lambda: dict(draft_lens=z(1, dtype=I32)), ValueError),
    (lambda: dict(out_tokens=z(2, 3, dtype=I32)), ValueError), (lambda: dict(target_probs=z(4, 2, 10, dtype=F32).transpose(0, 1)), ValueError),
    (lambda: dict(target_probs=z(2, 4, 10, dtype=F32, device="cpu")), TypeError),
])
def test_verify_drafts(pa, kw, error):
    with pytest.raises(error):
        pa.pa_verify_drafts(**{**verify_args(), **kw()})
    assert pa.pa_device_error() == 0


def test_verify_drafts_over_its_own_lengths(pa):
    a = verify_args()
    a["target_probs"].fill_(0.1)
    a["draft_probs"].fill_(0.1)
    a["accept_u"][1, 1] = 1.0
    lens = torch.tensor([9, 7], dtype=I32, device=DEV)
    got = pa.pa_verify_drafts(**a, context_lens=lens, new_lens=lens)
    assert got[2] is lens and lens.tolist() == [9, 5] and got[1].tolist() == [3, 1]


def test_both_ways_of_calling_agree(pa):
    """A call on the current stream goes through compiled checks, one on a stream that is
    named through the binding's own: the same results, strided arguments among them."""
    assert pa._fast is not None
    here = torch.cuda.current_stream()
    g = torch.Generator().manual_seed(3)
    rnd = lambda *s: torch.randn(*s, generator=g).half().to(DEV)  # noqa: E731
    qkv = rnd(20, 8, 64)
    turns, axis = pa.rope_table(64, device=DEV)
    got = []
    for stream in (None, here):
        r = rope_args() | dict(q_out=z(20, 4, 64), q=qkv[:, :4], k=qkv[:, 4:6], v=qkv[:, 6:],
                               positions=torch.arange(20, dtype=I32, device=DEV),
                               slot_mapping=torch.arange(20, device=DEV), turns=turns, pair_axis=axis)
        pa.pa_rope_append(**r, stream=stream)
        tables = torch.tensor([[0, 1], [1, 0]], dtype=I32, device=DEV)
        lens = torch.tensor([20, 17], dtype=I32, device=DEV)
        out, scores = z(2, 1, 4, 64), z(2, 2, 32, dtype=F32)
        ws = z(pa.pa_decode_scored_workspace_size(2, 4, 1, 64, 1, 2, 16), dtype=torch.uint8)
        pa.pa_decode_scored(out, scores, r["q_out"][:2].view(2, 1, 4, 64).contiguous(), r["k_cache"], r["v_cache"],
                            tables, lens, 0.125, workspace=ws, stream=stream)
        pos = torch.arange(32, dtype=I32, device=DEV).repeat(2, 2, 1)
        new = z(2, dtype=I32)
        we = z(pa.pa_evict_workspace_size(2, 2, 12), dtype=torch.uint8)
        pa.pa_evict(r["k_cache"], r["v_cache"], scores, pos, tables[:, :].contiguous(), lens.clamp_max(12), lens, 12,
                    1, 2, new_lens=new, workspace=we, stream=stream)
        v = verify_args()
        v["target_probs"] = torch.softmax(torch.arange(80, device=DEV).view(2, 4, 10) / 7.0, -1)
        v["sample_u"].fill_(0.4)
        v["accept_u"].fill_(0.9)
        toks, acc = z(2, 4, dtype=I32), z(2, dtype=I32)
        pa.pa_verify_drafts(**v, out_tokens=toks, num_accepted=acc, stream=stream)
        got.append([r["q_out"], r["k_cache"], r["v_cache"], out, scores, pos, new, toks, acc])
    torch.cuda.synchronize()
    assert pa.pa_device_error() == 0
    for x, y in zip(*got):
        assert torch.equal(x, y)
    assert got[0][3].abs().sum() > 0 and got[0][7].min() >= -1
