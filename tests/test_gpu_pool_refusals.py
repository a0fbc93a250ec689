"""What the binding of the block-scaled cache, the pool's bookkeeping and the logits'
adjustment refuses before a launch (needs a GPU)."""
import pytest
import torch

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32, F32, U8 = torch.int32, torch.float32, torch.uint8


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


def refused(pa, fn, args, kw, error):
    before = {k: v.clone() for k, v in args.items() if isinstance(v, torch.Tensor)}
    with pytest.raises(error):
        getattr(pa, fn)(**{**args, **kw})
    torch.cuda.synchronize()
    assert pa.pa_device_error() == 0
    for k, v in before.items():
        assert torch.equal(args[k].view(U8), v.view(U8)), k


def append_args():
    return dict(k_cache=z(4, 2, 16, 128, dtype=U8), v_cache=z(4, 2, 16, 128, dtype=U8), kv_scales=z(4, 2, 2, dtype=F32),
                k_new=z(2, 2, 128), v_new=z(2, 2, 128), block_tables=z(2, 2, dtype=I32), context_lens=z(2, dtype=I32))


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(k_cache=z(4, 2, 16, 128)), TypeError), (lambda: dict(v_cache=z(4, 2, 8, 128, dtype=U8)), ValueError),
    (lambda: dict(kv_scales=z(4, 2, dtype=F32)), ValueError), (lambda: dict(kv_scales=z(4, 2, 2)), TypeError),
    (lambda: dict(k_new=z(2, 2, 128, dtype=F32)), TypeError), (lambda: dict(v_new=z(2, 2, 128, dtype=torch.bfloat16)), TypeError),
    (lambda: dict(k_new=z(3, 2, 128)), ValueError), (lambda: dict(k_new=z(2, 128, 2).transpose(1, 2)), ValueError),
    (lambda: dict(k_new=z(2, 2, 128).cpu()), TypeError), (lambda: dict(q_len=2), ValueError),
    (lambda: dict(block_tables=z(4, dtype=I32)), ValueError), (lambda: dict(context_lens=z(2, dtype=torch.int64)), TypeError),
    (lambda: dict(k_cache=z(4, 2, 16, 64, dtype=U8), v_cache=z(4, 2, 16, 64, dtype=U8), k_new=z(2, 2, 64),
                  v_new=z(2, 2, 64)), RuntimeError),
    (lambda: dict(k_cache=None), Exception),
])
def test_append(pa, kw, error):
    refused(pa, "pa_append_kv_block_scaled", append_args(), kw(), error)


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(q=z(2, 2, 4, 128)), ValueError), (lambda: dict(out=z(2, 1, 4, 64)), ValueError),
    (lambda: dict(out=z(2, 1, 4, 128, dtype=torch.bfloat16)), TypeError), (lambda: dict(k_cache=z(4, 2, 16, 128)), TypeError),
    (lambda: dict(kv_scales=z(2, 2, 2, dtype=F32)), ValueError), (lambda: dict(num_splits=0), RuntimeError),
    (lambda: dict(num_splits=2, workspace=z(16, dtype=U8)), RuntimeError), (lambda: dict(scale=float("inf")), RuntimeError),
    (lambda: dict(q=z(2, 1, 3, 128), out=z(2, 1, 3, 128)), RuntimeError), (lambda: dict(q=z(2, 128)), ValueError),
    (lambda: dict(context_lens=z(3, dtype=I32)), ValueError),
])
def test_attend(pa, kw, error):
    a = append_args()
    args = dict(out=z(2, 1, 4, 128), q=z(2, 1, 4, 128), scale=0.1,
                **{k: a[k] for k in ("k_cache", "v_cache", "kv_scales", "block_tables", "context_lens")})
    refused(pa, "pa_decode_block_scaled", args, kw(), error)


def pool_args(**more):
    return dict(block_tables=z(2, 4, dtype=I32), ref_counts=z(9, dtype=I32), **more)


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(keep_lens=z(3, dtype=I32)), ValueError), (lambda: dict(keep_lens=z(2)), TypeError),
    (lambda: dict(block_size=10), RuntimeError), (lambda: dict(ref_counts=z(9, 1, dtype=I32)), ValueError),
    (lambda: dict(block_tables=z(2, 8, dtype=I32)[:, ::2]), ValueError), (lambda: dict(block_tables=z(2, 4, dtype=I32).cpu()), TypeError),
    (lambda: dict(ref_counts=z(9, dtype=I32).cpu()), TypeError),
])
def test_free(pa, kw, error):
    refused(pa, "pa_free_blocks", pool_args(keep_lens=z(2, dtype=I32), block_size=16), kw(), error)


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(lens=z(3, dtype=I32)), ValueError), (lambda: dict(missing=z(2, dtype=I32)), ValueError),
    (lambda: dict(workspace=z(16, dtype=U8)), RuntimeError), (lambda: dict(block_size=0), RuntimeError),
    (lambda: dict(ref_counts=z(9, dtype=torch.int64)), TypeError),
])
def test_reserve(pa, kw, error):
    refused(pa, "pa_reserve_blocks", pool_args(lens=z(2, dtype=I32), block_size=16), kw(), error)


def test_counts_inside_the_tables(pa):
    both = z(64, dtype=I32)
    with pytest.raises(RuntimeError):
        pa.pa_free_blocks(both[:32].view(4, 8), both[16:], z(4, dtype=I32), 16)
    with pytest.raises(RuntimeError):
        pa.pa_reserve_blocks(both[:32].view(4, 8), both[32:], both[4:8], 16)
    assert bool((both == 0).all())


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(src_seqs=z(3, dtype=I32)), ValueError), (lambda: dict(dst_seqs=z(2, dtype=I32)), ValueError),
    (lambda: dict(src_blocks=z(2, dtype=I32)), ValueError), (lambda: dict(counts=z(1, dtype=I32)), ValueError),
    (lambda: dict(context_lens=z(3, dtype=I32)), ValueError),
    (lambda: dict(src_seqs=z(3, dtype=I32), dst_seqs=z(3, dtype=I32)), RuntimeError),  # more forks than rows
    (lambda: dict(workspace=z(32, dtype=U8)), RuntimeError),
])
def test_fork(pa, kw, error):
    args = pool_args(context_lens=z(2, dtype=I32), src_seqs=z(1, dtype=I32), dst_seqs=torch.ones(1, dtype=I32, device=DEV),
                     block_size=16)
    refused(pa, "pa_fork_blocks", args, kw(), error)


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(block_tables_out=z(2, 4, dtype=I32)), ValueError),
    (lambda: dict(block_tables_out=z(2, 3, dtype=I32), ref_counts_out=z(9, dtype=I32)), ValueError),
    (lambda: dict(block_tables_out=z(2, 4, dtype=I32), ref_counts_out=z(8, dtype=I32)), ValueError),
    (lambda: dict(src_blocks=z(5, dtype=I32)), ValueError), (lambda: dict(counts=z(2)), TypeError),
])
def test_compact(pa, kw, error):
    refused(pa, "pa_compact_blocks", pool_args(), kw(), error)


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(v_cache=z(4, 2, 16, 64)), ValueError), (lambda: dict(kv_scales=z(4, 2, 2, dtype=F32)), RuntimeError),
    (lambda: dict(k_cache=z(4, 2, 16, 128, dtype=F32), v_cache=z(4, 2, 16, 128, dtype=F32)), TypeError),
    (lambda: dict(dst_blocks=z(4, dtype=I32)), ValueError), (lambda: dict(counts=z(1, dtype=I32)), ValueError),
    (lambda: dict(src_blocks=z(3, dtype=torch.int64)), TypeError),
])
def test_copy(pa, kw, error):
    args = dict(k_cache=z(4, 2, 16, 128), v_cache=z(4, 2, 16, 128), src_blocks=z(3, dtype=I32), dst_blocks=z(3, dtype=I32),
                counts=z(2, dtype=I32))
    refused(pa, "pa_copy_pages", args, kw(), error)


@pytest.mark.parametrize("kw,error", [
    (lambda: dict(logits=z(2, 3, 100, dtype=torch.float64)), TypeError), (lambda: dict(logits=z(6, 100, dtype=F32)), ValueError),
    (lambda: dict(out=z(2, 3, 99, dtype=F32)), ValueError), (lambda: dict(probs=True), TypeError),
    (lambda: dict(history=z(2, 5, dtype=I32)), ValueError), (lambda: dict(history_lens=z(2, dtype=I32)), ValueError),
    (lambda: dict(prompt_lens=z(2, dtype=I32)), ValueError), (lambda: dict(drafts=z(2, 3, dtype=I32)), ValueError),
    (lambda: dict(repetition=z(3, dtype=F32)), ValueError), (lambda: dict(temperature=z(2)), TypeError),
    (lambda: dict(bias_ids=z(2, 4, dtype=I32)), ValueError),
    (lambda: dict(bias_ids=z(2, 4, dtype=I32), bias_values=z(2, 3, dtype=F32)), ValueError),
    (lambda: dict(bias_ids=z(2, 1025, dtype=I32), bias_values=z(2, 1025, dtype=F32)), RuntimeError),
    (lambda: dict(mask=z(2, 3, 3, dtype=I32)), ValueError), (lambda: dict(mask=z(2, 3, 4)), TypeError),
    (lambda: dict(mask=z(2, 3, 8, dtype=I32)[:, :, ::2]), ValueError),
    (lambda: dict(logits=z(2, 3, 200)[:, :, ::2], out=z(2, 3, 100)), ValueError),
    (lambda: dict(logits=z(2, 4, 100, dtype=F32)[:, :3]), ValueError),  # rows not evenly spaced
    (lambda: dict(logits=z(1, 1, 262145, dtype=F32), out=None), RuntimeError),
])
def test_logits(pa, kw, error):
    refused(pa, "pa_adjust_logits", dict(out=z(2, 3, 100), logits=z(2, 3, 100)), kw(), error)


def test_logits_over_their_inputs(pa):
    x = torch.zeros(1, 1, 4000, device=DEV)
    half = x.view(torch.float16)[:, :, :4000]
    with pytest.raises(RuntimeError):
        pa.pa_adjust_logits(x, half, probs=True)
    with pytest.raises(RuntimeError):
        pa.pa_adjust_logits(x[:, :, 4:], x[:, :, :-4])
    with pytest.raises(RuntimeError):
        pa.pa_adjust_logits(x, torch.zeros_like(x), repetition=x[0, 0, 8:9])
    assert bool((x == 0).all())
