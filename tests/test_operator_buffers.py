"""Where the binding takes the buffers that a call does not give: from the allocator's pool
of the stream that the call runs on.  Memory of another stream's pool may be handed out
again as soon as the call returns, while its kernels still use it (no GPU needed: the
library, the streams and the allocations are stand-ins)."""
import contextlib

import pytest
import torch

import paged_kv_cache_20_gb300 as pa

I32, I64, F32, F16 = torch.int32, torch.int64, torch.float32, torch.float16


class Library:
    """Every size is 512 bytes, every call succeeds."""
    def __getattr__(self, name):
        return lambda *a: 512 if name.endswith("_size") else 0


class Stream:
    """What the binding reads of a stream."""
    cuda_stream = 0x7F0000
    device = torch.device("cpu")


@pytest.fixture
def made(monkeypatch):
    """[(function, the stream in force)] of the allocations made by a call."""
    got, current = [], [None]

    @contextlib.contextmanager
    def on(stream):
        current[0], before = stream, current[0]
        yield
        current[0] = before

    def spy(name):
        real = getattr(torch, name)

        def make(*a, **kw):
            got.append((name, current[0]))
            return real(*a, **kw)
        return make

    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("empty", "empty_like", "zeros"):
        monkeypatch.setattr(torch, name, spy(name))
    monkeypatch.setattr(pa, "load", Library)
    monkeypatch.setattr(pa, "_lib", None)
    monkeypatch.setattr(pa, "_cuda", lambda t, name, dtype=None: t.data_ptr())
    monkeypatch.setattr(pa, "_ptr", lambda t, name, dtype, dev: t.data_ptr())
    monkeypatch.setattr(pa, "_device_of", lambda t: 0)
    monkeypatch.setattr(pa, "_prob_rows", lambda t, name, n, r, dev: (t.data_ptr(), t.shape[2]))
    return got


def z(*shape, dtype=F16):
    return torch.full(shape, 0, dtype=dtype)


def calls(stream):
    kv = dict(k_cache=z(4, 2, 16, 64), v_cache=z(4, 2, 16, 64))
    at = dict(block_tables=z(2, 2, dtype=I32), context_lens=z(2, dtype=I32), scale=0.1)
    new = dict(k_new=z(2, 2, 64), v_new=z(2, 2, 64))
    q = dict(q=z(2, 1, 4, 64), out=z(2, 1, 4, 64))
    codes = {k: z(4, 2, 16, 64, dtype=torch.uint8) for k in kv}
    scales = dict(k_scale=z(2, dtype=F32), v_scale=z(2, dtype=F32))
    ledger = dict(scores=z(2, 2, 32, dtype=F32), row_pos=z(2, 2, 32, dtype=I32))
    probs = dict(target_probs=z(2, 4, 10, dtype=F32), draft_probs=z(2, 3, 10, dtype=F32),
                 draft_tokens=z(2, 3, dtype=I32), accept_u=z(2, 3, dtype=F32), sample_u=z(2, dtype=F32))
    step = {**at, **kv, **new, "q": q["q"]}
    lens = dict(seq_lens=z(2, dtype=I32))
    return {
        "pa_slot_mapping": (1, lambda: pa.pa_slot_mapping(at["block_tables"], at["context_lens"], 16, stream=stream)),
        "pa_decode_fp8": (1, lambda: pa.pa_decode_fp8(**q, **codes, **scales, **at, num_splits=2, stream=stream)),
        "pa_append_decode": (1, lambda: pa.pa_append_decode(**q, **kv, **new, **at, num_splits=2, stream=stream)),
        "pa_decode_cascade": (1, lambda: pa.pa_decode_cascade(**q, **kv, **at, prefix_blocks=1, stream=stream)),
        "step": (2, lambda: pa.paged_decode_step(**step, stream=stream)),
        "step in partitions": (3, lambda: pa.paged_decode_step(**step, num_splits=2, stream=stream)),
        "fused step": (1, lambda: pa.paged_decode_step(**step, fused=True, stream=stream)),
        "pa_decode_scored": (1, lambda: pa.pa_decode_scored(**q, **kv, **at, scores=ledger["scores"], stream=stream)),
        "pa_evict": (2, lambda: pa.pa_evict(**kv, **ledger, **lens, block_tables=at["block_tables"],
                                            context_lens=at["context_lens"], budget=8, stream=stream)),
        "pa_verify_drafts": (3, lambda: pa.pa_verify_drafts(**probs, context_lens=at["context_lens"], stream=stream)),
    }


@pytest.mark.parametrize("name", sorted(calls(None)))
def test_on_the_stream_that_is_named(made, name):
    stream = Stream()
    number, call = calls(stream)[name]
    call()
    assert len(made) == number
    assert all(at is stream for _, at in made), made


@pytest.mark.parametrize("name", sorted(calls(None)))
def test_on_the_current_stream_when_none_is_named(made, name, monkeypatch):
    monkeypatch.setattr(pa, "_stream", lambda s: 0)
    monkeypatch.setattr(pa, "_stream_on", lambda s, dev: 0)
    monkeypatch.setattr(pa, "_fast", None)
    number, call = calls(None)[name]
    call()
    assert [at for _, at in made] == [None] * number


def test_raw_handles(made, monkeypatch):
    """A handle stands for its stream, 0 and 1 (the legacy stream) for the default one; the
    per-thread default stream (2) is another one in every thread, so nothing is made on it."""
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device: (handle, device))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device: ("default", device))
    tables, lens = z(2, 2, dtype=I32), z(2, dtype=I32)
    cpu = torch.device("cpu")
    for handle, want in ((0x55AA00, (0x55AA00, cpu)), (0, ("default", cpu)), (1, ("default", cpu))):
        pa.pa_slot_mapping(tables, lens, 16, stream=handle)
        assert made[-1][1] == want
    with pytest.raises(ValueError, match="per-thread"):
        pa.pa_slot_mapping(tables, lens, 16, stream=2)
    pa.pa_slot_mapping(tables, lens, 16, out=z(2, dtype=I64), stream=2)


def test_a_stream_of_another_device_is_refused(made):
    stream = Stream()
    stream.device = torch.device("meta")
    with pytest.raises(ValueError, match="stream"):
        pa.pa_slot_mapping(z(2, 2, dtype=I32), z(2, dtype=I32), 16, stream=stream)
