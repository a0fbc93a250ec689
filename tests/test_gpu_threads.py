"""Calls that wait for room in the driver's launch queue: the process's other Python threads
go on meanwhile (needs a GPU)."""
import threading
import time

import pytest
import torch

from tests import test_gpu_operator_refusals as args
from tests.test_gpu_operator_refusals import pa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu
DEV = "cuda"
I32 = torch.int32


def calls(pa):  # noqa: F811
    """Each of the calls that go through the compiled checks, every buffer given."""
    rope, scored, evict, verify = args.rope_args(), args.scored_args(), args.evict_args(), args.verify_args()
    rope["turns"], rope["pair_axis"] = pa.rope_table(64, device=DEV)
    scored["workspace"] = args.z(pa.pa_decode_scored_workspace_size(2, 4, 1, 64, 1, 2, 16), dtype=torch.uint8)
    evict.update(new_lens=args.z(2, dtype=I32), workspace=args.z(pa.pa_evict_workspace_size(2, 2, 8), dtype=torch.uint8))
    verify["target_probs"].fill_(0.1)
    verify.update(out_tokens=args.z(2, 4, dtype=I32), num_accepted=args.z(2, dtype=I32))
    return {"pa_rope_append": rope, "pa_decode_scored": scored, "pa_evict": evict, "pa_verify_drafts": verify}


@pytest.mark.parametrize("name", ["pa_rope_append", "pa_decode_scored", "pa_evict", "pa_verify_drafts"])
def test_other_threads_go_on(pa, name):  # noqa: F811
    kw, call = calls(pa)[name], getattr(pa, name)
    for _ in range(3):
        call(**kw)
    torch.cuda.synchronize()
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.is_set():
            ticks.append(time.perf_counter())
            time.sleep(0.002)

    clock = threading.Thread(target=tick)
    clock.start()
    try:
        torch.cuda._sleep(1_200_000_000)   # about 0.6 s: the queue behind it fills
        begin = time.perf_counter()
        for _ in range(3000):
            call(**kw)
        took = time.perf_counter() - begin
        torch.cuda.synchronize()
    finally:
        stop.set()
        clock.join()
    if took < 0.3:
        pytest.skip("the queue took every call: none had to wait")
    inside = [t for t in ticks if begin <= t <= begin + took]
    gaps = [b - a for a, b in zip([begin] + inside, inside + [begin + took])]
    assert max(gaps) < 0.2, max(gaps)   # (a thread that is kept waiting stands still for `took`)
    assert pa.pa_device_error() == 0
