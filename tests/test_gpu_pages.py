"""The block pool's bookkeeping on the GPU against a simulation: whole numbers, equal."""
import numpy as np
import pytest
import torch

from tests import _pool_ref as ref

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


def i32(x):
    return torch.as_tensor(np.ascontiguousarray(np.asarray(x, np.int32))).to(DEV)


class Pool:
    """A pool on the GPU beside its simulation."""

    def __init__(self, pa, seqs, width, blocks, bs):
        self.pa, self.bs, self.blocks = pa, bs, blocks
        self.tables, self.refs = np.full((seqs, width), -1, np.int32), np.zeros(blocks, np.int32)
        self.lens = np.zeros(seqs, np.int32)
        self.t, self.r, self.l = i32(self.tables), i32(self.refs), i32(self.lens)

    def same(self):
        torch.cuda.synchronize()
        assert np.array_equal(self.t.cpu().numpy(), self.tables)
        assert np.array_equal(self.r.cpu().numpy(), self.refs)
        flat = self.tables[self.tables >= 0]
        assert np.array_equal(np.bincount(flat, minlength=self.blocks), self.refs)

    def reserve(self, lens):
        missing = self.pa.pa_reserve_blocks(self.t, self.r, i32(lens), self.bs)
        assert int(missing) == ref.reserve(self.tables, self.refs, lens, self.bs)
        self.same()
        return int(missing)

    def free(self, keep):
        self.pa.pa_free_blocks(self.t, self.r, i32(keep), self.bs)
        ref.free(self.tables, self.refs, keep, self.bs)
        self.same()

    def fork(self, src, dst):
        self.l = i32(self.lens)
        sb, db, counts = self.pa.pa_fork_blocks(self.t, self.l, self.r, i32(src), i32(dst), self.bs)
        pairs, missing = ref.fork(self.tables, self.lens, self.refs, src, dst, self.bs)
        self.same()
        assert np.array_equal(self.l.cpu().numpy(), self.lens)
        assert counts.tolist() == [len(pairs), missing]
        n = len(pairs)
        assert [tuple(p) for p in zip(sb[:n].tolist(), db[:n].tolist())] == [tuple(map(int, p)) for p in pairs]
        return missing

    def compact(self, in_place=True):
        if in_place:
            sb, db, counts = self.pa.pa_compact_blocks(self.t, self.r)
        else:
            was = self.t.clone(), self.r.clone()
            out = torch.full_like(self.t, -9), torch.full_like(self.r, -9)
            sb, db, counts = self.pa.pa_compact_blocks(self.t, self.r, *out)
            assert torch.equal(self.t, was[0]) and torch.equal(self.r, was[1])
            self.t, self.r = out
        self.tables, self.refs, pairs, live = ref.compact(self.tables, self.refs)
        self.same()
        n = len(pairs)
        assert counts.tolist() == [n, live]
        assert list(zip(sb[:n].tolist(), db[:n].tolist())) == pairs


SIZES = [(1, 1, 1), (1, 5, 3), (3, 7, 40), (5, 33, 128), (7, 3, 129), (16, 100, 1500), (64, 77, 5000),
         (2, 4097, 9001), (300, 13, 40000)]


@pytest.mark.parametrize("seqs,width,blocks", SIZES)
@pytest.mark.parametrize("bs", [8, 32])
def test_reserve_and_free(pa, seqs, width, blocks, bs):
    rng = np.random.default_rng(seqs * width + blocks)
    p = Pool(pa, seqs, width, blocks, bs)
    for _ in range(4):
        lens = rng.integers(0, width * bs + 1, seqs)
        lens[rng.random(seqs) < 0.2] = 0
        p.reserve(lens)
        keep = (lens * rng.random(seqs)).astype(np.int64)
        keep[rng.random(seqs) < 0.3] = 0
        keep[rng.random(seqs) < 0.2] = width * bs  # nothing to free
        p.free(keep)
    assert pa.pa_device_error() == 0


def test_a_pool_too_small(pa):
    p = Pool(pa, 6, 20, 50, 16)
    assert p.reserve([320] * 6) == 70
    assert p.reserve([320] * 6) == 70   # nothing left to take
    p.free([0, 320, 320, 320, 320, 320])
    assert p.reserve([0, 0, 33, 320, 0, 320]) > 0
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("seqs,width,blocks", [s for s in SIZES if s[0] >= 3])
@pytest.mark.parametrize("bs", [8, 16])
def test_fork_and_compact(pa, seqs, width, blocks, bs):
    rng = np.random.default_rng(seqs + blocks)
    p = Pool(pa, seqs, width, blocks, bs)
    for step in range(3):
        parents = rng.permutation(seqs)[:max(1, seqs // 3)]
        lens = np.zeros(seqs, np.int64)
        room = max(1, blocks // (2 * seqs)) * bs
        lens[parents] = rng.integers(0, min(width * bs, room) + 1, len(parents))
        if step == 0:
            lens[parents[0]] = min(width, max(1, blocks // 4)) * bs  # whole blocks alone
        p.free(np.zeros(seqs))
        p.reserve(lens)
        p.lens = lens.astype(np.int32)
        others = [s for s in range(seqs) if s not in set(parents.tolist())]
        dst = rng.permutation(others)[:rng.integers(1, len(others) + 1)]
        src = rng.choice(parents, len(dst))
        p.fork(src, dst)
        p.compact(in_place=step % 2 == 0)
        keep = np.where(rng.random(seqs) < 0.5, p.lens, 0)
        p.free(keep)
        p.compact(in_place=step % 2 == 1)
    assert pa.pa_device_error() == 0


def test_forks_without_a_free_block(pa):
    p = Pool(pa, 8, 4, 9, 16)
    p.reserve([40, 33, 0, 0, 0, 0, 0, 0])      # 3 + 3 blocks
    p.lens = np.array([40, 33, 0, 0, 0, 0, 0, 0], np.int32)
    assert p.fork([0, 1, 0, 1, 0], [2, 3, 4, 5, 6]) == 2
    assert p.lens.tolist() == [40, 33, 40, 33, 40, 32, 32, 0]
    assert pa.pa_device_error() == 0


def test_no_forks(pa):
    p = Pool(pa, 3, 4, 9, 16)
    p.reserve([40, 33, 0])
    counts = torch.full((2,), 7, dtype=torch.int32, device=DEV)
    e = torch.empty(0, dtype=torch.int32, device=DEV)
    pa.pa_fork_blocks(p.t, p.l, p.r, e, e, 16, counts=counts)
    assert counts.tolist() == [0, 0]
    p.same()


def test_compact_where_nothing_moves(pa):
    p = Pool(pa, 3, 40, 300, 16)
    p.compact()                     # an empty pool
    p.reserve([100, 640, 1])
    p.compact()                     # its front already
    q = Pool(pa, 2, 10, 20, 16)
    q.reserve([160, 160])           # full
    q.compact(in_place=False)


def test_entries_that_do_not_fit_the_pool(pa):
    """Ids outside it, and blocks that were not counted: reported, nothing else disturbed."""
    t, r = i32([[3, 99, 1], [-1, -1, -1]]), i32([0, 1, 0, 0])
    pa.pa_free_blocks(t, r, i32([0, 0]), 16)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert t.tolist() == [[-1] * 3] * 2 and r.tolist() == [0, 0, 0, 0]
    t, r = i32([[2, 9, -5]]), i32([0, 0, 1, 0])
    pa.pa_compact_blocks(t, r)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert t.tolist() == [[0, -1, -5]] and r.tolist() == [1, 0, 0, 0]
    t, r = i32([[-1, -1]]), i32([0, 0, 0])
    assert int(pa.pa_reserve_blocks(t, r, i32([50]), 16)) == 0  # longer than its row
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert t.tolist() == [[0, 1]]
    t, r, lens = i32([[0, 7], [-1, -1], [-1, -1]]), i32([1, 0, 0]), i32([20, 0, 0])
    sb, db, counts = pa.pa_fork_blocks(t, lens, r, i32([0, 5, 2]), i32([1, 0, 2]), 16)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    assert counts.tolist() == [0, 0] and lens.tolist() == [20, 16, 0]
    assert t.tolist() == [[0, 7], [0, -1], [-1, -1]] and r.tolist() == [2, 0, 0]


@pytest.mark.parametrize("bs,h,d,dtype", [(16, 8, 128, torch.float16), (8, 1, 64, torch.bfloat16),
                                          (32, 3, 128, torch.uint8), (16, 40, 128, torch.float8_e4m3fn)])
def test_copy_pages(pa, bs, h, d, dtype):
    rng = np.random.default_rng(h)
    nb, most = 50, 20
    raw = [torch.from_numpy(rng.integers(0, 256, (nb, h, bs, d * (1 if dtype.itemsize == 1 else 2))).astype(np.uint8))
           for _ in range(2)]
    scales = torch.from_numpy(rng.random((nb, h, 2)).astype(np.float32)) if dtype.itemsize == 1 else None
    order = rng.permutation(nb)
    src, dst = order[:most], order[most:2 * most]
    for count in (0, 1, 13, 20, 25, -3):
        k, v = (x.to(DEV).view(dtype) for x in raw)
        s = None if scales is None else scales.to(DEV)
        pa.pa_copy_pages(k, v, i32(src), i32(dst), i32([count, 0]), kv_scales=s)
        torch.cuda.synchronize()
        n = max(0, min(count, most))
        for got, was in ((k, raw[0]), (v, raw[1])):
            want = was.clone()
            want[dst[:n]] = was[src[:n]]
            assert torch.equal(got.view(torch.uint8).cpu(), want)
        if s is not None:
            want = scales.clone()
            want[dst[:n]] = scales[src[:n]]
            assert torch.equal(s.cpu(), want)
    assert pa.pa_device_error() == 0
    k, v = (x.to(DEV).view(dtype) for x in raw)
    pa.pa_copy_pages(k, v, i32([nb, 3, -1]), i32([4, 5, 6]), i32([3, 0]))
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    want = raw[0].clone()
    want[5] = raw[0][3]
    assert torch.equal(k.view(torch.uint8).cpu(), want)


def test_copy_past_four_gigabytes(pa):
    h, bs, d = 32, 32, 128
    nb = (5 << 30) // (h * bs * d)
    k, v = (torch.empty(nb, h, bs, d, dtype=torch.uint8, device=DEV) for _ in range(2))
    scales = torch.zeros(nb, h, 2, device=DEV)
    k[nb - 1], v[nb - 1], scales[nb - 1] = 5, 7, 0.5
    k[nb - 2] = v[nb - 2] = k[0] = v[0] = 1
    pa.pa_copy_pages(k, v, i32([nb - 1, nb - 1]), i32([0, nb - 2]), i32([2, 0]), kv_scales=scales)
    for b in (0, nb - 2):
        assert bool((k[b] == 5).all()) and bool((v[b] == 7).all()) and bool((scales[b] == 0.5).all())
    assert pa.pa_device_error() == 0
