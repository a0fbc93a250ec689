"""The block pool's bookkeeping where a warp's part passes one step of its walk: large pools and
tables, very many sequences and forks, against the simulation."""
import numpy as np
import pytest

from tests.test_gpu_pages import Pool, i32, pa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu


class Large(Pool):
    """The same simulation without a loop an entry."""

    def reserve(self, lens):
        missing = self.pa.pa_reserve_blocks(self.t, self.r, i32(lens), self.bs)
        need = -(-np.maximum(np.asarray(lens, np.int64), 0) // self.bs)
        want = np.flatnonzero((np.arange(self.tables.shape[1]) < need[:, None]) & (self.tables < 0))
        empty = np.flatnonzero(self.refs == 0)[:len(want)]
        self.tables.reshape(-1)[want[:len(empty)]] = empty
        self.refs[empty] = 1
        assert int(missing) == len(want) - len(empty)
        self.same()

    def free(self, keep):
        self.pa.pa_free_blocks(self.t, self.r, i32(keep), self.bs)
        kept = -(-np.maximum(np.asarray(keep, np.int64), 0) // self.bs)
        gone = (np.arange(self.tables.shape[1]) >= kept[:, None]) & (self.tables >= 0)
        np.subtract.at(self.refs, self.tables[gone], 1)
        self.tables[gone] = -1
        self.same()


def scattered(p, rng, room):
    """Lengths of `room` blocks a row at most; most rows given up again, so that the blocks in use
    and the free ones lie anywhere."""
    seqs, width = p.tables.shape
    lens = rng.integers(0, min(width, room) * p.bs + 1, seqs)
    p.reserve(lens)
    p.free(np.where(rng.random(seqs) < 0.6, 0, (lens * rng.random(seqs)).astype(np.int64)))


@pytest.mark.parametrize("blocks", [131072, 131073, 300007])
@pytest.mark.parametrize("in_place", [True, False])
def test_pools_of_more_than_four_steps_a_warp(pa, blocks, in_place):  # noqa: F811
    """512 counts a warp stay in registers; of larger pools they are read again."""
    rng = np.random.default_rng(blocks)
    p = Large(pa, 300, 1000, blocks, 16)   # (1172 entries a warp: more than the eight steps kept as flags)
    scattered(p, rng, 2 * blocks // 300)
    scattered(p, rng, blocks // 300)
    p.lens = np.zeros(300, np.int32)
    used = (p.tables >= 0).cumprod(1).sum(1)
    p.lens[:] = np.maximum(used * 16 - rng.integers(0, 16, 300), 0)
    empty = np.flatnonzero(p.lens == 0)
    parents = rng.permutation(np.flatnonzero(p.lens > 0))[:20]
    p.fork(rng.choice(parents, len(empty)), empty)
    p.compact(in_place)
    p.free(np.where(rng.random(300) < 0.5, 0, 1 << 20))
    p.compact(not in_place)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("seqs,width", [(20000, 1), (20000, 3), (9000, 40), (1, 300000)])
@pytest.mark.parametrize("bs", [8, 32])
def test_tables_of_many_rows(pa, seqs, width, bs):  # noqa: F811
    """More rows than a thread block keeps the needs of (1024), parts of more steps than flags."""
    rng = np.random.default_rng(seqs + width)
    p = Large(pa, seqs, width, seqs * width // 2 + 5, bs)
    for _ in range(2):
        scattered(p, rng, width)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("late", [0, 1023, 1024, 2499, 2500, 17000, 19999])
def test_a_row_past_its_table(pa, late):  # noqa: F811
    """A length past the table's width anywhere in a large batch is recorded, and takes the width."""
    p = Large(pa, 20000, 3, 200, 16)
    lens = np.zeros(20000, np.int64)
    lens[late] = 49
    p.reserve(lens)
    assert pa.pa_device_error() == pa.PA_ERR_DEVICE_CHECK
    lens[late] = 48
    p.reserve(lens)
    assert pa.pa_device_error() == 0


@pytest.mark.parametrize("blocks,width,children", [(4000, 3, 33), (4000, 3, 70), (5000, 9, 255), (5000, 9, 256),
                                                   (5000, 9, 300), (40000, 3, 8192), (40000, 3, 9000)])
def test_many_forks(pa, blocks, width, children):  # noqa: F811
    """More children than warps, and than a warp's lanes times warps."""
    rng = np.random.default_rng(children)
    p = Large(pa, children + 5, width, blocks, 16)
    lens = np.zeros(children + 5, np.int64)
    lens[:5] = rng.integers(1, width * 16 + 1, 5)
    lens[3] = 16 * (width - 1)
    p.reserve(lens)
    p.lens = lens.astype(np.int32)
    order = rng.permutation(np.arange(5, children + 5))
    p.fork(rng.integers(0, 5, children), order)
    p.compact()
    assert pa.pa_device_error() == 0
