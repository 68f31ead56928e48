"""The block pool's kernels on rows that end with a whole block (a fork shares them
whole, their first new token takes a block) and on empty ones, many of each."""
import numpy as np
import pytest
import torch

from gpu_util import L
from oracle import blocks as ob
from test_gpu_blocks import BS, SIZES, Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _pool(size, seed):
    n, longest, blocks, group, shared = size
    rng = np.random.default_rng(seed)
    lens = rng.integers(0, longest + 1, n) + shared * BS
    kind = rng.random(n)
    lens = np.where(kind < 0.4, np.maximum(lens // BS, 1) * BS, np.where(kind < 0.6, 0, lens))
    p = Pool(lens, blocks + 4 * n, seed, group, shared)
    assert (lens % BS == 0)[lens > 0].sum() > n // 4 and (lens == 0).sum() > n // 10
    return p, rng


@pytest.mark.parametrize("size", [s for s in SIZES if s[0] >= 64])
def test_fork(size):
    p, rng = _pool(size, 21)
    n, group = size[0], size[3]
    for step in range(3):
        first = np.arange(n) // group * group
        parents = np.minimum(first + rng.integers(0, group, n), n - 1) if step < 2 else rng.integers(-1, n, n)
        # kept to a whole block, to a token before and one behind it, and to nothing
        keep = rng.integers(0, size[1] // BS + 2, n) * BS + rng.choice([-1, 0, 0, 0, 1], n)
        keep = np.where(rng.random(n) < 0.3, 0, np.maximum(keep, 0)) if step else np.full(n, -1)
        pairs = p.fork(parents, keep).cpu().numpy()
        whole = np.asarray(p.lens) % BS == 0
        assert (pairs[whole] == -1).all() and whole.sum() > n // 10  # nothing to copy
        ob.check(p.tables, p.lens, p.refs)
    assert L().cb_last_error() == 0


@pytest.mark.parametrize("size", [s for s in SIZES if s[0] >= 64])
def test_grow(size):
    p, rng = _pool(size, 22)
    n = size[0]
    for q in (np.ones(n, int), rng.integers(0, 3, n), BS * rng.integers(0, 2, n)):
        need = sum(ob.n_blocks(a + b) - ob.n_blocks(a) for a, b in zip(p.lens, q))
        before = (p.refs > 0).sum()
        _, stay = p.grow(q)
        assert not stay and (p.refs > 0).sum() - before == need
        ob.check(p.tables, p.lens, p.refs)


@pytest.mark.parametrize("size", [s for s in SIZES if s[0] >= 64])
def test_compact(size):
    p, rng = _pool(size, 23)
    n = size[0]
    p.fork(np.where(rng.random(n) < 0.4, -1, np.arange(n)), rng.integers(0, size[1] // BS + 2, n) * BS)
    p.compact()
    ob.check(p.tables, p.lens, p.refs)
    live = int((p.refs > 0).sum())
    assert (p.refs[:live] > 0).all()
