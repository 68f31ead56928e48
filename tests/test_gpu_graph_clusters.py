"""One graph object whose recordings differ in their kernels' clusters only: an
update in place would keep the first one's."""
import numpy as np
import pytest
import torch

from cross_util import Batch
from gpu_util import L
from oracle import blocks as ob
from test_gpu_blocks import Pool

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _ints(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


class Steps:
    """A pool's calls on prepared arguments, each with the oracle's part."""

    def __init__(self, rows, blocks, longest, seed, new=3):
        rng = np.random.default_rng(seed)
        self.p = Pool(rng.integers(1, longest, rows), blocks, seed, group=4, shared=1, width=longest // 16 + 2 + 8 * new // 4)
        n = rows
        self.parents = np.minimum(np.arange(n) // 4 * 4 + rng.integers(0, 4, n), n - 1)
        self.q = rng.integers(0, new + 1, n)
        cu = np.concatenate([[0], np.cumsum(self.q)])
        self.d_parents, self.d_cu = _ints(self.parents), _ints(cu)
        self.pairs, self.ctx = _ints(np.zeros((n, 2))), _ints(np.zeros(n))
        self.slots = torch.zeros(int(cu[-1]), dtype=torch.int64, device="cuda")
        self.map, self.moves, self.counts = _ints(np.zeros(blocks)), _ints(np.zeros((blocks // 2, 2))), _ints(np.zeros(2))

    def fork(self):
        p = self.p
        L().cb_fork_blocks(self.d_parents, None, p.d_tables, p.d_lens, p.d_refs, self.pairs, p.ws)

    def forked(self):
        p = self.p
        pairs, cut = ob.fork(self.parents, None, p.tables, p.lens, p.refs)
        assert not cut and np.array_equal(self.pairs.cpu().numpy(), pairs)
        p.same()

    def grow(self):
        p = self.p
        L().cb_grow_blocks(self.d_cu, p.d_tables, p.d_lens, p.d_refs, self.ctx, self.slots, p.ws)

    def grown(self):
        p = self.p
        ctx, slots, stay = ob.grow(self.q, p.tables, p.lens, p.refs)
        assert not stay and np.array_equal(self.ctx.cpu().numpy(), ctx) and np.array_equal(self.slots.cpu().numpy(), slots)
        p.same()

    def compact(self):
        p = self.p
        L().cb_compact_blocks(p.d_tables, p.d_lens, p.d_refs, self.map, self.moves, self.counts, p.ws)

    def compacted(self):
        p = self.p
        block_map, moves, live = ob.compact(p.tables, p.lens, p.refs)
        assert self.counts.tolist() == [live, len(moves)] and np.array_equal(self.map.cpu().numpy(), block_map)
        p.same()


class Recorder:
    def __init__(self):
        self.s, self.g = torch.cuda.Stream(), L().Graph()

    def run(self, *calls):
        torch.cuda.synchronize()
        self.g.begin(self.s)
        with torch.cuda.stream(self.s):
            for c in calls:
                c()
        self.g.end(self.s)
        assert L().cb_last_error(self.s) == 0


@pytest.fixture
def recorder():
    for steps in (Steps(8, 200, 60, 1), Steps(100, 9000, 60, 2), Steps(100, 20000, 60, 3), Steps(100, 20000, 60, 4, new=400)):
        for call in (steps.fork, steps.grow, steps.compact):              # outside a capture first
            call()
    assert L().cb_last_error() == 0
    r = Recorder()
    yield r
    r.g.close()


@pytest.mark.parametrize("op,check", [("fork", "forked"), ("grow", "grown"), ("compact", "compacted")])
def test_one_call_on_small_and_large_pools(op, check, recorder):
    """One CTA, eight, and back: the pool's size decides."""
    small, large = Steps(8, 200, 60, 1), Steps(100, 20000, 60, 3)
    for steps in (small, large, small, small, large, large, small):
        recorder.run(getattr(steps, op))
        getattr(steps, check)()


def test_other_calls_behind_a_pools(recorder):
    """Ordinary and cooperative kernels in the place of a cluster's, and the other way round."""
    lib = L()
    large = Steps(100, 20000, 60, 3)
    many = Steps(100, 20000, 60, 4, new=400)
    assert many.slots.numel() > 8192
    b = Batch([(2, 300), (1, 40)], 8, 4, 64, seed=3)
    out, ws = torch.full_like(b.q, 7.0), b.workspace()
    b.run(out, ws)
    new = torch.randn(3, 4, 64, device="cuda").to(torch.bfloat16)
    k, v = (torch.zeros(5, 4, 16, 64, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    where = torch.tensor([3, 77, 20], device="cuda")
    append = lambda: lib.cb_kv_append(new, new, where, k, v)  # noqa: E731
    append()
    for _ in range(2):
        recorder.run(large.fork)
        large.forked()
        k.zero_()
        recorder.run(append)
        assert torch.equal(k.transpose(1, 2).reshape(-1, 4, 64)[where], new)
        recorder.run(large.compact)
        large.compacted()
        out.fill_(7.0)
        recorder.run(lambda: b.run(out, ws, check=False))
        b.compare(out)
        recorder.run(many.grow)
        many.grown()
        recorder.run(large.grow)
        large.grown()


def test_a_step_of_several_calls(recorder):
    small, large = Steps(8, 200, 60, 1), Steps(100, 20000, 60, 3)
    caches = {id(t): [torch.arange(len(t.p.refs), device="cuda").view(1, -1, 1).expand(2, -1, 16).contiguous()] for t in (small, large)}
    for t in (small, large, small, large, large, small):
        cache, before = caches[id(t)], caches[id(t)][0].clone()
        recorder.run(t.fork, lambda: L().cb_copy_blocks_layers(t.pairs, cache), t.grow)
        pairs, _ = ob.fork(t.parents, None, t.p.tables, t.p.lens, t.p.refs)
        assert np.array_equal(t.pairs.cpu().numpy(), pairs)
        for src, dst in pairs:
            if src >= 0:
                before[:, dst] = before[:, src]
        assert torch.equal(cache[0], before)
        t.grown()


def test_recorded_while_the_last_one_runs(recorder):
    """Small and large pools in turn, all launched before one synchronisation."""
    small, large = Steps(8, 200, 60, 1), Steps(100, 20000, 60, 3)
    torch.cuda.synchronize()
    for _ in range(5):
        for t in (small, large):
            recorder.g.begin(recorder.s)
            with torch.cuda.stream(recorder.s):
                t.fork()
                t.compact()
            recorder.g.end(recorder.s)
    assert L().cb_last_error(recorder.s) == 0
    for t in (small, large):
        for _ in range(5):
            pairs, cut = ob.fork(t.parents, None, t.p.tables, t.p.lens, t.p.refs)
            assert not cut
            block_map, _, _ = ob.compact(t.p.tables, t.p.lens, t.p.refs)
        assert np.array_equal(t.pairs.cpu().numpy(), pairs) and np.array_equal(t.map.cpu().numpy(), block_map)
        t.p.same()
