"""The block pool's kernels against the oracle: every integer equal."""
import numpy as np
import pytest
import torch

from gpu_util import L
from oracle import blocks as ob

pytestmark = pytest.mark.gpu

BS = 16


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Pool:
    """A random pool on the device and its copy for the oracle.  Rows in groups share
    their group's first blocks; spare table entries hold `junk`."""

    def __init__(self, lens, num_blocks, seed=0, group=1, shared=0, width=None, junk=-1, outside=()):
        rng = np.random.default_rng(seed)
        lens = np.asarray(lens, np.int64)
        ids = rng.permutation(num_blocks)
        width = width or max(1, max((ob.n_blocks(n) for n in lens), default=1)) + 2
        self.tables = np.full((len(lens), width), junk, np.int64)
        self.refs = np.zeros(num_blocks, np.int64)
        at = 0
        for r, n in enumerate(lens):
            k = min(shared, n // BS)
            if r % group == 0:
                prefix = ids[at:at + shared]
                at += shared
            own = ob.n_blocks(n) - k
            self.tables[r, :k] = prefix[:k]
            self.tables[r, k:k + own] = ids[at:at + own]
            assert at + own <= num_blocks
            at += own
            for e in self.tables[r, :k + own]:
                self.refs[e] += 1
        self.outside = np.zeros(num_blocks, np.int64)
        for b in outside:
            self.outside[b] += 1
        self.refs += self.outside
        self.lens = lens
        i = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
        self.d_tables, self.d_lens, self.d_refs = i(self.tables), i(self.lens), i(self.refs)
        n = L().cb_block_ops_workspace_size(len(lens), width, num_blocks)
        self.ws = torch.full((n,), 0xFF, dtype=torch.uint8, device="cuda")

    def fork(self, parents, keep=None):
        n = len(self.lens)
        i = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
        pairs = torch.full((n, 2), 77, dtype=torch.int32, device="cuda")
        L().cb_fork_blocks(i(parents), None if keep is None else i(keep), self.d_tables, self.d_lens, self.d_refs, pairs,
                           self.ws)
        want, cut = ob.fork(parents, keep, self.tables, self.lens, self.refs)
        assert L().cb_last_error() == (L().CB_ESTATE if cut else 0)
        assert np.array_equal(pairs.cpu().numpy(), want)
        self.same()
        return pairs

    def grow(self, q_lens, pad=0, stay=None):
        n = len(self.lens)
        cu = np.concatenate([[0], np.cumsum(q_lens)]).astype(np.int32)
        slots = torch.full((int(cu[-1]) + pad,), 99, dtype=torch.int64, device="cuda")
        ctx = torch.full((n,), 99, dtype=torch.int32, device="cuda")
        L().cb_grow_blocks(torch.from_numpy(cu).cuda(), self.d_tables, self.d_lens, self.d_refs, ctx, slots, self.ws)
        want_ctx, want, staying = ob.grow(q_lens, self.tables, self.lens, self.refs)
        status = L().cb_last_error()
        assert status != 0 if staying else status == 0
        assert np.array_equal(ctx.cpu().numpy(), want_ctx)
        assert np.array_equal(slots.cpu().numpy(), np.concatenate([want, np.full(pad, -1)]))
        self.same()
        return status, staying

    def compact(self, max_pairs=None):
        nb = len(self.refs)
        cap = nb // 2 if max_pairs is None else max_pairs
        block_map = torch.full((nb,), 77, dtype=torch.int32, device="cuda")
        pairs = torch.full((cap, 2), 77, dtype=torch.int32, device="cuda")
        counts = torch.full((2,), 77, dtype=torch.int32, device="cuda")
        L().cb_compact_blocks(self.d_tables, self.d_lens, self.d_refs, block_map, pairs, counts, self.ws)
        want_map, moves, live = ob.compact(self.tables, self.lens, self.refs, cap)
        assert L().cb_last_error() == 0
        assert counts.tolist() == [live, len(moves)]
        assert np.array_equal(block_map.cpu().numpy(), want_map)
        outside, self.outside = self.outside, np.zeros(nb, np.int64)
        for b in np.flatnonzero(outside):
            self.outside[want_map[b]] += outside[b]
        want = np.full((cap, 2), -1)
        want[:len(moves)] = moves
        assert np.array_equal(pairs.cpu().numpy(), want)
        self.same()
        return pairs

    def same(self):
        assert np.array_equal(self.d_tables.cpu().numpy(), self.tables)
        assert np.array_equal(self.d_lens.cpu().numpy(), self.lens)
        assert np.array_equal(self.d_refs.cpu().numpy(), self.refs)


SIZES = [
    # rows, longest, blocks, group, shared blocks
    (1, 1, 1, 1, 0),
    (3, 40, 30, 1, 0),
    (8, 100, 100, 4, 2),
    (64, 300, 2000, 8, 5),
    (65, 300, 8193, 5, 5),         # one row and one block past what a single CTA takes
    (300, 900, 40001, 6, 10),
    (2048, 60, 20000, 8, 1),
]


def _pool(size, seed, **kw):
    n, longest, blocks, group, shared = size
    rng = np.random.default_rng(seed + 1)
    lens = rng.integers(0, longest + 1, n) + shared * BS
    lens[rng.random(n) < 0.2] //= BS * BS       # whole and empty ones
    return Pool(lens, max(blocks, 1), seed, group, shared, **kw), rng


@pytest.mark.parametrize("size", SIZES)
def test_fork_random(size):
    p, rng = _pool(size, 3)
    n, group = size[0], size[3]
    for step in range(4):
        first = np.arange(n) // group * group
        parents = np.minimum(first + rng.integers(0, group, n), n - 1)
        if step == 1:
            parents[rng.random(n) < 0.3] = -1
        if step == 2:
            parents = rng.integers(-1, n, n)                      # any row from any
        keep = None if step == 0 else np.where(rng.random(n) < 0.5, -1, rng.integers(0, size[1] + 200, n))
        p.fork(parents, keep)
        if len(p.refs) > 4 * n:
            ob.check(p.tables, p.lens, p.refs)


@pytest.mark.parametrize("size", SIZES)
def test_grow_random(size):
    p, rng = _pool(size, 4)
    n = size[0]
    for q in (np.ones(n, int), rng.integers(0, 40, n), np.zeros(n, int), rng.integers(0, 3, n)):
        p.grow(q, pad=int(rng.integers(0, 5)))


@pytest.mark.parametrize("size", SIZES)
def test_compact_random(size):
    p, rng = _pool(size, 5, outside=rng_blocks(size))
    p.compact(max_pairs=3)
    p.compact()
    pairs = p.compact()                                            # nothing left to move
    assert (pairs == -1).all()
    n = size[0]
    p.fork(np.where(rng.random(n) < 0.4, -1, np.arange(n)))
    p.compact()
    p.grow(rng.integers(0, 20, n))
    ob.check(p.tables, p.lens, p.refs, p.outside)


def rng_blocks(size):
    """Blocks that something other than the tables holds."""
    return np.random.default_rng(size[2]).integers(0, max(size[2], 1), min(5, size[2]))


def test_fork_of_prefixes():
    """Kept lengths on every place of a block, of a parent that goes on and of one that ends."""
    for parent_goes_on in (True, False):
        n = 36
        lens = [50] + [0] * (n - 1)
        p = Pool(lens, 200, 7)
        parents = np.zeros(n, int)
        if not parent_goes_on:
            parents[0] = -1
        p.fork(parents, np.array([-1] + list(range(14, 14 + n - 1))))
        ob.check(p.tables, p.lens, p.refs)
        p.fork(np.arange(n), np.arange(n) // 2)                      # cut in place
        ob.check(p.tables, p.lens, p.refs)


def test_fork_when_blocks_run_out():
    for n, blocks in ((6, 4), (70, 40)):
        p = Pool([40] + [0] * (n - 1), blocks, 1)
        p.fork(np.zeros(n, int))
        assert (p.refs[p.refs > 0].sum() == sum(ob.n_blocks(x) for x in p.lens)) and (p.lens == 32).any()


def test_grow_when_blocks_run_out():
    for blocks, width in ((12, None), (9000, None), (9000, 1200)):
        p = Pool([16] * 8 + [3] * 2, blocks, 1, width=width)
        status, stay = p.grow([16 * (blocks // 8)] * 8 + [1, 1])
        # (9000 blocks and a table of 3 entries a row: the rows outgrow their tables first)
        assert status == (L().CB_EDEVICE if blocks == 9000 and width is None else L().CB_ESTATE)
        assert stay and stay[-1] < 8                                 # rows without need grow all the same


def test_a_row_that_would_outgrow_its_table_stays():
    p = Pool([30, 30, 30], 20, 1, width=3)
    cu = torch.tensor([0, 18, 37, 38], dtype=torch.int32, device="cuda")
    slots = torch.zeros(38, dtype=torch.int64, device="cuda")
    ctx = torch.zeros(3, dtype=torch.int32, device="cuda")
    L().cb_grow_blocks(cu, p.d_tables, p.d_lens, p.d_refs, ctx, slots, p.ws)
    assert L().cb_last_error() == L().CB_EDEVICE
    assert p.d_lens.tolist() == [48, 30, 31]
    assert (slots[18:37] == -1).all() and (slots[:18] >= 0).all() and int(slots[37]) >= 0
    assert int(p.d_refs.sum()) == 7


def test_entries_let_go_of_by_a_window():
    """Entries of -1 name no block: forked, freed and moved with the rest."""
    p = Pool([100, 100, 0], 40, 2)
    for r in range(2):
        for c in range(3):
            e = p.tables[r, c]
            p.refs[e] -= 1
            p.tables[r, c] = -1
    p.d_tables.copy_(torch.from_numpy(p.tables))
    p.d_refs.copy_(torch.from_numpy(p.refs))
    p.fork([0, 0, 1])
    p.grow([1, 20, 3])
    p.compact()
    p.fork([-1, 1, -1])
    ob.check(p.tables, p.lens, p.refs)


def test_bad_metadata_is_reported_and_harmless():
    """Ids and lengths out of range: no access through them, an error, the other rows as ever."""
    lib = L()
    p = Pool([40, 40, 40], 30, 2)
    p.d_tables[1, 1] = 30                                            # past the pool
    p.d_lens[2] = 1 << 30                                            # past the table
    pairs = torch.zeros(3, 2, dtype=torch.int32, device="cuda")
    i = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    lib.cb_fork_blocks(i(0, 1, 5), None, p.d_tables, p.d_lens, p.d_refs, pairs, p.ws)
    assert lib.cb_last_error() == lib.CB_EDEVICE
    assert p.d_lens.tolist() == [40, 40, 0]
    p = Pool([40, 40, 40], 30, 2)
    p.d_lens[1] = -5
    p.d_tables[0, 2] = 1 << 20
    slots, ctx = torch.zeros(9, dtype=torch.int64, device="cuda"), i(0, 0, 0)
    lib.cb_grow_blocks(i(0, 3, 6, 9), p.d_tables, p.d_lens, p.d_refs, ctx, slots, p.ws)
    assert lib.cb_last_error() == lib.CB_EDEVICE
    assert slots[:6].tolist() == [-1] * 6 and int(slots[8]) == int(p.tables[2, 2]) * BS + 10
    for cu in ((0, 5, 3, 9), (0, 3, 6, 90), (-2, 3, 6, 9)):
        p = Pool([40, 40, 40], 30, 2)
        lib.cb_grow_blocks(i(*cu), p.d_tables, p.d_lens, p.d_refs, ctx, slots, p.ws)
        assert lib.cb_last_error() == lib.CB_EDEVICE
    p = Pool([40, 40, 40], 30, 2)
    p.d_tables[0, 0] = 31
    m, ct = torch.zeros(30, dtype=torch.int32, device="cuda"), i(0, 0)
    lib.cb_compact_blocks(p.d_tables, p.d_lens, p.d_refs, m, torch.zeros(15, 2, dtype=torch.int32, device="cuda"), ct, p.ws)
    assert lib.cb_last_error() == lib.CB_EDEVICE and int(p.d_tables[0, 0]) == 31
    caches = [torch.zeros(2, 4, 16, device="cuda")]
    lib.cb_copy_blocks_layers(torch.tensor([[1, 4], [9, 0], [-1, 3], [2, -1]], dtype=torch.int32, device="cuda"), caches)
    assert lib.cb_last_error() == lib.CB_EDEVICE and not caches[0].any()


def test_slots_of_a_row_whose_length_is_out_of_range():
    """Many tokens, and a length past the table that is just its nearest length plus the new tokens: the row has not
    grown, and nothing behind its table row is read."""
    lib = L()
    p = Pool([20, 0], 700, 3, width=600)
    p.d_lens[1] = 600 * BS + 9000
    cu = torch.tensor([0, 3, 9003], dtype=torch.int32, device="cuda")
    slots = torch.zeros(9003, dtype=torch.int64, device="cuda")
    ctx = torch.zeros(2, dtype=torch.int32, device="cuda")
    lib.cb_grow_blocks(cu, p.d_tables, p.d_lens, p.d_refs, ctx, slots, p.ws)
    assert lib.cb_last_error() == lib.CB_EDEVICE
    assert (slots[:3] >= 0).all() and (slots[3:] == -1).all() and p.d_lens.tolist() == [23, 600 * BS + 9000]


def test_many_tokens_recorded():
    """Growth by more tokens than one cluster gives slots to, recorded and replayed."""
    lib = L()
    p = Pool([0, 5, 100], 3000, 4, width=900)
    q = np.array([4000, 3000, 3500])
    cu = torch.from_numpy(np.concatenate([[0], np.cumsum(q)]).astype(np.int32)).cuda()
    slots = torch.zeros(10500 + 7, dtype=torch.int64, device="cuda")
    ctx = torch.zeros(3, dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        call = lambda: lib.cb_grow_blocks(cu, p.d_tables, p.d_lens, p.d_refs, ctx, slots, p.ws)  # noqa: E731
        call()
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            call()
        graph.replay()
        assert lib.cb_last_error(s) == 0
    for _ in range(2):
        want_ctx, want, _ = ob.grow(q, p.tables, p.lens, p.refs)
    assert np.array_equal(slots.cpu().numpy(), np.concatenate([want, [-1] * 7]))
    assert np.array_equal(ctx.cpu().numpy(), want_ctx)
    p.same()


@pytest.mark.parametrize("layers,blocks,shapes,n", [
    (1, 5, [(2, 16, 64)], 2),
    (3, 40, [(1, 16, 128), (1, 16, 128), (1, 16), (1, 16)], 17),
    (2, 5000, [(2, 16, 64)], 2300),                                # more pairs than a tile of them
    (7, 64, [(5, 16, 128), (3, 32)], 31),
    (32, 24, [(8, 16, 128), (8, 16, 128)], 12),
])
def test_copies(layers, blocks, shapes, n):
    g = torch.Generator(device="cuda").manual_seed(n)
    rng = np.random.default_rng(n)
    caches = []
    for k, s in enumerate(shapes):
        t = torch.randint(0, 256, (layers, blocks, *s), device="cuda", generator=g, dtype=torch.uint8)
        caches.append(t.to(torch.bfloat16) if k % 2 == 0 and len(s) == 3 else t)
    want = [t.clone() for t in caches]
    ids = rng.permutation(blocks)
    pairs = np.stack([ids[:n], ids[n:2 * n]], 1)
    pairs[rng.random(n) < 0.3, 0] = -1
    for src, dst in pairs:
        if src >= 0:
            for t in want:
                t[:, dst] = t[:, src]
    L().cb_copy_blocks_layers(torch.from_numpy(pairs.astype(np.int32)).cuda(), caches)
    assert L().cb_last_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(caches, want))


def test_copies_past_4_gib():
    """Offsets of more than 32 bits: the last block of the last layer."""
    t = torch.zeros(3, 50000, 2, 16, 1024, dtype=torch.uint8, device="cuda")        # 4.9 GB
    t[2, 7] = 5
    t[0, 7] = 3
    L().cb_copy_blocks_layers(torch.tensor([[7, 49999]], dtype=torch.int32, device="cuda"), [t])
    assert L().cb_last_error() == 0
    assert (t[2, 49999] == 5).all() and (t[0, 49999] == 3).all() and not t[1, 49999].any()


def test_on_another_stream_and_recorded():
    """A beam step recorded as a graph and replayed follows the oracle step by step."""
    lib = L()
    p = Pool([33] * 8, 100, 9, group=4, shared=2)
    parents = torch.zeros(8, dtype=torch.int32, device="cuda")
    pairs = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    cu = torch.arange(9, dtype=torch.int32, device="cuda")
    ctx, slots = torch.zeros(8, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int64, device="cuda")
    cache = torch.arange(100, device="cuda").view(1, 100, 1).expand(2, 100, 16).contiguous()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())

    def step():
        lib.cb_fork_blocks(parents, None, p.d_tables, p.d_lens, p.d_refs, pairs, p.ws)
        lib.cb_copy_blocks_layers(pairs, [cache])
        lib.cb_grow_blocks(cu, p.d_tables, p.d_lens, p.d_refs, ctx, slots, p.ws)

    def oracle(pa):
        want, _ = ob.fork(pa, None, p.tables, p.lens, p.refs)
        for src, dst in want:
            if src >= 0:
                content[dst] = content[src]
        return ob.grow([1] * 8, p.tables, p.lens, p.refs)[1]

    content = np.arange(100)
    rng = np.random.default_rng(0)
    with torch.cuda.stream(s):
        parents.copy_(torch.arange(8))
        step()
        oracle(np.arange(8))
        s.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            step()
        for _ in range(40):
            pa = np.arange(8) // 4 * 4 + rng.integers(0, 4, 8)
            parents.copy_(torch.from_numpy(pa.astype(np.int32)))
            graph.replay()
            want = oracle(pa)
            s.synchronize()
            assert np.array_equal(slots.cpu().numpy(), want)
            p.same()
            assert np.array_equal(cache[1, :, 3].cpu().numpy(), content)
        assert lib.cb_last_error(s) == 0


def test_results_do_not_depend_on_the_run():
    outs = []
    for _ in range(3):
        p, rng = _pool(SIZES[5], 11)
        n = len(p.lens)
        p.fork(rng.integers(0, n, n), rng.integers(0, 900, n))
        outs.append(p.d_tables.clone())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


def test_no_rows():
    lib = L()
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    ws = torch.zeros(lib.cb_block_ops_workspace_size(0, 4, 8), dtype=torch.uint8, device="cuda")
    lib.cb_fork_blocks(i(0), None, i(0, 4), i(0), i(8), i(0, 2), ws)
    lib.cb_grow_blocks(i(1), i(0, 4), i(0), i(8), i(0), torch.zeros(0, dtype=torch.int64, device="cuda"), ws)
    refs, m, pairs, ct = i(8), i(8), i(4, 2), i(2)
    refs[5] = 2                                                    # a pool that only others hold blocks of
    lib.cb_compact_blocks(i(0, 4), i(0), refs, m, pairs, ct, ws)
    lib.cb_copy_blocks_layers(i(0, 2), [torch.zeros(1, 8, 16, device="cuda")])
    assert lib.cb_last_error() == 0
    assert refs.tolist() == [2] + [0] * 7 and pairs[0].tolist() == [5, 0] and ct.tolist() == [1, 1]


def test_binding_refusals():
    lib = L()
    p = Pool([20, 20], 9, 1)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
    pool = (p.d_tables, p.d_lens, p.d_refs)
    slots = torch.zeros(2, dtype=torch.int64, device="cuda")
    for call in (
            lambda: lib.cb_fork_blocks(i(3), None, *pool, i(2, 2), p.ws),
            lambda: lib.cb_fork_blocks(i(2), i(3), *pool, i(2, 2), p.ws),
            lambda: lib.cb_fork_blocks(i(2), None, *pool, i(2, 3), p.ws),
            lambda: lib.cb_fork_blocks(i(2).long(), None, *pool, i(2, 2), p.ws),
            lambda: lib.cb_grow_blocks(i(2), *pool, i(2), slots, p.ws),
            lambda: lib.cb_grow_blocks(i(3), *pool, i(2), i(2), p.ws),
            lambda: lib.cb_grow_blocks(i(3), p.d_tables.t(), p.d_lens, p.d_refs, i(2), slots, p.ws),
            lambda: lib.cb_compact_blocks(*pool, i(8), i(4, 2), i(2), p.ws),
            lambda: lib.cb_compact_blocks(*pool, i(9), i(4, 2), i(3), p.ws),
            lambda: lib.cb_copy_blocks_layers(i(1, 2), []),
            lambda: lib.cb_copy_blocks_layers(i(1, 2), torch.zeros(2, 8, 4, 16, device="cuda")),
            lambda: lib.cb_copy_blocks_layers(i(1, 2), [torch.zeros(2, 8, 16, device="cuda")] * 9),
            lambda: lib.cb_copy_blocks_layers(i(1, 2), [torch.zeros(2, 8, device="cuda")]),
            lambda: lib.cb_copy_blocks_layers(i(1, 2), [torch.zeros(2, 8, 16, device="cuda"), torch.zeros(2, 9, 16, device="cuda")]),
    ):
        with pytest.raises(ValueError):
            call()
    with pytest.raises(lib.CBError):
        lib.cb_fork_blocks(i(2), None, *pool, i(2, 2), p.ws[:16])
    with pytest.raises(lib.CBError):                               # 72 bytes: not a multiple of 16
        lib.cb_copy_blocks_layers(i(1, 2), [torch.zeros(7, 64, 3, 24, dtype=torch.uint8, device="cuda")])
