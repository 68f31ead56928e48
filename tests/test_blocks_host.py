"""The block pool without a GPU: the oracle pinned by hand, and what the entry
points refuse before anything is enqueued."""
import ctypes
import math
import os

import numpy as np
import pytest
import torch

from oracle import blocks as ob
from test_fp8_host import _Fake


def _lib():
    from paged_kv_cache_cb_gb300 import _lib as L
    if not os.path.exists(L.LIB_PATH):
        from paged_kv_cache_cb_gb300 import build
        build.build()
    return L


# ------------------------------------------------------------------ the oracle
def _pool(rows, num_blocks, width=6):
    """Rows as (length, blocks)."""
    tables = np.full((len(rows), width), -1, np.int64)
    refs = np.zeros(num_blocks, np.int64)
    for r, (n, blocks) in enumerate(rows):
        tables[r, :len(blocks)] = blocks
        for b in blocks:
            refs[b] += 1
    return tables, np.array([n for n, _ in rows], np.int64), refs


def test_fork_worked_by_hand():
    # two beams of one prompt: block 4 shared, 7 and 2 their own partial ones
    tables, lens, refs = _pool([(20, [4, 7]), (20, [4, 2])], 9)
    pairs, cut = ob.fork([1, 1], None, tables, lens, refs)
    assert tables[:, :2].tolist() == [[4, 2], [4, 0]]        # row 0 keeps block 2, row 1 has a copy in the lowest free
    assert pairs.tolist() == [[-1, -1], [2, 0]] and not cut
    assert refs[[0, 2, 4, 7]].tolist() == [1, 1, 2, 0]
    # a prefix of a row that goes on: the row itself keeps what it will write
    tables, lens, refs = _pool([(40, [1, 2, 3]), (0, [])], 5)
    pairs, cut = ob.fork([0, 0], [-1, 18], tables, lens, refs)
    assert tables[1, :2].tolist() == [1, 0] and pairs.tolist() == [[-1, -1], [2, 0]]   # block 2 is whole in row 0
    # freed, and cut to whole blocks where no block is left for the copy
    tables, lens, refs = _pool([(20, [0, 1]), (0, [])], 2)
    pairs, cut = ob.fork([0, 0], None, tables, lens, refs)
    assert cut == [1] and lens.tolist() == [20, 16] and refs.tolist() == [2, 1]
    assert tables[1, :2].tolist() == [0, -1]
    ob.fork([-1, -1], None, tables, lens, refs)
    assert lens.tolist() == [0, 0] and not refs.any() and (tables == -1).all()


def test_grow_worked_by_hand():
    tables, lens, refs = _pool([(15, [3]), (16, [1]), (0, [])], 6)
    ctx, slots, stay = ob.grow([1, 1, 17], tables, lens, refs)
    assert lens.tolist() == [16, 17, 17] and ctx.tolist() == [15, 16, 0] and not stay
    assert tables[1, 1] == 0 and tables[2, :2].tolist() == [2, 4]
    assert slots.tolist() == [3 * 16 + 15, 0] + [2 * 16 + i for i in range(16)] + [64]
    ctx, slots, stay = ob.grow([16, 1, 2], tables, lens, refs)      # one block left: row 0 takes it
    assert stay == [] and tables[0, 1] == 5
    ctx, slots, stay = ob.grow([1, 1, 1], tables, lens, refs)       # none left: row 0 stays
    assert stay == [0] and slots.tolist() == [-1, 2, 4 * 16 + 3]


def test_compact_worked_by_hand():
    tables, lens, refs = _pool([(30, [5, 0]), (20, [5, 6])], 8)
    block_map, moves, live = ob.compact(tables, lens, refs)
    assert live == 3 and moves.tolist() == [[5, 1], [6, 2]]
    assert tables[:, :2].tolist() == [[1, 0], [1, 2]] and refs.tolist() == [1, 2, 1, 0, 0, 0, 0, 0]
    assert block_map.tolist() == [0, -1, -1, -1, -1, 1, 2, -1]


# ------------------------------------------------------------------ refusals of the C ABI
D = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4098)


def test_pool_arguments():
    L = _lib().lib()

    def fork(pa=D, ke=None, bt=D, w=4, n=2, ln=D, rf=D, nb=8, bs=16, pr=D, ws=D, wsb=1 << 20):
        return L.cb_fork_blocks(pa, ke, bt, w, n, ln, rf, nb, bs, pr, ws, wsb, None)

    def grow(pa=D, bt=D, w=4, n=2, ln=D, rf=D, nb=8, bs=16, ctx=D, sl=D, nt=3, ws=D, wsb=1 << 20):
        return L.cb_grow_blocks(pa, bt, w, n, ln, rf, nb, bs, ctx, sl, nt, ws, wsb, None)

    def compact(bt=D, w=4, n=2, ln=D, rf=D, nb=8, bs=16, mp=D, pr=D, m=4, ct=D, ws=D, wsb=1 << 20):
        return L.cb_compact_blocks(bt, w, n, ln, rf, nb, bs, mp, pr, m, ct, ws, wsb, None)

    for f in (fork, grow):
        assert f(n=0) == 0
        assert f(pa=None) == -1 and f(pa=ODD) == -1
    for f in (fork, grow, compact):
        for bad in (dict(n=-1), dict(n=2049), dict(w=0), dict(nb=0), dict(bs=32), dict(bt=None), dict(ln=None), dict(rf=None),
                    dict(bt=ODD), dict(ln=ODD), dict(rf=ODD), dict(ws=None), dict(ws=ctypes.c_void_p(4100)),
                    dict(w=1 << 30), dict(w=1 << 27, n=1)):
            assert f(**bad) == -1, (f.__name__, bad)
    assert fork(pr=None) == -1 and fork(pr=ODD) == -1 and fork(ke=ODD) == -1 and fork(wsb=8) == -3
    assert grow(ctx=None) == -1 and grow(sl=None) == -1 and grow(sl=ctypes.c_void_p(4100)) == -1 and grow(nt=-1) == -1
    assert grow(wsb=8) == -3
    assert compact(mp=None) == -1 and compact(pr=None) == -1 and compact(m=-1) == -1 and compact(ct=None) == -1
    assert compact(pr=ODD) == -1 and compact(wsb=8) == -3


def test_workspace_size():
    L = _lib()
    f = L.cb_block_ops_workspace_size
    assert f(-1, 4, 8) == 0 and f(2049, 4, 8) == 0 and f(4, 0, 8) == 0 and f(4, 4, 0) == 0 and f(4, 4, 8, 32) == 0
    assert f(0, 4, 8) > 0
    assert f(2048, 100, 8) >= 2048 * 100 * 4 and f(1, 1, 1 << 20) >= (1 << 20) * 4
    with pytest.raises(ValueError):
        f(1 << 33, 4, 8)


def test_copy_arguments():
    L = _lib().lib()

    def copy(p=D, n=1, ptrs=(4096, 8192), sizes=(64, 16), k=None, layers=2, nb=8):
        a, b = (ctypes.c_void_p * len(ptrs))(*ptrs), (ctypes.c_size_t * len(sizes))(*sizes)
        return L.cb_copy_blocks_layers(p, n, a, b, len(ptrs) if k is None else k, layers, nb, None)

    assert copy(n=0) == 0
    for bad in (dict(n=-1), dict(k=0), dict(k=9), dict(layers=0), dict(nb=0), dict(ptrs=(None, 4096)), dict(ptrs=(4100, 8192)),
                dict(sizes=(24, 16)), dict(sizes=(64, 0)), dict(p=None), dict(p=ODD), dict(sizes=(1 << 30, 16))):
        assert copy(**bad) == -1, bad
    assert L.cb_copy_blocks_layers(D, 1, None, None, 1, 1, 1, None) == -1


def test_binding_refuses_host_tensors():
    L = _lib()
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    ws = torch.zeros(4096, dtype=torch.uint8)
    with pytest.raises(ValueError):
        L.cb_fork_blocks(i(2), None, i(2, 4), i(2), i(8), i(2, 2), ws)
    with pytest.raises(ValueError):
        L.cb_grow_blocks(i(3), i(2, 4), i(2), i(8), i(2), torch.zeros(3, dtype=torch.int64), ws)
    with pytest.raises(ValueError):
        L.cb_compact_blocks(i(2, 4), i(2), i(8), i(8), i(4, 2), i(2), ws)
    with pytest.raises(ValueError):
        L.cb_copy_blocks_layers(i(1, 2), [torch.zeros(1, 8, 16)])


# ------------------------------------------------------------------ cross attention's arguments
def test_cross_attention_arguments():
    L = _lib().lib()

    def cross(q=D, cu=D, kv=D, bt=D, w=4, n=2, nt=3, mq=2, mkv=40, k=D, v=D, nb=16, out=D, scale=0.1, hq=8, hk=4, a=128, bs=16,
              ws=D, wsb=1 << 30):
        return L.cb_paged_cross_attention(q, cu, kv, bt, w, n, nt, mq, mkv, k, v, nb, out, scale, hq, hk, a, bs, ws, wsb, None)

    assert cross(n=0) == 0 and cross(nt=0) == 0
    for bad in (dict(hq=6), dict(hq=12), dict(hq=256), dict(hk=0), dict(a=96), dict(bs=32), dict(n=-1), dict(n=2049),
                dict(nt=-1), dict(mq=0), dict(mkv=-1), dict(w=0), dict(nb=0), dict(nb=1 << 29), dict(scale=0.0),
                dict(scale=float("nan")), dict(mkv=0x7FFFFFFF, nt=1 << 20), dict(q=None), dict(cu=None), dict(kv=None),
                dict(bt=None), dict(k=None), dict(v=None), dict(out=None), dict(ws=None), dict(q=ODD), dict(k=ODD), dict(v=ODD),
                dict(out=ODD), dict(ws=ODD)):
        assert cross(**bad) == -1, bad
    assert cross(wsb=16) == -3


def test_cross_attention_workspace_size():
    f = _lib().cb_paged_cross_attention_workspace_size
    assert f(2, 3, 1, 40, 8, 4, 128, 16) == 320 * 4 * 130 * 4        # two rows of a token, four kept
    assert f(2, 3, 1 << 20, 40, 8, 4, 64, 16) == 320 * 256 * 66 * 4
    assert f(2, 3, 1, 0, 32, 1, 128, 16) > 0
    for bad in ((-1, 3, 1, 40, 8, 4, 128, 16), (2, -1, 1, 40, 8, 4, 128, 16), (2, 3, 0, 40, 8, 4, 128, 16),
                (2, 3, 1, -1, 8, 4, 128, 16), (2, 3, 1, 40, 24, 8, 128, 16), (2, 3, 1, 40, 8, 4, 80, 16), (2, 3, 1, 40, 8, 4, 128, 8)):
        assert f(*bad) == 0
    with pytest.raises(ValueError):
        f(2, 3, 1 << 40, 40, 8, 4, 128, 16)


@pytest.mark.parametrize("n,nt,hk,mkv,want", [
    (1, 0x7FFFFFFF, 1 << 26, 524288, -1),           # the product of groups, KV heads and key tiles passes 63 bits
    (1, 0x7FFFFFFF, 1 << 26, 1 << 30, -1),
    (2048, 0x7FFFFFFF, 1 << 26, 0, -1),
    (2, 1 << 20, 4, 1 << 30, -1),
    (2, 256 * 2046, 1 << 12, 3841, -1),             # 2^23 items of 6 + 4 * 31 units
    (2, 256 * 2046, 1 << 12, 3840, -3),             # of 126: fewer than 2^30 in all; the workspace is too small
])
def test_cross_attention_work_is_bounded(n, nt, hk, mkv, want):
    L = _lib().lib()
    assert L.cb_paged_cross_attention(D, D, D, D, 4, n, nt, 1, mkv, D, D, 1, D, 0.1, hk, hk, 64, 16, D, 16, None) == want


def test_pairs_that_32_bits_cannot_index():
    """The kernels count the ints of pairs in 32 bits: 2^30 pairs are the most."""
    L = _lib().lib()
    a, b = (ctypes.c_void_p * 1)(4096), (ctypes.c_size_t * 1)(64)
    for n in ((1 << 30) + 1, 0x7FFFFFFF):
        assert L.cb_copy_blocks_layers(D, n, a, b, 1, 1, 8, None) == -1
        assert L.cb_compact_blocks(D, 4, 2, D, D, 8, 16, D, D, n, D, D, 1 << 20, None) == -1


def test_pools_that_32_bits_cannot_cut():
    """A CTA's share of the pool is counted in 32 bits: 2^30 blocks are the most."""
    L = _lib()
    for nb in ((1 << 30) + 1, 0x7FFFFFFF):
        assert L.lib().cb_fork_blocks(D, None, D, 4, 2, D, D, nb, 16, D, D, 1 << 40, None) == -1
        assert L.lib().cb_grow_blocks(D, D, 4, 2, D, D, nb, 16, D, D, 3, D, 1 << 40, None) == -1
        assert L.lib().cb_compact_blocks(D, 4, 2, D, D, nb, 16, D, D, 4, D, D, 1 << 40, None) == -1
        assert L.cb_block_ops_workspace_size(2, 4, nb) == 0
    assert L.cb_block_ops_workspace_size(2, 4, 1 << 30) >= 12 << 29


def test_cross_attention_workspace_of_refused_lengths():
    """No workspace for more keys than the call takes."""
    L = _lib()
    f = L.cb_paged_cross_attention_workspace_size
    assert f(2, 3, 1, 1 << 30, 8, 4, 128, 16) > 0
    for keys in ((1 << 30) + 1, 0x7FFFFFFF):
        assert f(2, 3, 1, keys, 8, 4, 128, 16) == 0


# ------------------------------------------------------------------ sizes beyond 32 bits in the binding
class _Tensor(_Fake):
    def numel(self):
        return math.prod(self.shape)

    @property
    def nbytes(self):
        return self.numel() * self.dtype.itemsize


def _made(**kw):
    i, u8, bf = torch.int32, torch.uint8, torch.bfloat16
    made = dict(pa=(i, 3), ke=(i, 3), bt=(i, 3, 4), ln=(i, 3), rf=(i, 8), pr=(i, 3, 2), cu=(i, 4), ctx=(i, 3),
                sl=(torch.int64, 5), mp=(i, 8), ct=(i, 2), ws=(u8, 1 << 20), c1=(u8, 2, 8, 64), c2=(u8, 2, 8, 16),
                q=(bf, 5, 4, 64), kv=(i, 3), k=(bf, 8, 2, 16, 64), v=(bf, 8, 2, 16, 64), out=(bf, 5, 4, 64))
    made.update(kw)
    return {name: _Tensor(*x) for name, x in made.items()}


def _step(L, f):
    pool = (f["bt"], f["ln"], f["rf"])
    return {"fork": lambda: L.cb_fork_blocks(f["pa"], f["ke"], *pool, f["pr"], f["ws"], stream=1),
            "grow": lambda: L.cb_grow_blocks(f["cu"], *pool, f["ctx"], f["sl"], f["ws"], stream=1),
            "compact": lambda: L.cb_compact_blocks(*pool, f["mp"], f["pr"], f["ct"], f["ws"], stream=1),
            "copy": lambda: L.cb_copy_blocks_layers(f["pr"], [f["c1"], f["c2"]], stream=1),
            "cross": lambda: L.cb_paged_cross_attention(f["q"], f["cu"], f["kv"], f["bt"], f["k"], f["v"], f["out"], 0.1,
                                                        f["ws"], 3, 60, stream=1)}


BIG = 1 << 32
INT, BYTE, BF = torch.int32, torch.uint8, torch.bfloat16


@pytest.mark.parametrize("calls,kw", [
    ("fork grow compact cross", dict(bt=(INT, 3, 4 + BIG))),
    ("fork grow compact", dict(rf=(INT, 8 + BIG), mp=(INT, 8 + BIG))),
    ("fork", dict(pa=(INT, 3 + BIG), ke=(INT, 3 + BIG), bt=(INT, 3 + BIG, 4), ln=(INT, 3 + BIG), pr=(INT, 3 + BIG, 2))),
    ("grow", dict(sl=(torch.int64, 5 + BIG))),
    ("grow", dict(sl=(torch.int64, 1 << 31))),
    ("compact copy", dict(pr=(INT, 3 + BIG, 2))),
    ("copy", dict(c1=(BYTE, 2 + BIG, 8, 64), c2=(BYTE, 2 + BIG, 8, 16))),
    ("copy", dict(c1=(BYTE, 2, 8 + BIG, 64), c2=(BYTE, 2, 8 + BIG, 16))),
    ("cross", dict(kv=(INT, 3 + BIG), cu=(INT, 4 + BIG), bt=(INT, 3 + BIG, 4))),
    ("cross", dict(q=(BF, 5 + BIG, 4, 64), out=(BF, 5 + BIG, 4, 64))),
    ("cross", dict(q=(BF, 5, 4 + BIG, 64), out=(BF, 5, 4 + BIG, 64))),
    ("cross", dict(k=(BF, 8 + BIG, 2, 16, 64), v=(BF, 8 + BIG, 2, 16, 64))),
    ("cross", dict(k=(BF, 8, 2 + BIG, 16, 64), v=(BF, 8, 2 + BIG, 16, 64))),
    ("cross", dict(k=(BF, 8, 2, 16 + BIG, 64), v=(BF, 8, 2, 16 + BIG, 64))),
])
def test_binding_refuses_sizes_beyond_32_bits(calls, kw, monkeypatch):
    """A pool of 2^32 + 8 blocks is not one of 8."""
    L = _lib()
    monkeypatch.setattr(L._tc(), "device", lambda: 0)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, _Fake))

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(L, "lib", Lib)
    for name in calls.split():
        _step(L, _made())[name]()
        with pytest.raises(ValueError):
            _step(L, _made(**kw))[name]()
