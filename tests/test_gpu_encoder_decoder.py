"""The cross attention and the block pool as a decoder uses them: beam search over
encoder states, every step on the device and recorded as one graph."""
import math

import numpy as np
import pytest
import torch

from gpu_util import L
from oracle import blocks as ob

pytestmark = pytest.mark.gpu

BS, LAYERS, REQS, BEAMS, HQ, HK, A = 16, 2, 3, 4, 8, 4, 64
ROWS = REQS * BEAMS


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _attend(q, k, v, scale):
    """q [Hq, A], k and v [Hkv, n, A], float64 -> [Hq, A] and the sum of the weights times |v|."""
    g = q.shape[0] // k.shape[0]
    s = torch.einsum("hgd,hnd->hgn", q.view(k.shape[0], g, -1), k) * scale
    p = torch.softmax(s, -1)
    return torch.einsum("hgn,hnd->hgd", p, v).reshape(q.shape), torch.einsum("hgn,hnd->hgd", p, v.abs()).reshape(q.shape)


def test_beam_search_over_encoder_states():
    """Each step: rows grow by a token, each layer stores its K/V and attends to them, then to the encoder's states;
    beams are then reordered by parents that only the device knows, with the copies of every layer, and in the end the
    pool is compacted.  Every row's outputs are those of its own history of tokens, kept as plain lists."""
    lib = L()
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda *s: torch.randn(*s, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    i32 = lambda a: torch.tensor(a, dtype=torch.int32, device="cuda")  # noqa: E731
    enc = [70, 33, 0]                                        # the last request has an empty document
    nb, width, scale = 80, 8, 1.0 / math.sqrt(A)
    k_self, v_self = torch.zeros(2, LAYERS, nb, HK, BS, A, device="cuda", dtype=torch.bfloat16).unbind(0)
    tables, lens, refs = i32(np.full((ROWS, width), -1)), i32([0] * ROWS), i32([0] * nb)
    ws = torch.empty(lib.cb_block_ops_workspace_size(ROWS, width, nb), dtype=torch.uint8, device="cuda")
    # the encoder's states: every beam of a request is a token of that request's cross attention
    need = [-(-n // BS) for n in enc]
    e_tables = np.full((REQS, max(need)), -1, np.int32)
    e_tables[0, :need[0]] = np.arange(need[0])
    e_tables[1, :need[1]] = need[0] + np.arange(need[1])
    k_enc, v_enc = rnd(LAYERS, sum(need) + 1, HK, BS, A), rnd(LAYERS, sum(need) + 1, HK, BS, A)
    cu_enc, kv_enc, e_tab = i32([r * BEAMS for r in range(REQS + 1)]), i32(enc), torch.from_numpy(e_tables).cuda()
    cross_ws = torch.empty(lib.cb_paged_cross_attention_workspace_size(ROWS, ROWS, BEAMS, max(enc), HQ, HK, A, BS),
                           dtype=torch.uint8, device="cuda")
    self_ws = torch.empty(lib.cb_paged_attention_workspace_size(ROWS, ROWS, 1, width * BS, HQ, HK, A, BS),
                          dtype=torch.uint8, device="cuda")
    cu = i32(range(ROWS + 1))
    ctx, slots = i32([0] * ROWS), torch.zeros(ROWS, dtype=torch.int64, device="cuda")
    parents, pairs = i32([0] * ROWS), i32(np.zeros((ROWS, 2)))
    k_new, v_new, q = (rnd(LAYERS, ROWS, h, A) for h in (HK, HK, HQ))
    out, cross = torch.zeros_like(q), torch.zeros_like(q)
    caches = [k_self, v_self]

    def step():
        lib.cb_fork_blocks(parents, None, tables, lens, refs, pairs, ws)
        lib.cb_copy_blocks_layers(pairs, caches)
        lib.cb_grow_blocks(cu, tables, lens, refs, ctx, slots, ws)
        for layer in range(LAYERS):
            lib.cb_kv_append_paged_attention(k_new[layer], v_new[layer], slots, q[layer], cu, ctx, tables, k_self[layer],
                                             v_self[layer], out[layer], scale, self_ws, 1, width * BS)
            lib.cb_paged_cross_attention(out[layer], cu_enc, kv_enc, e_tab, k_enc[layer], v_enc[layer], cross[layer], scale,
                                         cross_ws, BEAMS, max(enc))

    history = [[] for _ in range(ROWS)]                      # (k, v) of every layer, of each of a row's tokens
    rng = np.random.default_rng(2)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        graph = None
        for t in range(45):
            pa = np.arange(ROWS) if t < 2 else np.arange(ROWS) // BEAMS * BEAMS + rng.integers(0, BEAMS, ROWS)
            for x in (k_new, v_new, q):
                x.copy_(rnd(*x.shape))
            parents.copy_(torch.from_numpy(pa.astype(np.int32)))
            history = [list(history[p]) for p in pa]
            for r in range(ROWS):
                history[r].append((k_new[:, r].double(), v_new[:, r].double()))
            if t < 2:
                step()
            else:
                if graph is None:
                    s.synchronize()
                    graph = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(graph, stream=s):
                        step()
                graph.replay()
            assert lib.cb_last_error(s) == 0
            assert lens.tolist() == [t + 1] * ROWS
            ob.check(tables.cpu().numpy().astype(np.int64), lens.cpu().numpy(), refs.cpu().numpy())
            if t % 6 and t < 40:
                continue
            for layer in range(LAYERS):
                for r in range(ROWS):
                    k = torch.stack([h[0][layer] for h in history[r]], 1)
                    v = torch.stack([h[1][layer] for h in history[r]], 1)
                    ref, size = _attend(q[layer, r].double(), k, v, scale)
                    # the output's and the weights' rounding to bf16, 2^-8 each; sums in fp32 are far below 2^-12
                    assert ((out[layer, r].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * size).all()
                    n = enc[r // BEAMS]
                    if not n:
                        assert not cross[layer, r].any()
                        continue
                    blk = e_tab[r // BEAMS, :-(-n // BS)].long()
                    k, v = (x[layer][blk].transpose(0, 1).reshape(HK, -1, A)[:, :n].double() for x in (k_enc, v_enc))
                    ref, size = _attend(out[layer, r].double(), k, v, scale)
                    assert ((cross[layer, r].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -12) * size).all()
        # requests 0 and 2 end; the pool is compacted, and request 1 goes on reading its tokens
        parents.copy_(torch.from_numpy(np.where(np.arange(ROWS) // BEAMS == 1, np.arange(ROWS), -1).astype(np.int32)))
        lib.cb_fork_blocks(parents, None, tables, lens, refs, pairs, ws)
        lib.cb_copy_blocks_layers(pairs, caches)
        block_map, moves, counts = i32([0] * nb), i32(np.zeros((nb // 2, 2))), i32([0, 0])
        lib.cb_compact_blocks(tables, lens, refs, block_map, moves, counts, ws)
        lib.cb_copy_blocks_layers(moves, caches)
        assert lib.cb_last_error(s) == 0
        live, _ = counts.tolist()
        assert live == int((refs > 0).sum()) and not refs[live:].any()
        ob.check(tables.cpu().numpy().astype(np.int64), lens.cpu().numpy(), refs.cpu().numpy())
        for r in range(BEAMS, 2 * BEAMS):
            for pos, (k, v) in enumerate(history[r]):
                e = int(tables[r, pos // BS])
                assert torch.equal(k_self[:, e, :, pos % BS].double(), k) and torch.equal(v_self[:, e, :, pos % BS].double(), v)


def test_drafts_cut_back():
    """Drafted tokens are stored, and the ones that do not stand are cut off by lengths that the device holds."""
    lib = L()
    rng = np.random.default_rng(3)
    n, nb, width = 7, 90, 12
    tables, lens, refs = np.full((n, width), -1, np.int64), np.zeros(n, np.int64), np.zeros(nb, np.int64)
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()  # noqa: E731
    d = [i32(tables), i32(lens), i32(refs)]
    ws = torch.empty(lib.cb_block_ops_workspace_size(n, width, nb), dtype=torch.uint8, device="cuda")
    ctx, pairs = i32(lens), i32(np.zeros((n, 2)))
    for _ in range(25):
        draft = rng.integers(0, 9, n)
        slots = torch.zeros(int(draft.sum()), dtype=torch.int64, device="cuda")
        lib.cb_grow_blocks(i32(np.concatenate([[0], np.cumsum(draft)])), *d, ctx, slots, ws)
        want = ob.grow(draft, tables, lens, refs)[1]
        assert np.array_equal(slots.cpu().numpy(), want)
        keep = np.maximum(lens - rng.integers(0, 5, n), 0)
        lib.cb_fork_blocks(i32(np.arange(n)), i32(keep), *d, pairs, ws)
        ob.fork(np.arange(n), keep, tables, lens, refs)
        assert (pairs == -1).all() and lib.cb_last_error() == 0
        for got, w in zip(d, (tables, lens, refs)):
            assert np.array_equal(got.cpu().numpy(), w)
        if (lens > 150).any():
            break
