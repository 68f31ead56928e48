"""Attention over the 8-bit cache where items of several tokens, and single tokens
of the large groups, are cut between CTAs and joined again."""
import numpy as np
import pytest
import torch

from fp8_util import BS, Step, check
from gpu_util import L

pytestmark = pytest.mark.gpu

LEAD, JOIN_TILES = {False: 4, True: 2}, 9          # the kernel's kLead and kJoinTiles


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L().lib()


def pieces(reqs, hq, hk, window, ctas, single=False):
    """The chunk kernel's plan: (request, pair of query tiles, KV head, first key
    tile, end, piece's first tile, piece's end) of every piece, or None where items
    stay whole."""
    tok2 = 2 * 128 // (hq // hk)
    items = []
    for r, (q, c) in enumerate(reqs):
        if q == 0 or (q == 1) != single:
            continue
        for pair in range(-(-q // tok2) - 1, -1, -1):
            first = max(0, c + pair * tok2 - window + 1) // 128 if window else 0
            end = -(-(c + min(q, (pair + 1) * tok2)) // 128)
            items += [(r, pair, g, first, end) for g in range(hk)]
    lead = LEAD[single]
    total = sum(lead + e - f for *_, f, e in items)
    longest = max(e - f for *_, f, e in items)
    if longest + (-(-len(items) // ctas) - 1) * (total // len(items)) <= -(-total // ctas) + JOIN_TILES:
        return None
    eff = min(ctas, total)
    borders = {total * b // eff for b in range(eff + 1)}
    out, at = [], 0
    for item in items:
        f, e = item[3:]
        at += lead                                   # the place of its first tile
        cuts = sorted({at, at + e - f} | {b for b in borders if at < b < at + e - f})
        out += [(*item, f + x - at, f + y - at) for x, y in zip(cuts, cuts[1:])]
        at += e - f
    return out


def records(s, ws, single):
    """What a call left in its workspace of the items cut in it: (request, KV head,
    pieces, pair of query tiles)."""
    lib = L()
    first = lib.cb_paged_attention_fp8_workspace_size(1, 1, 1, 64, s.hq, s.hk, s.a, BS)     # behind the single tokens' part
    rec = ws[(0 if single else first):][:16 * _ctas()].view(torch.int32).view(-1, 4).cpu().tolist()
    return [tuple(x) for x in rec if x[2] > 1]


def _ctas():
    return min(torch.cuda.get_device_properties(0).multi_processor_count, 160)


def _cut(s, single=False):
    """The step's pieces, by the rule and by what a run has recorded."""
    p = pieces(s.reqs, s.hq, s.hk, s.window, _ctas(), single)
    assert p is not None and len(p) > 64
    ws = s.workspace()
    s.run(workspace=ws)
    count = {}
    for x in p:
        count[x[:3]] = count.get(x[:3], 0) + 1
    cut = sorted((r, g, n, 0 if single else pair) for (r, pair, g), n in count.items() if n > 1)
    assert cut and sorted((r, g, n, 0 if single else pair) for r, g, n, pair in records(s, ws, single)) == cut
    return p


SHAPES = [(4, 4, 64), (8, 4, 64), (32, 8, 64), (40, 5, 64), (32, 32, 128), (16, 8, 128), (32, 8, 128), (64, 8, 128), (8, 1, 128),
          (32, 2, 128), (32, 1, 128)]


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("reqs", [[(40, 5000)], [(2, 9000)], [(300, 3500)], [(3, 4000), (1, 700), (129, 6000), (0, 3), (2, 30)]])
def test_cut_items(hq, hk, a, reqs):
    s = Step(reqs, hq, hk, a, seed=hq + a)
    _cut(s)
    cache, meta = s.cache(), s.meta()
    out = s.run(cache=cache, meta=meta)
    check(out, *s.reference(), "cut items")
    assert torch.equal(s.run(cache=cache, meta=meta, workspace=s.workspace(fill=0x5A)), out)


def _unseen(q, c, hq, hk, window):
    """Does a piece lie before the window of one of its rows, or behind its position?"""
    tok2 = 2 * 128 // (hq // hk)
    return any(y * 128 <= c + i - window + 1 or x * 128 > c + i for _, pair, _, _, _, x, y in pieces([(q, c)], hq, hk, window, _ctas())
               for i in (pair * tok2, min(q, (pair + 1) * tok2) - 1))


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("q_len", [40, 140, 256])
def test_cut_items_under_a_window(hq, hk, a, q_len):
    """A window of more tiles than whole items may have, at a length where pieces lie
    out of sight of some of their rows (140 tokens: for every shape but the largest groups')."""
    ctx = next((c for c in range(6000, 6256) if _unseen(q_len, c, hq, hk, 4500)), None)
    assert ctx or q_len != 140 or hq // hk >= 16
    s = Step([(q_len, ctx or 6000)], hq, hk, a, seed=3, window=4500)
    _cut(s)
    check(s.run(), *s.reference(), "cut items under a window")


@pytest.mark.parametrize("hq,hk,a", [(4, 4, 64), (32, 32, 128), (32, 8, 128), (64, 8, 128), (32, 2, 128), (32, 1, 128)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("window", [0, 4500])
def test_a_row_of_nans_in_a_piece_in_the_middle(hq, hk, a, which, window):
    """It reaches the tokens that see it and their KV head alone, whatever piece it
    stands in: rows that see it get NaNs, the others the bits they had without it."""
    q_len, ctx, p = 100, 6000, 6000 + 50 - 4500 + 1 if window else 3000
    s = Step([(q_len, ctx), (1, 60)], hq, hk, a, seed=13, window=window)
    _cut(s)
    clean = s.run()
    blk, off, g = s.tables[0, p // BS], p % BS, hk - 1
    (s.k_codes if which == "k" else s.v_codes)[blk, g, off] = 0
    (s.k_exps if which == "k" else s.v_exps)[blk, g, off] = 255
    out = s.run()
    G = hq // hk
    hit = torch.zeros(q_len + 1, hq, dtype=torch.bool)
    hit[:51 if window else q_len, g * G:(g + 1) * G] = True      # token 50 is the last whose window holds it
    assert out.cpu()[hit].isnan().all()
    assert torch.equal(out.cpu()[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("hq,hk", [(32, 2), (32, 1)])
@pytest.mark.parametrize("window", [0, 1000, 5003])
def test_single_tokens_of_large_groups_cut(hq, hk, window):
    s = Step([(1, 9000), (1, 6011), (0, 0), (1, 20)], hq, hk, 128, seed=4, window=window)
    if window != 1000:
        _cut(s, single=True)
    out = s.run()
    check(out, *s.reference(), "single tokens")
    for which, codes, exps in (("k", s.k_codes, s.k_exps), ("v", s.v_codes, s.v_exps)):
        blk, off = s.tables[0, 8500 // BS], 8500 % BS
        keep = codes[blk, hk - 1, off].copy(), exps[blk, hk - 1, off]
        codes[blk, hk - 1, off], exps[blk, hk - 1, off] = 0, 255
        got = s.run()
        G = hq // hk
        assert got[0, (hk - 1) * G:].isnan().all()
        assert torch.equal(got[0, :(hk - 1) * G], out[0, :(hk - 1) * G]) and torch.equal(got[1:], out[1:])
        codes[blk, hk - 1, off], exps[blk, hk - 1, off] = keep


@pytest.mark.parametrize("hq,hk,a", [(4, 4, 64), (32, 32, 128), (32, 8, 128), (64, 8, 128), (32, 2, 128), (32, 1, 128)])
def test_cut_items_with_a_growing_maximum(hq, hk, a):
    """Every piece has a larger maximum than the one before it, and value rows of
    very different sizes: the joining's factors matter."""
    s = Step([(30, 5000)], hq, hk, a, seed=5, qscale=2.0, vspread=20)
    _cut(s)
    for p in range(5030):
        s.k_exps[s.tables[0, p // BS], :, p % BS] = 116 + p // 700
    check(s.run(), *s.reference(), "growing maximum")


@pytest.mark.parametrize("hq,hk,a,reqs", [(32, 8, 128, [(2048, 0)]), (64, 8, 128, [(2048, 0)]), (32, 32, 128, [(2048, 0)]),
                                          (32, 1, 128, [(2048, 0)]), (32, 8, 128, [(512, 1024), (512, 2048)] + [(1, 900)] * 20),
                                          (4, 4, 64, [(100, 0)] * 80)])
def test_items_stay_whole_where_cutting_would_cost_more(hq, hk, a, reqs):
    """Prompts without stored keys (their items are short: cut by tiles alone they
    took twice as long), and items that fill the multiprocessors evenly."""
    s = Step(reqs, hq, hk, a, seed=6)
    assert pieces(s.reqs, hq, hk, 0, _ctas()) is None
    ws = s.workspace()
    s.run(workspace=ws)
    assert records(s, ws, False) == []
