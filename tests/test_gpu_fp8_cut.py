"""Attention over the 8-bit cache where items of several tokens, and single tokens
of the large groups, are cut between CTAs and joined again."""
import numpy as np
import pytest
import torch

from fp8_util import BS, Step, check
from gpu_util import L

pytestmark = pytest.mark.gpu

CUT_TILES = 10           # the kernel's kCutTiles


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L().lib()


def pieces(reqs, hq, hk, window, ctas, single=False):
    """The chunk kernel's plan: (request, pair of query tiles, first key tile, end,
    piece's first tile, piece's end) of every piece, or None where items stay whole."""
    tok2 = 2 * 128 // (hq // hk)
    items = []
    for r, (q, c) in enumerate(reqs):
        if q == 0 or (q == 1) != single:
            continue
        for pair in range(-(-q // tok2) - 1, -1, -1):
            first = max(0, c + pair * tok2 - window + 1) // 128 if window else 0
            end = -(-(c + min(q, (pair + 1) * tok2)) // 128)
            items += [(r, pair, first, end)] * hk
    total = sum(e - f for _, _, f, e in items)
    longest = max(e - f for _, _, f, e in items)
    if -(-len(items) // ctas) * longest <= -(-total // ctas) + CUT_TILES:
        return None
    eff = min(ctas, total)
    borders = {total * b // eff for b in range(eff + 1)}
    out, at = [], 0
    for r, pair, f, e in items:
        cuts = sorted({at, at + e - f} | {b for b in borders if at < b < at + e - f})
        out += [(r, pair, f, e, f + x - at, f + y - at) for x, y in zip(cuts, cuts[1:])]
        at += e - f
    return out


def _ctas():
    return min(torch.cuda.get_device_properties(0).multi_processor_count, 160)


def _cut(s, single=False, least=3):
    p = pieces(s.reqs, s.hq, s.hk, s.window, _ctas(), single)
    assert p is not None and len(p) > 64
    assert max(sum(x[:4] == y[:4] for y in p) // s.hk for x in p) >= least - 1
    return p


SHAPES = [(4, 4, 64), (8, 4, 64), (32, 8, 64), (40, 5, 64), (32, 32, 128), (16, 8, 128), (32, 8, 128), (64, 8, 128), (8, 1, 128),
          (32, 2, 128), (32, 1, 128)]


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("reqs", [[(40, 5000)], [(2, 9000)], [(300, 3500)], [(3, 4000), (1, 700), (129, 6000), (0, 3), (2, 30)]])
def test_cut_items(hq, hk, a, reqs):
    s = Step(reqs, hq, hk, a, seed=hq + a)
    _cut(s, least=2)
    cache, meta = s.cache(), s.meta()
    out = s.run(cache=cache, meta=meta)
    check(out, *s.reference(), "cut items")
    assert torch.equal(s.run(cache=cache, meta=meta, workspace=s.workspace(fill=0x5A)), out)


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("q_len", [40, 256])
def test_cut_items_under_a_window(hq, hk, a, q_len):
    """A window of more tiles than whole items may have: pieces lie before the
    windows of some of their rows, or behind the positions of others."""
    s = Step([(q_len, 6000)], hq, hk, a, seed=3, window=4500)
    p = _cut(s, least=2)
    tok2 = 2 * 128 // (hq // hk)
    unseen = False
    for r, pair, f, e, x, y in p:
        for i in {pair * tok2, min(q_len, (pair + 1) * tok2) - 1}:
            unseen |= y * 128 <= 6000 + i - 4500 + 1 or x * 128 > 6000 + i
    assert unseen or (q_len == 256 and hq // hk >= 16)          # a pair of their tiles is 8 or 16 tokens
    check(s.run(), *s.reference(), "cut items under a window")


@pytest.mark.parametrize("hq,hk,a", [(4, 4, 64), (32, 32, 128), (32, 8, 128), (64, 8, 128), (32, 2, 128), (32, 1, 128)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("window", [0, 4500])
def test_a_row_of_nans_in_a_piece_in_the_middle(hq, hk, a, which, window):
    """It reaches the tokens that see it and their KV head alone, whatever piece it
    stands in: rows that see it get NaNs, the others the bits they had without it."""
    q_len, ctx, p = 100, 6000, 6000 + 50 - 4500 + 1 if window else 3000
    s = Step([(q_len, ctx), (1, 60)], hq, hk, a, seed=13, window=window)
    _cut(s, least=2)
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
    _cut(s, least=2)
    for p in range(5030):
        s.k_exps[s.tables[0, p // BS], :, p % BS] = 116 + p // 700
    check(s.run(), *s.reference(), "growing maximum")
