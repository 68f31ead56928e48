"""Attention over the 8-bit cache at the ends of its number range: keys and
queries of the largest and smallest sizes, and query rows of a wide spread."""
import numpy as np
import pytest
import torch

from fp8_util import BS, Step, check
from gpu_util import L
from oracle import attention as oa
from oracle import fp8 as of8

pytestmark = pytest.mark.gpu

SHAPES = [(4, 4, 64), (32, 32, 128), (16, 8, 128), (32, 8, 128), (64, 8, 128), (32, 2, 128), (32, 1, 128)]


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L().lib()


def _every_row(s):
    """(block, slice, offset) of every stored row of every request."""
    for r, (q, c) in enumerate(s.reqs):
        for p in range(q + c):
            yield s.tables[r, p // BS], slice(None), p % BS


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("kexp", [(245, 248), (232, 240), (90, 93), (5, 8), (1, 3)])
@pytest.mark.parametrize("q_len", [1, 3, 40])
def test_keys_of_any_size_with_moderate_scores(hq, hk, a, kexp, q_len):
    """Keys around 2^120 and around 2^-120, queries as much the other way: the
    scores are those of normal rows (the bound's rounding errors are too: every
    factor is a power of two, the queries' subnormals are in the oracle's inputs)."""
    mid = (kexp[0] + kexp[1] - 1) / 2
    s = Step([(q_len, 300), (q_len, 15)], hq, hk, a, seed=61, kexp=kexp, qscale=2.0 ** (121 - mid))
    check(s.run(), *s.reference(), "keys of any size")


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("q_len", [1, 40])
def test_keys_of_all_sizes_side_by_side(hq, hk, a, q_len):
    """Most keys so small that they score 0, some normal ones among them, one tile
    of small ones only."""
    s = Step([(q_len, 500)], hq, hk, a, seed=62)
    rng = np.random.default_rng(3)
    for i, at in enumerate(_every_row(s)):
        s.k_exps[at] = rng.choice([1, 2, 40, 80]) if 128 <= i < 256 or i % 3 else 121
    check(s.run(), *s.reference(), "keys of all sizes")


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("kexp,large", [(87, 220), (87, 247), (10, 230), (121, 247), (1, 126)])
@pytest.mark.parametrize("q_len", [1, 20])
def test_a_large_key_does_not_hide_small_ones(hq, hk, a, kexp, large, q_len):
    """Keys up to 2^240 times the others, at right angles to the queries; with several
    tokens also one that only the last token, whose query is 0, sees."""
    s = Step([(q_len, 300)], hq, hk, a, seed=67, kexp=(kexp, kexp + 2), qscale=2.0 ** (121 - kexp))
    s.q[..., 1] = 0
    for p in (3, 140, 290) + ((319,) if q_len > 1 else ()):
        at = s.tables[0, p // BS], slice(None), p % BS
        s.k_exps[at] = large
        if p < 319:
            s.k_codes[at] = 0
            s.k_codes[at][:, 1] = 0x7E
    if q_len > 1:
        s.q[-1] = 0
    check(s.run(), *s.reference(), "a large key")


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("q_len", [1, 20])
def test_the_smallest_queries_keep_their_scale(hq, hk, a, q_len):
    """Rows of 2^-119 in line with keys of 2^108, on either side: small scores, but
    not nothing, from a factor below the normal numbers."""
    s = Step([(q_len, 300)], hq, hk, a, seed=68)
    s.q[:] = 2.0 ** -119
    for i, at in enumerate(_every_row(s)):
        s.k_codes[at], s.k_exps[at] = 0x7E if i % 2 else 0xFE, 227
        s.v_codes[at] = (s.v_codes[at] & 127) | (0 if i % 2 else 128)
    ref, mag = s.reference()
    assert np.abs(ref).max() > 0.01 * mag.max()
    check(s.run(), ref, mag, "small queries")


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("q_len", [1, 3])
def test_query_of_zeros_under_a_small_scale(hq, hk, a, q_len):
    """Every score is 0, whatever the scale; the keys out of sight stay out."""
    s = Step([(q_len, 77)], hq, hk, a, seed=64)
    s.q[:, ::2] = 0
    s.scale = 1e-12
    check(s.run(), *s.reference(), "small scale")


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("q_len", [1, 3])
def test_large_rows_at_right_angles(hq, hk, a, q_len):
    """Queries and keys of 2^100 in different channels: every score is 0."""
    s = Step([(q_len, 200)], hq, hk, a, seed=63)
    s.q.zero_()
    s.q[..., 0] = 2.0 ** 100
    for at in _every_row(s):
        s.k_codes[at] = 0
        s.k_codes[at][:, 1] = 0x7E
        s.k_exps[at] = 220
    check(s.run(), *s.reference(), "right angles")


@pytest.mark.parametrize("hq,hk,a", SHAPES)
@pytest.mark.parametrize("ratio", [2.0 ** 9, 2.0 ** 13, 2.0 ** 17])
@pytest.mark.parametrize("q_len", [1, 20])
def test_query_rows_of_a_wide_spread(hq, hk, a, ratio, q_len):
    """A query value many times the others, over keys that are 0 in its channel, so
    that the others alone decide the scores.  They enter as the documented two
    terms, and the weights follow from those within the usual bound."""
    s = Step([(q_len, 150), (q_len, 31)], hq, hk, a, seed=65)
    s.q[..., 5] = ratio
    for at in _every_row(s):
        s.k_codes[at][:, 5] = 0
    q = of8.as_queried(s.q.double().numpy())
    assert (np.abs(q - s.q.double().numpy()) <= 2.0 ** -17 * ratio).all()
    ks, vs = zip(*[s.rows(r) for r in range(len(s.reqs))])
    f = lambda v: oa.attention_step(q, s.q_lens, s.ctx, ks, v, s.scale, hq, hk)  # noqa: E731
    check(s.run(), f(vs), f([np.abs(v) for v in vs]), "wide spread")


@pytest.mark.parametrize("hq,hk,a", [x for x in SHAPES if x[0] // x[1] <= 8])
def test_single_tokens_weights_have_more_bits_than_bf16(hq, hk, a):
    """Two to nine keys whose values cancel in pairs, so that neither averaging nor
    the output's rounding hides the weights' error: at most 2^-11 (a half's
    rounding) and 2^-9 (its lowest five bits rounded to three) of each, and 2^-11
    of its exponent (a score's terms sum to about 20 in magnitude: 20 log2 e 128
    2^-24 < 2^-12, and as much for 2^x and the sums)."""
    s = Step([(1, 1 + 2 * (i % 5)) for i in range(60)], hq, hk, a, seed=66)
    for r, (q, c) in enumerate(s.reqs):
        for p in range(1, q + c, 2):
            at, one = ((s.tables[r, i // BS], slice(None), i % BS) for i in (p, p - 1))
            s.v_codes[at], s.v_exps[at] = s.v_codes[one] ^ 128, s.v_exps[one]
    ref, mag = s.reference()
    err = np.abs(s.run().double().cpu().numpy() - ref)
    assert (err <= 2.0 ** -8 * np.abs(ref) + (2.0 ** -9 + 2 * 2.0 ** -11) * mag).all()
