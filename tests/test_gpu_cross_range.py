"""Cross attention of finite queries and keys whose scores are far from 0: every
score is an exact product, so what the softmax is of is known."""
import math

import pytest
import torch

from cross_util import BS, Batch

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _patterns(n, g):
    """Whole numbers of up to 8 bits, one row per order in which a maximum can be met."""
    up = torch.arange(n) * 255 // n
    one = torch.zeros(n, dtype=torch.long)
    one[n // 2] = 1
    back = torch.where(torch.arange(n) < min(n, 140), -200, 0)           # far below 0, then 0
    ties = torch.randint(0, 8, (n,), generator=g)
    return torch.stack([up, up.flip(0), -1 - up, one, -one, back, ties, torch.full((n,), 3)])


@pytest.mark.parametrize("a", [64, 128])
@pytest.mark.parametrize("q", [3, 40, 200])                              # few rows, thread = row, two row tiles
@pytest.mark.parametrize("e", [20, 27, 28, 29, 31, 32, 33, 34, 41, 60, 90, 112])
def test_scores_far_from_zero(a, q, e):
    """Scores x 2^e scale, x whole: the keys of the largest x share the weight.  Every third token's are x scale, and
    every third -x 2^e scale: no row's result depends on another's.

    Scores far apart: the weights are 2^r for the largest and 0, r a rounding of fp32 (under 8, so 2^-20 in an exponent),
    a weight is rounded to bf16, and so is the output."""
    b = Batch([(q, 300), (q, 129), (q, 5000)], 8, 8, a, seed=e, kscale=0.0)
    g = torch.Generator().manual_seed(e)
    big = 2.0 ** (e // 2), 2.0 ** (e - e // 2)
    b.q.zero_()
    b.q[0::3, :, 5], b.q[1::3, :, 5], b.q[2::3, :, 5] = big[0], 1 / big[1], -big[0]
    xs = [_patterns(n, g).cuda() for n in b.kv]
    for r, n in enumerate(b.kv):
        blk = torch.from_numpy(b.tables[r, :-(-n // BS)].astype("int64")).cuda()
        rows = torch.arange(n, device="cuda")
        b.k[blk[rows // BS], :, rows % BS, 5] = (xs[r].T.double() * big[1]).to(torch.bfloat16)
    out = b.run()
    assert torch.equal(out.view(torch.int16), b.run().view(torch.int16))
    for r, n in enumerate(b.kv):
        t = torch.arange(r * q, (r + 1) * q, device="cuda")
        by = torch.tensor([2.0 ** e, 1.0, -2.0 ** e], device="cuda", dtype=torch.float64)[t % 3] * b.scale
        s = by[:, None, None] * xs[r].double()                           # [q, head, key]
        p = torch.softmax(s, -1)
        v = b.request(r)[1]
        ref, size = torch.einsum("qhn,hna->qha", p, v), torch.einsum("qhn,hna->qha", p, v.abs())
        near = (1 + 255 * b.scale) * 2.0 ** -20                          # of the scores x scale
        bound = (2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * math.expm1(near) + n * 2.0 ** -23) * size) * (1 + 2.0 ** -8)
        err = (out[r * q:(r + 1) * q].double() - ref).abs()
        assert (err <= bound).all(), (r, int((~(err <= bound)).sum()))


@pytest.mark.parametrize("a", [64, 128])
@pytest.mark.parametrize("q", [1, 40, 200])
@pytest.mark.parametrize("size", [2.0 ** 12, 2.0 ** 16, 2.0 ** 25, 2.0 ** 50])
def test_large_random_queries_and_keys(a, q, size):
    """Scores of either sign up to 2^100: finite, and the value of the key with the largest score where no other
    comes near it."""
    b = Batch([(q, 300), (q, 700)], 4, 2, a, seed=a + q, qscale=size, kscale=size)
    out = b.run()
    assert torch.isfinite(out).all()
    for r in range(2):
        k, v = b.request(r)
        for h in range(4):
            x = b.q[r * q:(r + 1) * q, h].double()
            s = x @ k[h // 2].T * b.scale
            top, at = s.topk(2, -1)
            off = 2 * a * 2.0 ** -23 * b.scale * (x.abs() @ k[h // 2].abs().T).amax(-1)    # two fp32 sums, any order
            clear = top[:, 0] - top[:, 1] > off + top.abs().amax(-1) * 2.0 ** -22 + 30
            assert clear.float().mean() > 0.5
            ref = v[h // 2][at[clear, 0]]
            err = (out[r * q:(r + 1) * q, h].double()[clear] - ref).abs()
            # a weight and the output are rounded to bf16; e^-30 of 700 others
            assert (err <= (2.0 ** -7 + 2.0 ** -15) * ref.abs() + 700 * math.exp(-30) * v.abs().max()).all()
