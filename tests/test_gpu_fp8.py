"""The 8-bit KV cache on the GPU: append and read-back bit for bit against the
float64 definition, attention against the fp64 oracle over the stored values."""
import math

import numpy as np
import pytest
import torch

import workloads as wl
from fp8_util import BS, Step, check
from gpu_util import L
from oracle import attention as oa
from oracle import fp8 as of8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L().lib()


def _empty(nb, hk, a, fill=0x5A):
    return (torch.full((nb, hk, BS, a), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
            torch.full((nb, hk, BS, a), fill, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn),
            torch.full((nb, hk, BS), fill, dtype=torch.uint8, device="cuda"),
            torch.full((nb, hk, BS), fill, dtype=torch.uint8, device="cuda"))


def _bits(cache):
    return [c.view(torch.uint8).cpu().numpy() for c in cache]


def _expected(before, rows, slots):
    want = [b.copy() for b in before]
    for which, x in enumerate(rows):
        codes, exps = of8.quantise(x.double().cpu().numpy())
        for t, s in enumerate(slots):
            if s >= 0:
                want[which][s // BS, :, s % BS] = codes[t]
                want[2 + which][s // BS, :, s % BS] = exps[t]
    return want


def _edge_rows(n, hk, a, seed):
    """Normal rows of many sizes, with rows of the format's edges among them."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, hk, a, generator=g) * torch.exp(6 * torch.randn(n, hk, 1, generator=g))
    x = x.to(torch.bfloat16)
    flat = x.view(n * hk, a)
    edges = [448.0, 449.0, 1.75, 1.7578125, 3.3895e38, 1.2e-38, 9.2e-41, 0.0, -0.0, 2.0 ** -118, 2.0 ** 120]
    for i, e in enumerate(edges):
        if i < n * hk:
            flat[i] = flat[i].sign() * 0
            flat[i, i % a] = e
            flat[i, (i + 7) % a] = -e / 3
    for i, e in enumerate([float("nan"), float("inf"), -float("inf")]):
        if len(edges) + i < n * hk:
            flat[len(edges) + i, (i * 11) % a] = e
    return x


# ------------------------------------------------------------------ append, read-back, copies
@pytest.mark.parametrize("n,hk,a", [(1, 1, 64), (1, 1, 128), (3, 5, 64), (37, 8, 128), (65, 3, 128), (130, 32, 64),
                                    (259, 7, 128)])
def test_append_is_the_definition_bit_for_bit(n, hk, a):
    rng = np.random.default_rng(n + hk)
    nb = -(-n // BS) + 2
    slots = rng.permutation(nb * BS)[:n].astype(np.int64)
    slots[n // 2] = -1 if n > 1 else slots[n // 2]
    k, v = _edge_rows(n, hk, a, 1).cuda(), _edge_rows(n, hk, a, 2).flip(0).contiguous().cuda()
    cache = _empty(nb, hk, a)
    before = _bits(cache)
    L().cb_kv_append_fp8(k, v, torch.from_numpy(slots).cuda(), *cache)
    assert L().cb_last_error() == 0
    assert L().cb_last_launch_count() == 1
    for got, want in zip(_bits(cache), _expected(before, (k, v), slots)):
        assert np.array_equal(got, want)              # rows without a slot in the call: as they were


def test_append_rounds_ties_to_even_over_all_fractions():
    """Every bf16 fraction at every distance below the row's largest value."""
    a = 128
    rows = torch.zeros(32, 1, a, dtype=torch.bfloat16)
    for d in range(32):
        rows[d, 0] = (1 + torch.arange(a) / 128) * 2.0 ** -d
        rows[d, 0, 0] = 1.75
        rows[d, 0, 1::2] *= -1
    cache = _empty(2, 1, a)
    before = _bits(cache)
    slots = np.arange(32, dtype=np.int64)
    L().cb_kv_append_fp8(rows.cuda(), rows.cuda(), torch.from_numpy(slots).cuda(), *cache)
    for got, want in zip(_bits(cache), _expected(before, (rows, rows), slots)):
        assert np.array_equal(got, want)


def test_append_bad_slot_is_skipped_and_reported():
    lib = L()
    rows = torch.randn(4, 2, 64).to(torch.bfloat16).cuda()
    cache = _empty(2, 2, 64)
    before = _bits(cache)
    slots = np.array([3, 32, -5, 1 << 40], np.int64)
    lib.cb_kv_append_fp8(rows, rows, torch.from_numpy(slots).cuda(), *cache)
    assert lib.cb_last_error() == lib.CB_EDEVICE and lib.cb_last_error() == 0
    slots[[1, 3]] = -1
    for got, want in zip(_bits(cache), _expected(before, (rows, rows), slots)):
        assert np.array_equal(got, want)


@pytest.mark.parametrize("n,hk,a", [(1, 1, 64), (50, 3, 128), (333, 8, 64), (1000, 8, 128)])
def test_read_back_is_exact(n, hk, a):
    """What was appended comes back as the stored values; rows with a negative
    slot stay as they were; a bad row comes back as NaNs."""
    lib = L()
    rng = np.random.default_rng(n)
    nb = -(-n // BS) + 1
    slots = rng.permutation(nb * BS)[:n].astype(np.int64)
    k, v = _edge_rows(n, hk, a, 3).cuda(), _edge_rows(n, hk, a, 4).cuda()
    cache = _empty(nb, hk, a)
    d = torch.from_numpy(slots).cuda()
    lib.cb_kv_append_fp8(k, v, d, *cache)
    slots[::3] = -1 if n > 1 else slots[0]
    out = [torch.full_like(k, 7.0), torch.full_like(v, 7.0)]
    lib.cb_kv_gather_fp8(torch.from_numpy(slots).cuda(), *cache, *out)
    assert lib.cb_last_error() == 0
    bits = _bits(cache)
    for which in (0, 1):
        want = torch.full_like(k, 7.0).cpu()
        for t, s in enumerate(slots):
            if s >= 0:
                x = of8.values(bits[which][s // BS, :, s % BS], bits[2 + which][s // BS, :, s % BS])
                want[t] = torch.from_numpy(x).to(torch.bfloat16)
        assert torch.equal(out[which].cpu().nan_to_num(nan=123.0), want.nan_to_num(nan=123.0))


def test_read_back_bad_slot_is_reported():
    lib = L()
    cache = _empty(2, 2, 64, fill=0x30)
    out = [torch.full((3, 2, 64), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    lib.cb_kv_gather_fp8(torch.tensor([31, 32, 0], device="cuda"), *cache, *out)
    assert lib.cb_last_error() == lib.CB_EDEVICE
    assert (out[0][1] == 5.0).all() and (out[0][0] != 5.0).all() and (out[1][2] != 5.0).all()


@pytest.mark.parametrize("hk,a", [(1, 64), (8, 128), (40, 64)])
def test_copy_blocks(hk, a):
    lib = L()
    g = torch.Generator().manual_seed(hk)
    cache = _empty(6, hk, a)
    for c in cache:
        c.view(torch.uint8).copy_(torch.randint(0, 256, c.shape, generator=g, dtype=torch.uint8))
    want = _bits(cache)
    for w in want:
        w[1], w[5] = w[4], w[0]
    lib.cb_copy_blocks_fp8(torch.tensor([[4, 1], [0, 5]], dtype=torch.int32, device="cuda"), *cache)
    assert lib.cb_last_error() == 0
    for got, w in zip(_bits(cache), want):
        assert np.array_equal(got, w)
    lib.cb_copy_blocks_fp8(torch.tensor([[6, 1], [0, -1]], dtype=torch.int32, device="cuda"), *cache)
    assert lib.cb_last_error() == lib.CB_EDEVICE
    for got, w in zip(_bits(cache), want):
        assert np.array_equal(got, w)


# ------------------------------------------------------------------ attention
SHAPES = [(4, 4, 64), (8, 4, 64), (32, 8, 64), (40, 5, 64), (2, 1, 64), (32, 8, 128), (32, 32, 128), (16, 8, 128),
          (64, 8, 128), (12, 12, 128), (24, 6, 128), (1, 1, 128), (8, 1, 128), (32, 2, 128), (32, 1, 128)]


@pytest.mark.parametrize("hq,hk,a", SHAPES)
def test_decode(hq, hk, a):
    """One key, block and tile boundaries, many splits, an empty request."""
    s = Step([(1, 0), (1, 14), (1, 15), (1, 16), (0, 0), (1, 127), (1, 128), (1, 1), (1, 1000), (1, 333)], hq, hk, a,
             seed=hq + a)
    check(s.run(), *s.reference(), "decode")


@pytest.mark.parametrize("hq,hk,a", SHAPES)
def test_chunks(hq, hk, a):
    """Chunks of 2 to 300 tokens, with and without stored keys, beside decodes."""
    s = Step([(2, 0), (1, 40), (17, 5), (3, 126), (0, 7), (130, 0), (1, 0), (300, 77)], hq, hk, a, seed=hq + a + 1)
    check(s.run(), *s.reference(), "chunks")


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (32, 32, 128), (64, 8, 128), (32, 2, 128), (32, 1, 128), (8, 4, 64)])
@pytest.mark.parametrize("window", [1, 2, 16, 100])
def test_window(hq, hk, a, window):
    """A rolling window: blocks before it are released and hold NaN patterns."""
    s = Step([(1, 0), (1, 15), (1, 300), (1, 131), (5, 200), (150, 40), (2, 0)], hq, hk, a, seed=window, window=window)
    check(s.run(), *s.reference(), "window")


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (64, 8, 128), (32, 1, 128)])
def test_one_long_request_is_split(hq, hk, a):
    s = Step([(1, 9000)], hq, hk, a, seed=5)
    check(s.run(), *s.reference(), "one long request")


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (64, 8, 128), (32, 2, 128), (32, 1, 128)])
@pytest.mark.parametrize("most", [40, 130])
def test_many_requests(hq, hk, a, most):
    """Several short sequences per CTA, run repeatedly: the same bits each time."""
    rng = np.random.default_rng(7)
    s = Step([(1, int(c)) for c in rng.integers(0, most, 300)], hq, hk, a, seed=8)
    cache, meta, ws = s.cache(), s.meta(), s.workspace()
    out = s.run(cache=cache, meta=meta, workspace=ws)
    check(out, *s.reference(), "many requests")
    for _ in range(20):
        assert torch.equal(s.run(cache=cache, meta=meta, workspace=ws), out)


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (8, 8, 64), (32, 1, 128)])
def test_many_chunks_of_one_and_two_query_tiles(hq, hk, a):
    """Short and long chunks mixed, several items per CTA, run repeatedly."""
    rng = np.random.default_rng(9)
    reqs = [(int(q), int(c)) for q, c in zip(rng.choice([2, 7, 40, 70], 150), rng.integers(0, 300, 150))]
    s = Step(reqs, hq, hk, a, seed=9)
    cache, meta, ws = s.cache(), s.meta(), s.workspace()
    out = s.run(cache=cache, meta=meta, workspace=ws)
    check(out, *s.reference(), "many chunks")
    for _ in range(20):
        assert torch.equal(s.run(cache=cache, meta=meta, workspace=ws), out)


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (64, 8, 128), (32, 2, 128), (32, 1, 128)])
@pytest.mark.parametrize("q_len", [1, 40])
def test_growing_maximum_and_wide_exponents(hq, hk, a, q_len):
    """Keys whose exponents grow along the sequence, so the running maximum keeps
    rising, and value rows of sizes 2^-20 to 2^20: the accumulators are rescaled."""
    s = Step([(q_len, 700), (q_len, 260)], hq, hk, a, seed=11, qscale=2.0, vspread=20)
    for r, (q, c) in enumerate(s.reqs):
        for p in range(q + c):
            s.k_exps[s.tables[r, p // BS], :, p % BS] = 116 + min(7, p // 90)
    check(s.run(), *s.reference(), "growing maximum")


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (64, 8, 128), (32, 2, 128), (32, 1, 128)])
@pytest.mark.parametrize("q_len", [1, 20])
def test_zero_rows_and_extreme_exponents(hq, hk, a, q_len):
    """Rows of zeros (exponent byte 1), keys and values of the ends of the range."""
    s = Step([(q_len, 200)], hq, hk, a, seed=12)
    at = lambda p: (s.tables[0, p // BS], slice(None), p % BS)  # noqa: E731
    for p in (0, 5, 33, 150):
        s.k_codes[at(p)], s.k_exps[at(p)] = 0, 1
        s.v_codes[at(p)], s.v_exps[at(p)] = 0, 1
    for p in (7, 90):
        s.k_exps[at(p)] = 20
        s.v_exps[at(p)] = 1
    ref, mag = s.reference()
    check(s.run(), ref, mag, "zero rows")
    for p in range(200 + q_len):                       # all values tiny, then all large
        s.v_exps[at(p)] = 12
    check(s.run(), *s.reference(), "tiny values")
    for p in range(200 + q_len):
        s.v_exps[at(p)] = 235
    check(s.run(), *s.reference(), "large values")


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (64, 8, 128), (32, 2, 128)])
@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("q_len", [1, 20])
def test_a_row_of_nans_reaches_its_own_head_only(hq, hk, a, which, q_len):
    """The row is visible to every token of request 0; the other heads' and the
    other request's outputs are those of the same step without it."""
    s = Step([(q_len, 150), (1, 60)], hq, hk, a, seed=13)
    clean = s.run()
    blk, off, g = s.tables[0, 77 // BS], 77 % BS, hk - 1
    (s.k_codes if which == "k" else s.v_codes)[blk, g, off] = 0
    (s.k_exps if which == "k" else s.v_exps)[blk, g, off] = 255
    out = s.run()
    G = hq // hk
    assert out[:q_len, g * G:(g + 1) * G].isnan().all()
    keep = torch.ones(hq, dtype=torch.bool)
    keep[g * G:(g + 1) * G] = False
    if hk > 1:
        assert torch.equal(out[:, keep], clean[:, keep])
    assert torch.equal(out[q_len:], clean[q_len:])


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (32, 1, 128)])
@pytest.mark.parametrize("which", ["k", "v"])
def test_a_row_of_nans_is_seen_from_its_position_on(hq, hk, a, which):
    """A bad row among the chunk's own tokens: the tokens before it do not see it,
    nor do those for which it has left the window."""
    s = Step([(200, 90)], hq, hk, a, seed=23, window=64)
    clean = s.run()
    p, g = 90 + 70, hk - 1
    blk, off = s.tables[0, p // BS], p % BS
    (s.k_codes if which == "k" else s.v_codes)[blk, g, off] = 0
    (s.k_exps if which == "k" else s.v_exps)[blk, g, off] = 255
    out = s.run()
    G = hq // hk
    hit = torch.zeros(200, hq, dtype=torch.bool)
    hit[70:70 + 64, g * G:(g + 1) * G] = True
    assert out.cpu()[hit].isnan().all()
    assert torch.equal(out.cpu()[~hit], clean.cpu()[~hit])


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (64, 8, 128), (32, 2, 128), (32, 1, 128)])
@pytest.mark.parametrize("q_len", [1, 50])
def test_every_code(hq, hk, a, q_len):
    """All 254 finite e4m3 codes, subnormals and zeros of both signs among them,
    over rows of exponents on both sides of the conversion's two ranges."""
    s = Step([(q_len, 250), (q_len, 31)], hq, hk, a, seed=22, qscale=0.05)
    rng = np.random.default_rng(1)
    finite = np.array([c for c in range(256) if c & 127 != 127], np.uint8)
    for r, (q, c) in enumerate(s.reqs):
        for p in range(q + c):
            at = (s.tables[r, p // BS], slice(None), p % BS)
            s.k_codes[at], s.v_codes[at] = rng.choice(finite, (hk, a)), rng.choice(finite, (hk, a))
            s.v_exps[at] = rng.integers(130, 140, hk)
    check(s.run(), *s.reference(), "every code")


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (32, 1, 128)])
@pytest.mark.parametrize("q_len", [1, 3])
def test_nan_in_q_stays_in_its_head(hq, hk, a, q_len):
    s = Step([(q_len, 90)], hq, hk, a, seed=14)
    clean = s.run()
    s.q[0, 2 % hq, 5] = float("nan")
    s.q[0, hq - 1, 6] = float("inf")
    out = s.run()
    bad = torch.zeros(q_len, hq, dtype=torch.bool)
    bad[0, 2 % hq] = bad[0, hq - 1] = True
    assert out.cpu()[bad].isnan().all()
    assert torch.equal(out.cpu()[~bad], clean.cpu()[~bad])


@pytest.mark.parametrize("qmag", [1e-30, 1e-3, 30.0, 1e30])
@pytest.mark.parametrize("q_len", [1, 3])
def test_query_rows_of_any_size(qmag, q_len):
    """Rows of one step from very small to very large, heads of unequal size, and
    a head of zeros; keys scaled so that the scores stay moderate."""
    s = Step([(q_len, 140)], 32, 8, 128, seed=15, qscale=1.0)
    shift = int(round(np.log2(qmag)))
    s.q = (s.q.double() * 2.0 ** shift * torch.tensor([1.0, 0.25, 1.0, 0.0] * 8)[None, :, None]).to(torch.bfloat16)
    used = s.k_exps[s.tables[0]]
    s.k_exps[s.tables[0]] = np.clip(used.astype(np.int64) - shift, 1, 247).astype(np.uint8)
    if shift < 0:
        s.k_exps[s.tables[0]] = np.clip(used.astype(np.int64) - shift, 1, 247).astype(np.uint8)
    ref, mag = s.reference()
    check(s.run(), ref, mag, "query sizes")


def test_rows_of_no_request_are_left_as_they_were():
    """Query rows past the last request (a batch padded for a captured graph)."""
    s = Step([(1, 50), (4, 20)], 32, 8, 128, seed=16)
    q, cu, ctx, tables = s.meta()
    qp = torch.cat([q, torch.full((11, 32, 128), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full_like(qp, 3.0)
    s.run(meta=(qp, cu, ctx, tables), out=out)
    check(out[:5], *s.reference(), "padded batch")
    assert (out[5:] == 3.0).all()


def test_padding_requests_without_tokens():
    """Requests of length zero before, between and after the others."""
    s = Step([(0, 0), (1, 50), (0, 0), (0, 33), (30, 20), (0, 0)], 32, 8, 128, seed=17)
    check(s.run(), *s.reference(), "empty requests")
    e = Step([(0, 0), (0, 5), (1, 0)], 16, 16, 64, seed=18)
    check(e.run(), *e.reference(), "one token")


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (16, 16, 64), (32, 1, 128)])
@pytest.mark.parametrize("q_len", [1, 30])
def test_bad_block_id_is_reported(hq, hk, a, q_len):
    lib = L()
    s = Step([(q_len, 100), (1, 64)], hq, hk, a, seed=19)
    want = s.run()
    for bad in (s.nb, -7, 1 << 30):
        t = s.tables.copy()
        t[0, 2] = bad
        q, cu, ctx, _ = s.meta()
        out = s.run(meta=(q, cu, ctx, torch.from_numpy(t).cuda()), status=lib.CB_EDEVICE)
        assert torch.equal(out[q_len:], want[q_len:])          # the other request is not touched by it
    assert lib.cb_last_error() == 0


@pytest.mark.parametrize("q_len", [1, 30])
def test_bad_lengths_are_reported(q_len):
    """Lengths beyond the table, beyond max_kv_len, or negative: reported, not read."""
    lib = L()
    s = Step([(q_len, 100), (1, 64)], 32, 8, 128, seed=20)
    want = s.run()
    q, cu, ctx, tables = s.meta()
    for bad in (-1, 5000, 2 ** 31 - 1):
        c = ctx.clone()
        c[0] = bad
        out = s.run(meta=(q, cu, c, tables), status=lib.CB_EDEVICE)
        assert torch.equal(out[q_len:], want[q_len:])


def test_same_call_twice_gives_the_same_bits():
    s = Step([(1, 3000), (1, 70), (1, 1500), (200, 500)], 32, 8, 128, seed=21)
    cache, meta = s.cache(), s.meta()
    a = s.run(cache=cache, meta=meta, workspace=s.workspace(fill=0))
    b = s.run(cache=cache, meta=meta, workspace=s.workspace(fill=0x5A))
    assert torch.equal(a, b)


# ------------------------------------------------------------------ a step, as it is used
def _fresh_step(reqs, hq, hk, a, seed):
    s = Step(reqs, hq, hk, a, seed=seed)
    slots = np.concatenate([s.tables[r, p // BS].astype(np.int64) * BS + p % BS
                            for r, (q, c) in enumerate(s.reqs) for p in [c + np.arange(q)]])
    g = torch.Generator().manual_seed(seed)
    rows = [torch.randn(len(slots), hk, a, generator=g).to(torch.bfloat16) for _ in range(2)]
    for which, x in enumerate(rows):
        codes, exps = of8.quantise(x.double().numpy())
        for t, sl in enumerate(slots):
            (s.k_codes, s.v_codes)[which][sl // BS, :, sl % BS] = codes[t]
            (s.k_exps, s.v_exps)[which][sl // BS, :, sl % BS] = exps[t]
    return s, [x.cuda() for x in rows], slots


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (4, 4, 64), (32, 1, 128), (64, 8, 128)])
def test_append_and_attention_as_one_call(hq, hk, a):
    """The one call = append, then attention; each token sees its own stored key;
    the stored rows read back are the ones attention used."""
    lib = L()
    s, (k, v), slots = _fresh_step([(1, 37), (1, 100), (3, 4), (20, 0), (1, 0)], hq, hk, a, 31)
    start = [c.clone() for c in s.cache()]
    for sl in slots:                                   # the new rows are not there yet
        for c in start:
            c.view(torch.uint8)[sl // BS, :, sl % BS] = 0x7F
    d = torch.from_numpy(slots).cuda()
    one, two = [c.clone() for c in start], [c.clone() for c in start]
    meta = s.meta()
    out1, out2 = torch.empty_like(meta[0]), torch.empty_like(meta[0])
    lib.cb_kv_append_paged_attention_fp8(k, v, d, *meta, *one, out1, s.scale, s.workspace(), s.max_q, s.max_kv)
    assert lib.cb_last_error() == 0
    lib.cb_kv_append_fp8(k, v, d, *two)
    lib.cb_paged_attention_fp8(*meta, *two, out2, s.scale, s.workspace(), s.max_q, s.max_kv)
    assert lib.cb_last_error() == 0
    for x, y in zip(one, two):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))
    assert torch.equal(out1, out2)
    check(out1, *s.reference(), "one call")
    back = [torch.empty_like(k), torch.empty_like(v)]
    lib.cb_kv_gather_fp8(d, *one, *back)
    for x, y in zip((k, v), back):                      # within e4m3's half step of what was appended
        err = (x.double() - y.double()).abs()
        assert (err <= 2.0 ** -4 * x.double().abs() + 2.0 ** -10 * x.double().abs().amax(-1, keepdim=True) / 224).all()


def test_recorded_as_a_graph_and_on_another_stream():
    """Direct calls, recorded ones (also updated in place for other lengths) and
    calls on another stream give the same bits; the error word is the stream's."""
    lib = L()
    st = torch.cuda.Stream()
    g = lib.Graph()
    for i, reqs in enumerate([[(1, 600), (1, 33)], [(1, 601), (1, 34)], [(1, 90), (25, 100)]]):
        s, (k, v), slots = _fresh_step(reqs, 32, 8, 128, 40 + i)
        d, meta = torch.from_numpy(slots).cuda(), s.meta()
        cache = s.cache()
        want = torch.empty_like(meta[0])
        ws = s.workspace()
        lib.cb_kv_append_paged_attention_fp8(k, v, d, *meta, *cache, want, s.scale, ws, s.max_q, s.max_kv)
        assert lib.cb_last_error() == 0
        out = torch.full_like(want, float("nan"))
        torch.cuda.synchronize()
        with torch.cuda.stream(st):
            lib.cb_kv_append_paged_attention_fp8(k, v, d, *meta, *cache, out, s.scale, ws, s.max_q, s.max_kv)
            assert lib.cb_last_error() == 0
            assert torch.equal(out, want)
            out.fill_(float("nan"))
            g.begin(st)
            for _ in range(3):                          # layers
                lib.cb_kv_append_paged_attention_fp8(k, v, d, *meta, *cache, out, s.scale, ws, s.max_q, s.max_kv)
            g.end(st)
            assert lib.cb_last_error() == 0
            assert torch.equal(out, want)
        torch.cuda.synchronize()


def test_two_graphs_replayed_at_once():
    """Two captured graphs with workspaces of their own, recorded on one stream and
    replayed on two at once."""
    lib = L()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    made = []
    with torch.cuda.stream(streams[0]):
        for seed in (51, 52):
            s = Step([(1, 2000), (1, 900), (70, 300)], 32, 8, 128, seed=seed)
            cache, meta, ws = s.cache(), s.meta(), s.workspace()
            out = torch.empty_like(meta[0])
            want = s.run(cache=cache, meta=meta, workspace=ws)
            torch.cuda.synchronize()
            gr = torch.cuda.CUDAGraph()
            with torch.cuda.graph(gr, stream=streams[0], capture_error_mode="thread_local"):
                for _ in range(8):
                    lib.cb_paged_attention_fp8(*meta, *cache, out, s.scale, ws, s.max_q, s.max_kv)
            made.append((gr, out, want, cache, meta, ws))
    torch.cuda.synchronize()
    for _ in range(3):
        for m in made:
            m[1].fill_(float("nan"))
        torch.cuda.synchronize()
        for m, st in zip(made, streams):
            with torch.cuda.stream(st):
                m[0].replay()
        torch.cuda.synchronize()
        for m in made:
            assert torch.equal(m[1], m[2])


# ------------------------------------------------------------------ a serving loop
@pytest.mark.parametrize("hq,hk,a,prefix,seed", [(32, 8, 128, 20, 0), (32, 1, 128, 37, 1), (4, 4, 64, 23, 3)])
def test_scheduled_trace_with_shared_prefixes(hq, hk, a, prefix, seed):
    """The scheduler's trace, prefixes shared through the block tables: each step's
    block copies, then its append and attention as one call.  Every request's output
    is that of its own quantised keys in fp64, and a finished step's rows read back
    are theirs."""
    lib = L()
    tr = wl.with_prefixes(wl.small_trace(seed, num_blocks=28), 3, prefix, seed=seed)
    max_len = max(p + o for _, p, o, _, _ in tr.requests)
    rng = np.random.default_rng(seed)
    bf = lambda *n: torch.from_numpy(rng.standard_normal(n)).to(torch.bfloat16)  # noqa: E731
    # contents 0 .. 2: the groups' prefixes; then a request's own rows
    K, V = bf(3 + len(tr.requests), max_len, hk, a), bf(3 + len(tr.requests), max_len, hk, a)
    Q = bf(len(tr.requests), max_len, hq, a)
    K8, V8 = (of8.values(*of8.quantise(x.double().numpy())) for x in (K, V))
    content = lambda r, p: tr.requests[r][3] if tr.requests[r][3] >= 0 and p < tr.requests[r][4] else 3 + r  # noqa: E731
    maxblk = max(-(-(p + o - 1) // BS) for _, p, o, _, _ in tr.requests)
    sched = lib.Scheduler(tr.num_blocks, BS, tr.token_budget, tr.token_budget, wl.free_order(tr.num_blocks, tr.seed), maxblk)
    for t in tr.requests:
        sched.add_request(*t)
    cache = [torch.full((tr.num_blocks, hk, BS, a), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
             for _ in range(2)] + [torch.full((tr.num_blocks, hk, BS), 254, dtype=torch.uint8, device="cuda") for _ in range(2)]
    scale = 1.0 / math.sqrt(a)
    ws = torch.empty(lib.cb_paged_attention_fp8_workspace_size(tr.token_budget, tr.token_budget, tr.token_budget, max_len, hq, hk,
                                                               a, BS), dtype=torch.uint8, device="cuda")
    copies = 0
    while not sched.done():
        m = sched.step()
        pairs = sched.step_copies()
        if len(pairs):
            lib.cb_copy_blocks_fp8(torch.from_numpy(pairs).cuda(), *cache)
            copies += len(pairs)
        b = len(m["req_ids"])
        if b == 0:
            continue
        rows = [(int(r), p) for r, c, n in zip(m["req_ids"], m["ctx_lens"], m["q_lens"]) for p in range(c, c + n)]
        k_new, v_new = (torch.stack([x[content(r, p), p] for r, p in rows]).cuda() for x in (K, V))
        q = torch.stack([Q[r, p] for r, p in rows]).cuda()
        out = torch.full_like(q, float("nan"))
        q_lens, ctx = m["q_lens"].astype(np.int32), m["ctx_lens"].astype(np.int32)
        slots = torch.from_numpy(m["slot_mapping"][:len(rows)]).cuda()
        lib.cb_kv_append_paged_attention_fp8(
            k_new, v_new, slots, q, torch.from_numpy(m["cu_q_lens"][:b + 1].astype(np.int32)).cuda(), torch.from_numpy(ctx).cuda(),
            torch.from_numpy(np.ascontiguousarray(m["block_tables"][:b])).cuda(), *cache, out, scale, ws, int(q_lens.max()),
            int((q_lens + ctx).max()))
        assert lib.cb_last_error() == 0
        ks, vs = ([np.stack([x[content(int(r), p), p] for p in range(c + n)]) for r, c, n in zip(m["req_ids"], ctx, q_lens)]
                  for x in (K8, V8))
        f = lambda v: oa.attention_step(q.double().cpu().numpy(), q_lens.tolist(), ctx.tolist(), ks, v, scale, hq, hk)  # noqa: E731
        check(out, f(vs), f([np.abs(v) for v in vs]), "step")
        back = [torch.empty_like(k_new), torch.empty_like(v_new)]
        lib.cb_kv_gather_fp8(slots, *cache, *back)
        for got, x in zip(back, (K8, V8)):
            assert np.array_equal(got.double().cpu().numpy(), np.stack([x[content(r, p), p] for r, p in rows]))
    assert copies > 0


# ------------------------------------------------------------------ the largest sizes
def test_blocks_far_into_a_large_cache():
    """Blocks past 4 GiB of each cache: the bits of the same step in a small one."""
    lib = L()
    s = Step([(1, 37), (1, 900), (20, 300), (300, 5)], 32, 8, 128, seed=77)
    n, small, meta = 300_000, s.cache(), s.meta()
    off = n - s.nb
    big = [torch.empty((n,) + c.shape[1:], dtype=c.dtype, device="cuda") for c in small]
    for b, c in zip(big, small):
        b.view(torch.uint8)[off:] = c.view(torch.uint8)
    far = meta[:3] + (torch.where(meta[3] >= 0, meta[3] + off, meta[3]),)
    assert torch.equal(s.run(cache=small, meta=meta), s.run(cache=big, meta=far))
    g = torch.Generator().manual_seed(5)
    k, v = (torch.randn(40, 8, 128, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    slots = torch.randperm(s.nb * BS, generator=g)[:40].cuda()
    pairs = torch.tensor([[1, 0], [3, 2]], dtype=torch.int32, device="cuda")
    outs = []
    for cache, d in ((small, 0), (big, off)):
        lib.cb_kv_append_fp8(k, v, slots + d * BS, *cache)
        lib.cb_copy_blocks_fp8(pairs + d, *cache)
        out = [torch.zeros_like(k), torch.zeros_like(v)]
        lib.cb_kv_gather_fp8(slots + d * BS, *cache, *out)
        assert lib.cb_last_error() == 0
        outs.append([c.view(torch.uint8)[d:] for c in cache] + [o.view(torch.int16) for o in out])
    for x, y in zip(*outs):
        assert torch.equal(x, y)


@pytest.mark.parametrize("hq,hk,a", [(8, 1, 128), (32, 2, 128), (4, 4, 64)])
def test_the_most_requests(hq, hk, a):
    """As many requests as a step may have, of one and of several tokens, some
    with none."""
    reqs = [((1, 1, 0, 1, 2, 1, 1)[i % 7], i % 23) for i in range(2048)]
    s = Step(reqs, hq, hk, a, seed=8)
    check(s.run(), *s.reference(), "2048 requests")
