"""Cross attention against its definition in float64."""
import math

import pytest
import torch

from cross_util import BS, Batch
from gpu_util import L

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


SHAPES = [(4, 4, 64), (8, 4, 64), (32, 8, 64), (16, 1, 64), (32, 1, 64), (12, 12, 128), (32, 8, 128), (64, 8, 128),
          (32, 2, 128), (32, 1, 128), (6, 3, 128), (96, 3, 128)]
EDGES = [(1, 1), (1, 15), (2, 16), (1, 17), (0, 40), (3, 127), (1, 128), (7, 129), (5, 0), (1, 255), (1, 0), (0, 0), (4, 257),
         (1, 1000)]


@pytest.mark.parametrize("hq,hk,a", SHAPES)
def test_edges(hq, hk, a):
    b = Batch(EDGES, hq, hk, a, seed=hq + a, extra_tokens=3)
    b.compare(b.run())


@pytest.mark.parametrize("hq,hk,a", SHAPES)
def test_tiles(hq, hk, a):
    """Token counts around half a tile, a tile, two and more of a group's rows."""
    tok = 128 // (hq // hk)
    reqs = [(max(1, tok + d), n) for d, n in ((-1, 300), (0, 128), (1, 513), (tok - 1, 77), (tok, 200), (tok + 1, 1),
                                              (3 * tok + 2, 700), (2 * tok + 1, 130))]
    b = Batch(reqs, hq, hk, a, seed=hq + hk, extra_tokens=1)
    b.compare(b.run())


@pytest.mark.parametrize("hq,hk,a,reqs", [
    (32, 1, 128, [(1, 20000)]),                     # one sequence over every SM
    (4, 4, 64, [(1, 3000)]),
    (32, 8, 128, [(1, 9000), (1, 3)]),
    (8, 8, 128, [(300, 5000)]),                     # wide items cut in pieces
    (32, 32, 128, [(4, 700)] * 9),
    (32, 8, 128, [(1, 256 + 131 * i) for i in range(48)]),
    (32, 8, 128, [(129, 4001), (1, 5000), (64, 1), (500, 2500)]),
])
def test_work_cut_between_ctas(hq, hk, a, reqs):
    b = Batch(reqs, hq, hk, a, seed=5)
    out = b.run()
    b.compare(out)
    assert torch.equal(out, b.run())                # pieces are joined in the same order every time


def test_many_requests():
    b = Batch([(i % 3, (i * 37) % 200) for i in range(2048)], 4, 2, 64, seed=6)
    b.compare(b.run(), requests=range(0, 2048, 7))


@pytest.mark.parametrize("qscale,kscale", [(8.0, 4.0), (0.0, 1.0), (1e-20, 1e-20), (300.0, 300.0)])
def test_sizes_of_scores(qscale, kscale):
    b = Batch([(1, 700), (40, 300), (300, 260)], 8, 4, 128, seed=7, qscale=qscale, kscale=kscale)
    b.compare(b.run())


def test_growing_scores():
    """Keys in order of their scores: the running max grows at every tile."""
    b = Batch([(2, 1500), (200, 1500)], 4, 4, 64, seed=8)
    for r in range(2):
        for i, blk in enumerate(b.tables[r, :94]):
            rows = min(BS, 1500 - i * BS)
            b.k[int(blk), :, :rows] = torch.linspace(i, i + 1, BS, device="cuda", dtype=torch.float32)[:rows, None].to(torch.bfloat16)
    b.q.copy_(torch.rand_like(b.q) * 0.2)
    b.compare(b.run())


def test_a_query_that_is_not_finite_stays_alone():
    b = Batch([(4, 300), (130, 300)], 8, 4, 128, seed=9)
    b.q[1, 3] = math.nan
    b.q[50, 2, 7] = math.inf
    out = b.run()
    nan = out.float().isnan().all(-1)
    want = torch.zeros_like(nan)
    want[1, 3] = want[50, 2] = True
    assert torch.equal(nan, want)
    b.q[1, 3] = 0
    b.q[50, 2] = 0
    clean = b.run()
    assert torch.equal(out[~want], clean[~want])


def test_infinite_scores():
    """A key of score -inf has no weight; rows of nothing else are NaN, as softmax has it."""
    b = Batch([(3, 200)], 2, 2, 64, seed=10)
    b.q.copy_(b.q.abs() + 0.5)
    blk = [int(x) for x in b.tables[0, :13]]
    for i in (0, 5, 8, 9, 10, 11, 12):              # the second tile's keys among them
        b.k[blk[i], 0, :min(BS, 200 - i * BS)] = -math.inf
    for i in range(13):
        b.k[blk[i], 1, :min(BS, 200 - i * BS)] = -math.inf
    out = b.run()
    assert out[:, 1].float().isnan().all()
    keep = [i for i in range(200) if i // BS not in (0, 5, 8, 9, 10, 11, 12)]
    k, v = b.request(0)
    s = torch.einsum("qd,nd->qn", b.q[:, 0].double(), k[0][keep]) * b.scale
    ref = torch.softmax(s, -1) @ v[0][keep]
    size = torch.softmax(s, -1) @ v[0][keep].abs()
    assert ((out[:, 0].double() - ref).abs() <= 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2.0 ** -13) * size).all()


def test_one_token_is_the_causal_decode():
    """A single new token over n keys: what cb_paged_attention gives for the last of n stored tokens."""
    lib = L()
    b = Batch([(1, 33), (1, 700), (1, 2000), (1, 1)], 32, 8, 128, seed=11)
    out = b.run()
    ws = torch.empty(lib.cb_paged_attention_workspace_size(4, 4, 1, 2000, 32, 8, 128, BS), dtype=torch.uint8, device="cuda")
    other = torch.empty_like(out)
    lib.cb_paged_attention(b.q, b.d_cu, b.d_kv - 1, b.d_tables, b.k, b.v, other, b.scale, ws, 1, 2000)
    assert lib.cb_last_error() == 0
    b.compare(out)
    b.compare(other)


def test_a_cache_past_4_gib():
    b = Batch([(1, 500), (200, 300)], 32, 8, 128, seed=12, num_blocks=140000, first=139900)
    b.compare(b.run())


def test_streams_and_replays():
    """Recorded once, replayed over changing lengths and tables; another stream at the same time."""
    lib = L()
    b = Batch([(1, 900), (3, 2000), (1, 40), (130, 600)], 16, 4, 128, seed=13)
    c = Batch([(2, 1500)] * 6, 8, 8, 64, seed=14)
    s, t = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        out, ws = torch.full_like(b.q, 7.0), b.workspace()
        b.run(out, ws)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            b.run(out, ws, check=False)
    with torch.cuda.stream(t):
        out2, ws2 = torch.full_like(c.q, 7.0), c.workspace()
        c.run(out2, ws2)
    torch.cuda.synchronize()
    for kv in ((900, 2000, 40, 600), (1, 0, 17, 599), (512, 1999, 33, 128)):
        b.kv, b.reqs = list(kv), list(zip(b.q_lens, kv))
        b.d_kv.copy_(torch.tensor(kv, dtype=torch.int32))
        # what a shorter request no longer holds may be anything
        out.fill_(7.0)
        torch.cuda.synchronize()
        for _ in range(3):
            with torch.cuda.stream(s):
                graph.replay()
            with torch.cuda.stream(t):
                c.run(out2, ws2, check=False)
        assert lib.cb_last_error(s) == 0 and lib.cb_last_error(t) == 0
        b.compare(out)
        c.compare(out2)


def test_recorded_with_the_librarys_graph():
    lib = L()
    b = Batch([(1, 900), (3, 2000)], 32, 8, 128, seed=15)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        want = b.run()
        out, ws = torch.full_like(b.q, 7.0), b.workspace()
        g = lib.Graph()
        s.synchronize()
        for _ in range(2):
            g.begin(s)
            b.run(out, ws, check=False, stream=s)
            g.end(s)
        assert lib.cb_last_error(s) == 0
    assert torch.equal(out, want)
    g.close()


def test_bad_metadata():
    """Reported; a bad id's rows are zeros, a bad request's rows stay, the others are as ever."""
    lib = L()
    reqs = [(2, 300), (3, 400), (1, 200)]

    def bad(change):
        b = Batch(reqs, 8, 4, 128, seed=16)
        change(b)
        out = b.run(check=False)
        assert lib.cb_last_error() == lib.CB_EDEVICE
        return b, out

    for e in (-1, 10 ** 6):
        def entry(b, e=e):
            b.d_tables[1, 3] = e
        b, out = bad(entry)
        b.compare(out, requests=(0, 2))
        blk = int(b.tables[1, 3])
        b.k[blk] = 0
        b.v[blk] = 0
        b.compare(out)
    for value in (-1, 1 << 30, 401, 16 * 27):
        def length(b, value=value):
            b.d_kv[1] = value
        b, out = bad(length)
        b.compare(out, requests=(0, 2))
        assert (out[2:5] == 7.0).all()
    for cu in ((0, 2, 1, 6), (0, 2, 5, 60), (-1, 2, 5, 6), (0, 2, 6, 6)):
        def offsets(b, cu=cu):
            b.d_cu.copy_(torch.tensor(cu, dtype=torch.int32))
        bad(offsets)


def test_refusals():
    lib = L()
    b = Batch([(2, 30)], 8, 4, 128, seed=17)
    ws, out = b.workspace(), torch.empty_like(b.q)
    good = dict(q=b.q, cu=b.d_cu, kv=b.d_kv, bt=b.d_tables, k=b.k, v=b.v, out=out, ws=ws)

    def call(scale=0.1, mq=2, mkv=30, **kw):
        x = {**good, **kw}
        lib.cb_paged_cross_attention(x["q"], x["cu"], x["kv"], x["bt"], x["k"], x["v"], x["out"], scale, x["ws"], mq, mkv)

    for kw in (dict(q=b.q.float()), dict(q=b.q[:, :, :64]), dict(out=out[:1]), dict(cu=b.d_cu[:1]), dict(cu=b.d_cu.long()),
               dict(kv=b.d_kv.cpu()), dict(bt=b.d_tables[:0]), dict(k=b.k[:1]), dict(v=b.v.half()), dict(ws=ws.int()),
               dict(k=b.k[..., :64].contiguous(), v=b.v[..., :64].contiguous()), dict(mkv=1 << 31)):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(scale=0.0), dict(scale=-1.0), dict(mq=0), dict(mkv=-1), dict(ws=ws[:64]), dict(scale=math.nan)):
        with pytest.raises(lib.CBError):
            call(**kw)
    for hq in (12, 3):                              # groups of 3, and none
        q = torch.zeros(2, hq, 128, device="cuda", dtype=torch.bfloat16)
        with pytest.raises(lib.CBError):
            call(q=q, out=q.clone())
    assert lib.cb_last_error() == 0
    e = torch.zeros(0, 8, 128, device="cuda", dtype=torch.bfloat16)
    call(q=e, out=e.clone(), cu=b.d_cu * 0)         # no tokens: nothing to do


@pytest.mark.parametrize("hq,hk,a,q", [(4, 4, 64, 2), (32, 1, 64, 1), (8, 4, 64, 16), (4, 4, 128, 2), (16, 1, 128, 1), (4, 2, 128, 8),
                                       (17 * 4, 17, 128, 4), (17, 17, 64, 32), (32, 1, 128, 1), (16, 2, 128, 4), (4, 4, 128, 32),
                                       (8, 8, 128, 33)])
def test_few_rows(hq, hk, a, q):
    """Items of up to 32 rows (and of 33), whose keys four warps share: lengths around a
    warp's 32 keys and a tile's 128, maxima that grow from tile to tile, and keys of score -inf."""
    lens = [1, 15, 16, 17, 31, 32, 33, 64, 65, 95, 97, 127, 128, 129, 255, 256, 257, 383, 385, 640, 1500]
    b = Batch([(1 + (r % q), n) for r, n in enumerate(lens)] + [(0, 70), (q, 0), (q, 900)], hq, hk, a, seed=hq + a)
    b.compare(b.run())
    for r, n in enumerate(b.kv):                    # scores that grow with the key
        for i in range(-(-n // BS)):
            rows = min(BS, n - i * BS)
            b.k[int(b.tables[r, i]), :, :rows] = torch.linspace(i, i + 1, BS, device="cuda")[:rows, None].to(torch.bfloat16)
    b.q.copy_(torch.rand_like(b.q) * 0.2)
    out = b.run()
    b.compare(out)
    b.q[0, 0] = math.nan                            # a row that is not finite stays alone
    bad = b.run()
    assert bad[0, 0].isnan().all()
    assert torch.equal(bad.flatten(0, 1)[1:], out.flatten(0, 1)[1:])


@pytest.mark.parametrize("a", [64, 128])
def test_few_rows_of_infinite_scores(a):
    b = Batch([(2, 200)], 2, 2, a, seed=20)
    b.q.copy_(b.q.abs() + 0.5)
    blk = [int(x) for x in b.tables[0, :13]]
    gone = (0, 1, 5, 8, 9, 10, 11, 12)              # a warp's whole share of the first tile, and the second tile
    for i in range(13):
        rows = min(BS, 200 - i * BS)
        if i in gone:
            b.k[blk[i], 0, :rows] = -math.inf
        b.k[blk[i], 1, :rows] = -math.inf
    out = b.run()
    assert out[:, 1].isnan().all()                  # softmax of nothing but -inf
    keep = [i for i in range(200) if i // BS not in gone]
    k, v = b.request(0)
    s = torch.einsum("qd,nd->qn", b.q[:, 0].double(), k[0][keep]) * b.scale
    p = torch.softmax(s, -1)
    ref, size = p @ v[0][keep], p @ v[0][keep].abs()
    e = a * 2.0 ** -23 * b.scale * (b.q[:, 0].double().abs() @ k[0][keep].abs().T).amax(-1, keepdim=True)      # as Batch.compare
    e = e + (1 + s.abs().amax(-1, keepdim=True)) * 2.0 ** -20
    bound = 2.0 ** -8 * ref.abs() + (2.0 ** -8 + 2 * torch.expm1(e) + 200 * 2.0 ** -23) * size
    assert ((out[:, 0].double() - ref).abs() <= bound * (1 + 2.0 ** -8)).all()


def test_few_rows_cut_between_ctas():
    for hq, hk, a in ((32, 8, 64), (32, 8, 128), (4, 4, 64), (4, 4, 128)):
        b = Batch([(1, 40000), (1, 3), (2, 5001), (1, 128 * 9)], hq, hk, a, seed=a)
        out = b.run()
        b.compare(out)
        assert torch.equal(out, b.run())
