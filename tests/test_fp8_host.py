"""The 8-bit cache without a GPU: the oracle's row format pinned by hand, and
what the entry points refuse before anything is enqueued."""
import ctypes
import os

import numpy as np
import pytest
import torch

from oracle import fp8 as of8


def _lib():
    from paged_kv_cache_cb_gb300 import _lib as L
    if not os.path.exists(L.LIB_PATH):
        from paged_kv_cache_cb_gb300 import build
        build.build()
    return L


# ------------------------------------------------------------------ the format
def test_values_are_e4m3():
    """Against torch's own e4m3 type, every finite code."""
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double()
    finite = ~want.isnan()
    assert int(finite.sum()) == 254
    got = np.where(np.arange(256) & 128, -1, 1) * np.append(of8.VALUES, np.nan)[np.arange(256) & 127]
    assert np.array_equal(got[finite.numpy()], want[finite].numpy())


def test_rows_worked_by_hand():
    row = np.zeros((1, 64))
    row[0, :4] = [448.0, 1.0, -0.0625, 2.0 ** -9]
    codes, exps = of8.quantise(row)
    assert exps[0] == 127                                   # 448 = 448 * 2^0
    assert list(codes[0, :4]) == [0x7E, 0x38, 0x98, 0x01]   # 1 = 1.0 * 2^(7-7); 2^-4; the least subnormal
    row[0, 0] = 449.0                                       # one step more: the next exponent
    codes, exps = of8.quantise(row)
    assert exps[0] == 128 and codes[0, 1] == 0x30
    row[0, 3] = 2.0 ** -9                                   # now half of the least subnormal: to even, zero
    assert codes[0, 3] == 0
    assert of8.quantise(np.zeros((1, 64)))[1][0] == 1       # e = -126
    row[0, 9] = np.nan
    codes, exps = of8.quantise(row)
    assert exps[0] == 255 and not codes.any()
    assert np.isnan(of8.values(codes, exps)).all()


def test_rounding_is_torchs():
    g = torch.Generator().manual_seed(0)
    x = torch.randn(200, 64, generator=g).to(torch.bfloat16)
    codes, exps = of8.quantise(x.double().numpy())
    y = (x.double() * torch.from_numpy(2.0 ** (127.0 - exps.astype(np.float64)))[:, None]).float()
    assert np.array_equal(y.to(torch.float8_e4m3fn).view(torch.uint8).numpy(), codes)
    back = of8.values(codes, exps)
    assert (np.abs(back - x.double().numpy()) <= 2.0 ** -4 * np.abs(x.double().numpy())
            + 2.0 ** -10 * 2.0 ** (exps.astype(np.float64) - 127)[:, None]).all()
    assert np.array_equal(torch.from_numpy(back).to(torch.bfloat16).double().numpy(), back)   # exact in bf16


# ------------------------------------------------------------------ refusals of the C ABI
D = ctypes.c_void_p(4096)
ODD = ctypes.c_void_p(4100)


def test_append_gather_and_copy_arguments():
    L = _lib().lib()

    def append(kn=D, vn=D, sl=D, n=4, kc=D, vc=D, ke=D, ve=D, nb=8, hk=2, a=128, bs=16):
        return L.cb_kv_append_fp8(kn, vn, sl, n, kc, vc, ke, ve, nb, hk, a, bs, None)

    def gather(sl=D, n=4, kc=D, vc=D, ke=D, ve=D, nb=8, ko=D, vo=D, hk=2, a=128, bs=16):
        return L.cb_kv_gather_fp8(sl, n, kc, vc, ke, ve, nb, ko, vo, hk, a, bs, None)

    def copy(p=D, n=1, kc=D, vc=D, ke=D, ve=D, nb=8, hk=2, a=128, bs=16):
        return L.cb_copy_blocks_fp8(p, n, kc, vc, ke, ve, nb, hk, a, bs, None)

    for f in (append, gather, copy):
        assert f(n=0) == 0
        for bad in (dict(n=-1), dict(a=96), dict(bs=32), dict(nb=0), dict(hk=0), dict(kc=None), dict(vc=ODD),
                    dict(ke=None), dict(ve=ODD), dict(nb=1 << 26, hk=2)):
            assert f(**bad) == -1, (f.__name__, bad)
    for bad in (dict(kn=None), dict(vn=ODD), dict(sl=None)):
        assert append(**bad) == -1
    for bad in (dict(ko=None), dict(vo=ODD), dict(sl=None)):
        assert gather(**bad) == -1
    assert copy(p=None) == -1 and copy(n=65536) == -1


def test_attention_arguments():
    L = _lib().lib()

    def args(**kw):
        return [kw.get(k, v) for k, v in [
            ("q", D), ("cu", D), ("ctx", D), ("bt", D), ("maxb", 4), ("nr", 2), ("nt", 3), ("mq", 2), ("mkv", 40),
            ("kc", D), ("vc", D), ("ke", D), ("ve", D), ("nb", 16), ("out", D), ("scale", 0.1), ("hq", 4), ("hk", 2),
            ("a", 128), ("bs", 16), ("w", 0), ("ws", D), ("wsb", 1 << 30), ("s", None)]]

    f = L.cb_paged_attention_fp8
    g = lambda *a: L.cb_kv_append_paged_attention_fp8(D, D, D, *a)  # noqa: E731
    for call in (f, g):
        assert call(*args(nr=0)) == 0 and call(*args(nt=0)) == 0
        for bad in (dict(hq=6, hk=4), dict(hq=64, hk=4), dict(hq=32, hk=2, a=64), dict(a=96), dict(bs=8), dict(nr=5000),
                    dict(nr=-1), dict(nt=-1), dict(mq=0), dict(mq=50), dict(mkv=0), dict(maxb=0), dict(scale=0.0),
                    dict(scale=float("nan")), dict(w=-1), dict(q=None), dict(q=ODD), dict(out=ODD), dict(cu=None),
                    dict(ctx=None), dict(bt=None), dict(kc=ODD), dict(ke=ODD), dict(ve=None), dict(ws=None),
                    dict(ws=ODD), dict(nb=0), dict(nb=1 << 26)):
            assert call(*args(**bad)) == -1, bad
        assert call(*args(wsb=16)) == -3
    for bad in ((None, D, D), (D, ODD, D), (D, D, None)):
        assert L.cb_kv_append_paged_attention_fp8(*bad, *args()) == -1
    # key tiles that 32 bits cannot count: of the single tokens, of the chunks
    big = dict(hq=8, hk=8, nr=1024, nt=1024, mkv=1 << 22, maxb=1 << 18)
    assert f(*args(mq=1, **big)) == -1 and f(*args(mq=1, **{**big, "maxb": 1 << 17}, wsb=16)) == -3
    assert f(*args(mq=1 << 20, **{**big, "maxb": 1 << 17, "nt": 1 << 27})) == -1


def test_workspace_size():
    L = _lib()
    f = L.cb_paged_attention_fp8_workspace_size
    assert f(4, 600, 512, 4096, 32, 8, 128, 16) > 0
    assert f(4, 600, 512, 4096, 32, 8, 96, 16) == 0
    assert f(5000, 600, 512, 4096, 32, 8, 128, 16) == 0
    assert f(4, 4, 1, 1 << 30, 32, 8, 128, 16) <= 1 << 27      # it does not grow with the lengths


# ------------------------------------------------------------------ refusals of the binding
def _cpu(nb=4, hk=2, a=64):
    k = torch.zeros(nb, hk, 16, a, dtype=torch.uint8).view(torch.float8_e4m3fn)
    e = torch.zeros(nb, hk, 16, dtype=torch.uint8)
    return k, k.clone(), e, e.clone()


def test_binding_refuses_host_tensors():
    L = _lib()
    x = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    sl = torch.zeros(3, dtype=torch.int64)
    cu, ctx = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([5], dtype=torch.int32)
    bt, ws = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1 << 10, dtype=torch.uint8)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    for call in (lambda: L.cb_kv_append_fp8(x, x, sl, *_cpu()), lambda: L.cb_kv_gather_fp8(sl, *_cpu(), x, x),
                 lambda: L.cb_copy_blocks_fp8(torch.zeros(1, 2, dtype=torch.int32), *_cpu()),
                 lambda: L.cb_paged_attention_fp8(q, cu, ctx, bt, *_cpu(), q, 0.1, ws, 3, 8),
                 lambda: L.cb_kv_append_paged_attention_fp8(x, x, sl, q, cu, ctx, bt, *_cpu(), q, 0.1, ws, 3, 8)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


class _Fake:
    """Stands for a CUDA tensor in the binding's checks (nothing is launched)."""

    is_cuda = True

    def __init__(self, dtype, *shape, device=0, contiguous=True):
        self.dtype, self.shape, self._device, self._contiguous = dtype, torch.Size(shape), device, contiguous

    def dim(self):
        return len(self.shape)

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return 4096

    def get_device(self):
        return self._device


def _fakes(**kw):
    bf, f8, u8, i32 = torch.bfloat16, torch.float8_e4m3fn, torch.uint8, torch.int32
    made = dict(q=_Fake(bf, 3, 4, 64), cu=_Fake(i32, 2), ctx=_Fake(i32, 1), bt=_Fake(i32, 1, 4),
                k=_Fake(f8, 4, 2, 16, 64), v=_Fake(f8, 4, 2, 16, 64), ke=_Fake(u8, 4, 2, 16), ve=_Fake(u8, 4, 2, 16),
                out=_Fake(bf, 3, 4, 64), ws=_Fake(u8, 1 << 20), kn=_Fake(bf, 3, 2, 64), vn=_Fake(bf, 3, 2, 64),
                sl=_Fake(torch.int64, 3))
    made.update(kw)
    return made


def _calls(L, f):
    cache = (f["k"], f["v"], f["ke"], f["ve"])
    step = (f["q"], f["cu"], f["ctx"], f["bt"], *cache, f["out"], 0.1, f["ws"], 3, 8)
    return {"append": lambda: L.cb_kv_append_fp8(f["kn"], f["vn"], f["sl"], *cache, stream=1),
            "gather": lambda: L.cb_kv_gather_fp8(f["sl"], *cache, f["kn"], f["vn"], stream=1),
            "attention": lambda: L.cb_paged_attention_fp8(*step, stream=1),
            "one": lambda: L.cb_kv_append_paged_attention_fp8(f["kn"], f["vn"], f["sl"], *step, stream=1)}


@pytest.mark.parametrize("bad,calls", [
    (dict(k=_Fake(torch.float8_e4m3fn, 4, 2, 16, 128)), "append gather attention one"),
    (dict(ke=_Fake(torch.uint8, 4, 2, 15)), "append gather attention one"),
    (dict(v=_Fake(torch.float8_e4m3fn, 5, 2, 16, 64)), "append gather attention one"),
    (dict(ve=_Fake(torch.uint8, 4, 1, 16)), "append gather attention one"),
    (dict(sl=_Fake(torch.int64, 4)), "append gather one"),
    (dict(vn=_Fake(torch.bfloat16, 3, 1, 64)), "append gather one"),
    (dict(out=_Fake(torch.bfloat16, 2, 4, 64)), "attention one"),
    (dict(cu=_Fake(torch.int32, 3)), "attention one"),
    (dict(bt=_Fake(torch.int32, 2, 4)), "attention one"),
    (dict(q=_Fake(torch.bfloat16, 3, 4, 64, contiguous=False)), "attention one"),
    (dict(k=_Fake(torch.float8_e5m2, 4, 2, 16, 64)), "append gather attention one"),
    (dict(ke=_Fake(torch.int8, 4, 2, 16)), "append gather attention one"),
    (dict(ws=_Fake(torch.float32, 1 << 20)), "attention one"),
    (dict(v=_Fake(torch.float8_e4m3fn, 4, 2, 16, 64, device=1)), "append gather attention one"),
    (dict(sl=_Fake(torch.int64, 3, device=1)), "append gather one"),
    (dict(q=_Fake(torch.bfloat16, 3, 4, 64, device=1)), "attention one"),
])
def test_binding_refuses_wrong_tensors(bad, calls, monkeypatch):
    L = _lib()
    tc = L._tc()
    monkeypatch.setattr(tc, "device", lambda: 0)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, _Fake))
    for name in calls.split():
        with pytest.raises(ValueError):
            _calls(L, _fakes(**bad))[name]()


# ------------------------------------------------------------------ what a query row enters as
def test_query_rows_are_two_terms_within_the_documented_limit():
    """Every value within 2^-17 of its row's largest; exact from 2^-9 of it on."""
    g = torch.Generator().manual_seed(4)
    x = torch.randn(400, 128, generator=g) * torch.exp(4 * torch.randn(400, 128, generator=g))
    x = (x * 2.0 ** torch.randint(-60, 60, (400, 1), generator=g)).to(torch.bfloat16).double().numpy()
    big = np.abs(x).max(-1, keepdims=True)
    y = of8.as_queried(x)
    assert (np.abs(y - x) <= 2.0 ** -17 * big).all()
    kept = np.abs(x) >= 2.0 ** -9 * big
    assert np.array_equal(y[kept], x[kept])
    assert not np.array_equal(y, x)
    assert np.array_equal(of8.as_queried(np.zeros((2, 64))), np.zeros((2, 64)))


def test_places_that_32_bits_cannot_count():
    """Short requests of very many KV heads: each takes some empty places beside its tiles."""
    L = _lib().lib()
    call = lambda hk, nr: L.cb_paged_attention_fp8(D, D, D, D, 1, nr, nr, 1, 16, D, D, D, D, 1, D, 0.1, hk, hk, 128, 16, 0, D, 16,  # noqa: E731
                                                   None)
    assert call((1 << 18) + 1, 2048) == -1
    assert call((1 << 16) + 1, 2048) == -3             # too small a workspace: the sizes were taken


@pytest.mark.parametrize("name,calls", [("kn", "append one"), ("vn", "append gather one"), ("sl", "append gather one"), ("k", "append gather attention one"),
                                        ("ke", "append gather attention one"), ("q", "attention one"), ("cu", "attention one"),
                                        ("ctx", "attention one"), ("bt", "attention one"), ("out", "attention one"), ("ws", "attention one"),
                                        ("pairs", "copy")])
def test_binding_refuses_tensors_without_dimensions(name, calls, monkeypatch):
    L = _lib()
    monkeypatch.setattr(L._tc(), "device", lambda: 0)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, _Fake))
    f = _fakes(pairs=_Fake(torch.int32, 1, 2))
    for shape in [(), (3,) * 5]:
        f = dict(f, **{name: _Fake(f[name].dtype, *shape)})
        made = dict(_calls(L, f), copy=lambda: L.cb_copy_blocks_fp8(f["pairs"], f["k"], f["v"], f["ke"], f["ve"], stream=1))
        for call in calls.split():
            with pytest.raises(ValueError):
                made[call]()


@pytest.mark.parametrize("sizes", [(3 + (1 << 32), 8, 0), (3, 8 + (1 << 32), 0), (3, 8, 5 + (1 << 32)), (3, 8, 1 << 32), (3, 8, 1 << 31)])
def test_binding_refuses_sizes_beyond_32_bits(sizes, monkeypatch):
    """A window of 2^32 + 5 is not one of 5."""
    L = _lib()
    monkeypatch.setattr(L._tc(), "device", lambda: 0)
    monkeypatch.setattr(torch, "Tensor", (torch.Tensor, _Fake))

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0

    monkeypatch.setattr(L, "lib", Lib)
    f = _fakes()
    step = (f["q"], f["cu"], f["ctx"], f["bt"], f["k"], f["v"], f["ke"], f["ve"], f["out"], 0.1, f["ws"])
    L.cb_paged_attention_fp8(*step, 3, 8, 0, stream=1)
    with pytest.raises(ValueError):
        L.cb_paged_attention_fp8(*step, *sizes, stream=1)
    with pytest.raises(ValueError):
        L.cb_kv_append_paged_attention_fp8(f["kn"], f["vn"], f["sl"], *step, *sizes, stream=1)
    if sizes[2] == 0:
        with pytest.raises(ValueError):
            L.cb_paged_attention_fp8_workspace_size(1, 3, sizes[0], sizes[1], 4, 2, 64, 16)
