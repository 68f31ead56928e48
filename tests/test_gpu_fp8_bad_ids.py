"""Block ids out of range and lengths that do not fit, over the 8-bit cache: what
the flagged request gets does not depend on what ran before."""
import numpy as np
import pytest
import torch

from fp8_util import Step, check
from gpu_util import L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L().lib()


@pytest.mark.parametrize("hq,hk,a", [(4, 4, 64), (32, 32, 128), (32, 8, 128), (64, 8, 128), (32, 2, 128), (32, 1, 128)])
@pytest.mark.parametrize("q_len,ctx", [(1, 100), (30, 100), (40, 5000)])
def test_rows_of_a_bad_block_count_as_zeros(hq, hk, a, q_len, ctx):
    """The same result as over a block of zero rows, bit for bit, after a step whose
    rows left NaNs and large values in shared memory and after another."""
    lib = L()
    s = Step([(q_len, ctx), (1, 64)], hq, hk, a, seed=19)
    zero = int(np.setdiff1d(np.arange(s.nb), s.tables[s.tables >= 0])[0])
    for codes, exps in ((s.k_codes, s.k_exps), (s.v_codes, s.v_exps)):
        codes[zero], exps[zero] = 0, 1
    good, bad = s.tables.copy(), s.tables.copy()
    good[0, 2], bad[0, 2] = zero, s.nb + 5
    s.tables = good
    cache = s.cache()
    want = s.run(cache=cache)
    check(want, *s.reference(), "a block of zeros")
    q, cu, ctxs, _ = s.meta()
    noise = [Step([(q_len, 900), (q_len, 400)], hq, hk, a, seed=i, vspread=60) for i in (20, 21)]
    noise[1].v_exps[:] = 255
    noise[1].k_exps[:] = 255
    for n in noise + noise[::-1]:
        n.run(cache=n.cache())
        out = s.run(cache=cache, meta=(q, cu, ctxs, torch.from_numpy(bad).cuda()), status=lib.CB_EDEVICE)
        assert torch.equal(out, want)


def test_lengths_that_count_tokens_many_times():
    """cu_q_lens that jumps back and forth: 33 requests of all 65,536 tokens at
    2^20 keys each would be more key tiles than 32 bits count.  Nothing is read or
    written; the error is reported, and the next call runs as ever."""
    lib = L()
    n, hq, ctx = 65536, 32, 1 << 20
    tables = torch.zeros(66, (ctx + n) // 16, dtype=torch.int32, device="cuda")
    cu = torch.tensor([0, n] * 33 + [0], dtype=torch.int32, device="cuda")
    ctxs = torch.full((66,), ctx, dtype=torch.int32, device="cuda")
    s = Step([(3, 20), (1, 64)], hq, 1, 128, seed=25)
    cache = s.cache()
    q = torch.zeros(n, hq, 128, dtype=torch.bfloat16, device="cuda")
    out = torch.full_like(q, 3.0)
    ws = torch.empty(lib.cb_paged_attention_fp8_workspace_size(66, n, n, ctx + n, hq, 1, 128, 16), dtype=torch.uint8, device="cuda")
    lib.cb_paged_attention_fp8(q, cu, ctxs, tables, *cache, out, 0.1, ws, n, ctx + n)
    assert lib.cb_last_error() == lib.CB_EDEVICE
    assert (out == 3.0).all()
    check(s.run(cache=cache), *s.reference(), "the next call")
