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
