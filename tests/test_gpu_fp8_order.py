"""The order of a call's kernels over the 8-bit cache: chunks beside single tokens
read the rows that the same call appends."""
import numpy as np
import pytest
import torch

from fp8_util import BS, Step
from gpu_util import L

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    L().lib()


def _slots(s):
    return torch.from_numpy(np.concatenate([s.tables[r, p // BS].astype(np.int64) * BS + p % BS for r, (q, c) in enumerate(s.reqs)
                                            for p in [c + np.arange(q)]])).cuda()


REQS = {"chunk": [(2000, 100)], "both": [(1, 300)] * 40 + [(700, 5), (300, 900)], "one": [(1, 3000), (2, 900)]}


@pytest.mark.parametrize("hq,hk,a", [(32, 8, 128), (32, 1, 128), (4, 4, 64)])
@pytest.mark.parametrize("reqs", list(REQS))
@pytest.mark.parametrize("recorded", [False, True])
def test_chunks_read_the_rows_of_their_own_call(hq, hk, a, reqs, recorded):
    """New rows in the same slots call after call: each call's output is, bit for
    bit, that of an append, a wait for the GPU and the attention."""
    lib = L()
    s = Step(REQS[reqs], hq, hk, a, seed=71)
    slots, meta, ws = _slots(s), s.meta(), s.workspace()
    cache = s.cache()
    n = s.q.shape[0]
    k, v = (torch.empty(n, hk, a, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    g = torch.Generator(device="cuda").manual_seed(1)
    out, want = torch.empty_like(meta[0]), torch.empty_like(meta[0])
    call = lambda: lib.cb_kv_append_paged_attention_fp8(k, v, slots, *meta, *cache, out, s.scale, ws, s.max_q, s.max_kv)  # noqa: E731
    k.zero_(), v.zero_()
    call()
    if recorded:
        st = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st, capture_error_mode="thread_local"):
            call()
        call = graph.replay
    for _ in range(20):
        k.normal_(generator=g), v.normal_(generator=g)
        torch.cuda.synchronize()
        call()
        torch.cuda.synchronize()
        lib.cb_kv_append_fp8(k, v, slots, *cache)
        torch.cuda.synchronize()
        lib.cb_paged_attention_fp8(*meta, *cache, want, s.scale, s.workspace(), s.max_q, s.max_kv)
        assert torch.equal(out, want)
    assert lib.cb_last_error() == 0


@pytest.mark.parametrize("fill", [0, 0xFF])
def test_a_call_leaves_its_workspace_without_a_ticket(fill):
    """The workspace's last 16 bytes, where the appended rows are announced, are
    clear after a call with chunks, so that a recorded call never finds the ticket
    of its own last run; without chunks they are not there."""
    lib = L()
    s = Step([(1, 90), (30, 100)], 32, 8, 128, seed=72)
    ws = s.workspace(fill=fill)
    s.run(workspace=ws)
    assert (ws[-16:-8] == 0).all() and (ws[-8:] == fill).all()
    one = lib.cb_paged_attention_fp8_workspace_size(2, 2, 1, 200, 32, 8, 128, BS)
    assert one + 16 < ws.numel()
