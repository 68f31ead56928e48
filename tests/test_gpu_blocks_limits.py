"""The block pool's calls at the ends of what their arguments may be."""
import pytest
import torch

from gpu_util import L

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def test_slots_of_the_most_tokens():
    """A step padded to 2^31 - 1 tokens: the number of CTAs that write the slots is not counted past 32 bits."""
    lib = L()
    tables = torch.full((2, 4), -1, dtype=torch.int32, device="cuda")
    lens, refs, ctx = _ints(0, 0), torch.zeros(9, dtype=torch.int32, device="cuda"), _ints(7, 7)
    slots = torch.zeros((1 << 31) - 1, dtype=torch.int64, device="cuda")            # 17 GB
    ws = torch.zeros(lib.cb_block_ops_workspace_size(2, 4, 9), dtype=torch.uint8, device="cuda")
    lib.cb_grow_blocks(_ints(0, 20, 23), tables, lens, refs, ctx, slots, ws)
    assert lib.cb_last_error() == 0
    assert lens.tolist() == [20, 3] and ctx.tolist() == [0, 0] and refs.tolist() == [1, 1, 1] + [0] * 6
    assert slots[:23].tolist() == list(range(20)) + [32, 33, 34]
    assert int(slots[23:].max()) == -1 and int(slots[23:].min()) == -1
