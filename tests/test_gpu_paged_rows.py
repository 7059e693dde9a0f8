"""The paged cache as a server holds it: entries that are no pages."""
import pytest
import torch

from block_sparse_long_score_b200 import xattn_get_device_status, xattn_paged_plan

pytestmark = pytest.mark.gpu

DEV = "cuda:0"


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------ plan

@pytest.mark.parametrize("n", [3, 1500])
@pytest.mark.parametrize("bad", [-1, 10, 1 << 20, -(1 << 31)])
def test_plan_reports_what_an_ended_request_gives_back(n, bad):
    """Request 0 ends with an entry that is no page: it goes to the ring as it is, and the
    step reports it."""
    fill = n - 3
    lens, fresh = [20, 16, 5] + [0] * fill, [-1, 0, 1] + [0] * fill
    table = [[3, bad], [1, -1], [2, -1]] + [[-1, -1]] * fill
    t = [_i32(x) for x in (lens, fresh, [8, 3], [6, 0, 0, 0, 0, 0, 0, 0, 4, 5], table)]
    out = (t[0], t[2], _i32([7] * (n + 1)), _i32([7] * 2))
    assert xattn_get_device_status() == 0
    xattn_paged_plan(*t, 16, out=out)
    torch.cuda.synchronize()
    assert xattn_get_device_status() == -1
    assert out[0].tolist() == [0, 16, 6] + [0] * fill and out[1].tolist() == [8, 5]
    assert out[2].tolist() == [0, 0, 0, 1] + [1] * fill and out[3].tolist() == [37, -1]
    assert t[3].tolist() == [6, 3, bad, 0, 0, 0, 0, 0, 4, 5] and t[4].tolist() == table
