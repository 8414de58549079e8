"""The token calls at the largest sizes that their checks admit."""
import pytest
import torch

from tests.test_token_ops_gpu import i32, vx  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("in_place", [False, True])
def test_plan_with_room_for_2_31_tokens(vx, in_place):  # noqa: F811
    """n_cap = 2^31 - 1, where the grid's step behind the last token passes 32 bits. Only the
    slots are asked for (8.6 GB), with words behind them that must stay."""
    n_cap, page, num, behind = 2 ** 31 - 1, 128, 40, 1 << 20
    slots = torch.full((n_cap + behind,), 7, dtype=torch.int32, device="cuda")
    add, lens, table = i32([5, 0, 300]), i32([1, 0, 130]), i32([[39, -1, -1, -1], [-1] * 4, [38, 37, -1, -1]])
    fl, fc, status = torch.arange(num, dtype=torch.int32, device="cuda"), i32([37]), i32([0])
    lens_out, fc_out = (lens, fc) if in_place else (torch.empty_like(lens), torch.empty_like(fc))
    cu = torch.empty(4, dtype=torch.int32, device="cuda")
    p = lambda t: t.data_ptr()  # noqa: E731
    rc = vx.lib.velox_paged_plan(p(add), p(lens), p(table), p(fl), p(fc), 3, 4, page, num, n_cap, p(lens_out),
                                 p(fc_out), p(cu), p(slots), None, None, p(status),
                                 torch.cuda.current_stream().cuda_stream)
    assert rc == 0 and status.item() == 0
    assert cu.tolist() == [0, 5, 5, 305] and lens_out.tolist() == [6, 0, 430] and fc_out.item() == 35
    assert slots[:5].tolist() == [39 * 128 + i for i in range(1, 6)]
    want = [id_ * 128 + t % 128 for t in range(130, 430) for id_ in [(38, 37, 36, 35)[t // 128]]]
    assert slots[5:305].tolist() == want
    step = 1 << 28
    assert all((slots[a:min(a + step, n_cap)] == -1).all() for a in range(305, n_cap, step))
    assert (slots[n_cap:] == 7).all()
