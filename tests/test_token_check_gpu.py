"""PagedCache.check() reads what calls on any stream reported."""
import pytest
import torch

from tests.test_token_ops_gpu import i32, vx  # noqa: F401

pytestmark = pytest.mark.gpu


def test_check_waits_for_calls_on_other_streams(vx):  # noqa: F811
    from geometry_routed_block_b200.paged import PagedCache
    c = PagedCache(1, 2, 1, 64, 16, 4, 4)
    add, side = i32([40, 40]), torch.cuda.Stream()      # six pages of four
    plan = c.new_plan(80)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):           # kernels loaded, nothing planned
        c.plan(torch.zeros_like(add), 80, out=plan)
        torch.cuda._sleep(1000)
    c.check()
    with torch.cuda.stream(side):
        torch.cuda._sleep(200_000_000)      # 0.1 s or more
        c.plan(add, 80, out=plan)
    with pytest.raises(vx.VeloxError):
        c.check()
    c.check()       # reported once
    assert c.lens.tolist() == [0, 0] and c.free_count.item() == 4
