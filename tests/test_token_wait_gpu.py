"""The token attention's bounded waits, made to run out on purpose without a fault: through
the test entry point some warps fetch nothing, so that they wait for copies that nobody
started. The call must report VELOX_STATUS_TIMEOUT, write nothing but its outputs and its
workspace, and leave the device usable: the next call gives the oracle's output with a clean
status."""
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as to
from tests.test_token_ops_gpu import attn_state, check_attn, host, i32, vx  # noqa: F401

pytestmark = pytest.mark.gpu

CASES = {  # H, Hkv, d, page, lens, pages that the table is wider than it need be
    "a CTA a row": (64, 64, 64, 16, [470, 0, 300, 37], 0),
    "clusters of a short history": (4, 2, 128, 32, [400, 90], 0),
    "clusters of one request": (24, 24, 128, 64, [3001], 200),
    "dealt out by length": (8, 2, 64, 16, [700, 3, 0, 2049], 300),
    "sixteen heads to a key head": (16, 1, 128, 64, [333, 1, 4097], 100),
}


NEED_NONE = ("a CTA a row", "clusters of a short history")


@pytest.mark.parametrize("name,workspace", [(n, True) for n in CASES] + [(n, False) for n in NEED_NONE])
def test_expired_waits_report_timeout_and_write_nothing_else(vx, name, workspace):  # noqa: F811
    H, Hkv, d, page, lens, wider = CASES[name]
    R = len(lens)
    kp, vp, table, _ = attn_state(R, Hkv, d, page, lens, seed=H + d)
    table = np.concatenate([table, np.full((R, wider), -1)], 1)
    needs_none = vx._needs_no_workspace(R * Hkv * -(-H // Hkv // 16), table.shape[1] * page)
    assert needs_none == (name in NEED_NONE)
    q = torch.randn(R, H, d, device="cuda").to(torch.bfloat16)
    t, n = i32(table), i32(lens)
    # a workspace of the size that the path needs: none at all, or what the library names
    size = 256 if needs_none else vx.lib.velox_paged_attn_workspace_size(R, H, Hkv, d)
    room = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = room[:size] if workspace else None
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    want = to.token_attention(host(q), host(kp), host(vp), table, lens)
    k0, v0 = kp.view(torch.int16).clone(), vp.view(torch.int16).clone()
    for skip in (1, 8, 2, 4, 6, 9, 15):     # the warp that begins a row, the one that ends it, ...
        vx.paged_attn_test(q, kp, vp, t, n, status, 0.02, skip, ws=ws)
        torch.cuda.synchronize()
        assert int(status.item()) == vx.VELOX_STATUS_TIMEOUT
        status.zero_()
        assert (room[size:] == 0xA5).all()
        if needs_none:
            assert (room == 0xA5).all()     # a row of one CTA or cluster leaves the workspace alone
        o, lse = vx.paged_attn(q, kp, vp, t, n, status=status)
        assert int(status.item()) == 0
        check_attn(o, lse, want, lens, 1 / math.sqrt(d), d, name)
    o2, l2 = vx.paged_attn_test(q, kp, vp, t, n, status, 2.0, 0, ws=ws)
    assert int(status.item()) == 0 and torch.equal(o, o2) and torch.equal(lse, l2)
    assert torch.equal(kp.view(torch.int16), k0) and torch.equal(vp.view(torch.int16), v0)
