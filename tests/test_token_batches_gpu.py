"""The token attention over batches larger than the lengths that a thread keeps: the kernels
look at the others twice (the attention from 513 requests on, its join from 1,025)."""
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as to
from tests.test_token_ops_gpu import attn_state, check_attn, flags, host, i32, vx  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,H,Hkv,d,most", [(2500, 2, 1, 64, 40), (2100, 4, 2, 128, 3), (65535, 1, 1, 64, 1)])
def test_large_batches_with_long_rows(vx, R, H, Hkv, d, most):  # noqa: F811
    """Short requests, some of none, and a few rows long enough to be shared by CTAs: the first,
    the last, and some in between that only the second look finds."""
    page = 16
    rng = np.random.default_rng(R)
    lens = rng.integers(0, most + 1, R)
    lens[rng.random(R) < 0.3] = 0
    lens[[0, 5, R // 2, R // 2 + 6, R - 2, R - 1]] = (9000, 700, 4000, 0, 3001, 5000)
    lens = lens.tolist()
    kp, vp, table, _ = attn_state(R, Hkv, d, page, lens, seed=R)
    q = torch.randn(R, H, d, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    o, lse = vx.paged_attn(q, kp, vp, i32(table), i32(lens), status=status)
    assert flags(vx, status) == 0
    want = to.token_attention(host(q), host(kp), host(vp), table, lens)
    check_attn(o, lse, want, lens, 1 / math.sqrt(d), d)
    o2, _ = vx.paged_attn(q, kp, vp, i32(table), i32(lens))
    assert torch.equal(o, o2)
