"""The token attention over batches larger than the lengths that a thread keeps: the kernels
look at the others twice (the attention from 513 requests on, its join from 1,025)."""
import math
import os
import subprocess
import sys

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


@pytest.mark.parametrize("most", [1, 8, 9, 10, 16])
@pytest.mark.parametrize("H,Hkv,d", [(24, 24, 128), (12, 12, 64), (32, 2, 128), (160, 10, 128)])
def test_one_request_where_large_clusters_cannot_be_placed(vx, H, Hkv, d, most):  # noqa: F811
    """A device that places no cluster of 16 or 10 CTAs (a part of a GPU) takes smaller ones, or
    deals the rows out by length: the same results up to rounding."""
    page, n = 64, 3001
    kp, vp, table, _ = attn_state(1, Hkv, d, page, [n], seed=H)
    table = np.concatenate([table, np.full((1, 200), -1)], 1)
    q = torch.randn(1, H, d, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ws = vx.paged_attn_workspace(1, H, Hkv, d)
    o, lse = vx.paged_attn_test(q, kp, vp, i32(table), i32([n]), status, 2.0, 0, ws=ws, most_cluster=most)
    assert flags(vx, status) == 0
    check_attn(o, lse, to.token_attention(host(q), host(kp), host(vp), table, [n]), [n], 1 / math.sqrt(d), d)
    if most == 16:
        o2, l2 = vx.paged_attn(q, kp, vp, i32(table), i32([n]))
        assert torch.equal(o, o2) and torch.equal(lse, l2)


FIRST_CALL = """
import torch
from geometry_routed_block_b200 import velox as vx
torch.manual_seed(0)
H, d = 24, 128
kp, vp = (torch.randn(50, H, 64, d, device="cuda").to(torch.bfloat16) for _ in range(2))
q = torch.randn(1, H, d, device="cuda").to(torch.bfloat16)
table = torch.arange(50, dtype=torch.int32, device="cuda")[None].repeat(1, 5).contiguous()
lens, out = torch.tensor([3001], dtype=torch.int32, device="cuda"), torch.zeros_like(q)
ws = vx.paged_attn_workspace(1, H, H, d)
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    vx.paged_attn(q, kp, vp, table, lens, ws=ws, out=out, want_lse=False)
g.replay()
assert torch.equal(out, vx.paged_attn(q, kp, vp, table, lens)[0]) and out.abs().sum() > 0
"""


def test_the_first_call_of_a_process_may_be_captured(vx):  # noqa: F811
    """What the library asks the device once (can it place a cluster?) is no part of a capture."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    subprocess.run([sys.executable, "-c", FIRST_CALL], cwd=root, check=True, timeout=300)
