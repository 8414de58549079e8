"""The README's token example, run as it stands, with scaled positions and an idle request."""
import math
import os
import re
import types

import numpy as np
import pytest
import torch

from oracle import token_oracle as to
from tests.test_token_ops_gpu import check_attn, host, i32, rope_tolerance, vx  # noqa: F401

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_the_example_gives_what_the_oracle_gives(vx):  # noqa: F811
    with open(README) as f:
        block, = [b for b in re.findall(r"```python\n(.*?)```", f.read(), re.S) if "PagedCache" in b]
    block, end, last = block.partition("cache.release(")
    R, H, Hkv, d, n_cap = 3, 4, 2, 128, 6
    scaling = dict(scaling="bands", factor=16.0, orig_len=64)
    scaled = types.SimpleNamespace(rope_freqs=lambda rot: vx.rope_freqs(rot, **scaling))
    f, mscale = to.freqs(d, **scaling)
    q, k, v = (torch.randn(n_cap, h, d, device="cuda").to(torch.bfloat16) for h in (H, Hkv, Hkv))
    add = [2, 0, 3]
    ns = dict(vx=scaled, torch=torch, layers=1, layer=0, R=R, Hkv=Hkv, H=H, n_cap=n_cap, q=q, k=k, v=v,
              new_tokens=i32(add), done=i32([1, 0, 0]))
    exec(block, ns)
    c, plan, o = ns["cache"], ns["plan"], ns["o"]
    c.check()
    pos = plan.pos.cpu().numpy()[None, :5, None]
    assert mscale > 1.2
    for x, got in ((q, ns["q"][:5]), (k, c.k[0][plan.slots[:5].long() // 128, :, plan.slots[:5].long() % 128])):
        want = to.rope(host(x[:5]), pos, f, "half", (d // 2,), mscale)
        assert (np.abs(host(got) - want) <= rope_tolerance(host(x[:5]), want, mscale, d, "half", True)).all()
    rows, lens = [1, 4], [2, 3]
    table = c.table.cpu().numpy()[[0, 2], :1]
    pages = [int(i) for i in table[:, 0]]
    want = to.token_attention(host(ns["q"][rows]), host(c.k[0][pages]), host(c.v[0][pages]),
                              np.array([[0], [1]]), lens)
    check_attn(o[rows], None, want, lens, 1 / math.sqrt(d), d)
    assert (o[[0, 2, 3, 5]] == 0).all()
    exec(end + last, ns)
    c.check()
    assert c.lens.tolist() == [0, 0, 3] and c.free_count.item() == 4095
