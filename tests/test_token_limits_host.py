"""Limits of the token calls that are checked before anything is launched, without a GPU."""
import ctypes

import pytest
import torch

from tests.test_token_ops_host import FAKE, OFF2, OK_PAST_CHECKS, rejects, vx  # noqa: F401


def attn_args(**kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, R=2, H=8, Hkv=2, d=64, page=16, np=32,
             mp=300, scale=0.125, o=FAKE, lse=None, ws=FAKE, n=1 << 30, status=FAKE)
    a.update(kw)
    return list(a.values())


def test_attn_test_entry_rejects(vx):  # noqa: F811
    def call(limit=1.0, skip=0, **kw):
        return vx.lib.velox_paged_attn_test(*attn_args(**kw), limit, skip, None)

    for bad in (0.0, -1.0, 20.0, float("nan"), 1e-4):
        rejects(call, -1, limit=bad)
    for bad in (-1, 16):
        rejects(call, -1, skip=bad)
    rejects(call, -1, q=None)
    rejects(call, -2, page=8)
    rejects(call, -1, ws=None)
    if not torch.cuda.is_available():
        assert call(limit=1e-3, skip=15) == OK_PAST_CHECKS
