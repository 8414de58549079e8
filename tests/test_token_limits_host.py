"""Limits of the token calls that are checked before anything is launched, without a GPU."""
import ctypes
import math
import time

import numpy as np
import pytest
import torch

from tests.test_token_ops_host import FAKE, OFF2, OK_PAST_CHECKS, rejects, spec, strides, vx  # noqa: F401


def attn_args(**kw):
    a = dict(q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, R=2, H=8, Hkv=2, d=64, page=16, np=32,
             mp=300, scale=0.125, o=FAKE, lse=None, ws=FAKE, n=1 << 30, status=FAKE)
    a.update(kw)
    return list(a.values())


def test_attn_test_entry_rejects(vx):  # noqa: F811
    def call(limit=1.0, skip=0, most=16, **kw):
        return vx.lib.velox_paged_attn_test(*attn_args(**kw), limit, skip, most, None)

    for bad in (0.0, -1.0, 20.0, float("nan"), 1e-4):
        rejects(call, -1, limit=bad)
    for bad in (-1, 16):
        rejects(call, -1, skip=bad)
    for bad in (0, 17):
        rejects(call, -1, most=bad)
    rejects(call, -1, q=None)
    rejects(call, -2, page=8)
    rejects(call, -1, ws=None)
    if not torch.cuda.is_available():
        assert call(limit=1e-3, skip=15) == OK_PAST_CHECKS


def test_attn_step_rejects(vx):  # noqa: F811
    def call(cu=FAKE, N=3, **kw):
        a = attn_args(**kw)
        return vx.lib.velox_paged_attn_step(*a[:5], cu, a[5], N, *a[6:], None)

    rejects(call, -1, cu=None)
    rejects(call, -1, cu=OFF2)
    rejects(call, -1, N=0)
    rejects(call, -1, N=2**28)          # 2^31 rows of heads
    rejects(call, -1, R=65536)
    rejects(call, -1, lens=None)
    rejects(call, -2, d=32)
    if not torch.cuda.is_available():
        assert call() == OK_PAST_CHECKS
        assert call(N=1) == OK_PAST_CHECKS


def test_binding_refuses_rows_that_are_not_the_requests(vx):  # noqa: F811
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="table"):
        vx.paged_attn(q, pages, pages, i(2, 4), i(2))          # three rows, two requests, no plan
    with pytest.raises(ValueError, match="cu"):
        vx.paged_attn(q, pages, pages, i(2, 4), i(2), cu=i(2))
    with pytest.raises(TypeError, match="cu"):
        vx.paged_attn(q, pages, pages, i(2, 4), i(2), cu=i(3).long())
    with pytest.raises(ValueError, match="CUDA"):
        vx.paged_attn(q, pages, pages, i(2, 4), i(2), cu=i(3))


def test_sibling_slices_are_told_apart_at_once(vx):  # noqa: F811
    """An output on the sibling slice of a fused projection, as rope(out=) checks it in every
    call: the time does not grow with the tokens (it did, to 25 ms at 46,080)."""
    heads, d = 4, 8
    for tokens in (46_080, 300_000):
        wide = torch.empty(1, tokens, 3 * heads, d, dtype=torch.bfloat16)
        q, k = (wide[:, :, i * heads:(i + 1) * heads].transpose(1, 2) for i in range(2))
        best = math.inf
        for _ in range(7):
            t = time.perf_counter()
            assert vx._apart(q, k)
            best = min(best, time.perf_counter() - t)
        assert best < 1e-3
        assert not vx._apart(q, wide[:, :, 1:heads + 1].transpose(1, 2))


def test_shared_elements_of_any_strides(vx):  # noqa: F811
    """_apart against the sets of addresses: strides that nest or do not, broadcast dimensions."""
    rng = np.random.default_rng(1)
    buf = torch.zeros(6000, dtype=torch.float32)
    count = {True: 0, False: 0}
    for _ in range(3000):
        shape = tuple(int(i) for i in rng.integers(1, 6, 3)) + (int(rng.integers(1, 6)),)
        s = tuple(int(i) for i in rng.choice([0, 1, 2, 3, 5, 6, 7, 12, 30, 31, 64, 200], 3)) + (1,)
        x, y = (buf.as_strided(shape, s, int(rng.integers(0, 400))) for _ in range(2))
        at = [set(torch.arange(6000).as_strided(shape, s, t.storage_offset()).flatten().tolist()) for t in (x, y)]
        apart = not (at[0] & at[1])
        assert vx._apart(x, y) == apart, (shape, s, x.storage_offset(), y.storage_offset())
        count[apart] += 1
    assert min(count.values()) > 200


def test_rotary_heads_whose_counters_would_pass_32_bits_are_refused(vx):  # noqa: F811
    """A part of the heads ends at first + heads a part, and 8 are taken at a time: neither may
    pass 2^31."""
    def rope(H):
        return vx.lib.velox_rope(FAKE, 0, 1, H, 1, 1, strides(0, 0, 0), None, 1, 0,
                                 ctypes.byref(spec(vx, rot=0, sections=(0, 0, 0), freqs=None)), FAKE,
                                 strides(0, 1, 1), None)

    def append(H, Hkv):
        return vx.lib.velox_paged_append(FAKE, FAKE, FAKE, 0, 1, H, Hkv, 64, strides(64, 64), strides(64, 64),
                                         strides(64, 64), FAKE, None, 1, None, FAKE, FAKE, FAKE, 16, 8, None,
                                         None)

    assert rope(2**31 - 1) == -1 and rope(2**30 + 1) == -1
    assert append(2**30, 1) == -1 and append(1, 2**29) == -1
    if not torch.cuda.is_available():
        assert rope(2**30) == OK_PAST_CHECKS and append(2**30 - 2, 1) == OK_PAST_CHECKS


def test_attn_refuses_scales_that_leave_float32(vx):  # noqa: F811
    """The kernel multiplies scores by scale * log2(e): infinite above 2.36e38, all scores of 0
    then became NaN."""
    def call(scale):
        return vx.lib.velox_paged_attn(*attn_args(scale=scale), None)

    assert call(2.4e38) == -1 and call(3.4e38) == -1
    if not torch.cuda.is_available():
        assert call(2.3e38) == OK_PAST_CHECKS


def test_misaligned_words_are_refused(vx):  # noqa: F811
    def plan(**kw):
        a = dict(add=FAKE, lens=FAKE, table=FAKE, fl=FAKE, fc=FAKE, R=4, mp=8, page=16, np=32, n_cap=8,
                 lo=FAKE, fo=FAKE, cu=FAKE, slots=FAKE, pos=FAKE, req=FAKE, status=FAKE)
        return vx.lib.velox_paged_plan(*{**a, **kw}.values(), None)

    def release(**kw):
        a = dict(done=FAKE, lens=FAKE, table=FAKE, fl=FAKE, fc=FAKE, R=4, mp=8, page=16, np=32, lo=FAKE,
                 fo=FAKE, status=FAKE)
        return vx.lib.velox_paged_release(*{**a, **kw}.values(), None)

    def append(**kw):
        a = dict(q=None, k=FAKE, v=FAKE, dtype=0, N=4, H=0, Hkv=2, d=64, qs=None, ks=strides(128, 64),
                 vs=strides(128, 64), slots=FAKE, pos=None, pa=0, rope=None, out=None, kp=FAKE, vp=FAKE,
                 page=16, np=8, status=FAKE)
        return vx.lib.velox_paged_append(*{**a, **kw}.values(), None)

    def attn(**kw):
        return vx.lib.velox_paged_attn(*attn_args(**kw), None)

    for name in ("cu", "slots", "pos", "req"):
        rejects(plan, -1, **{name: OFF2})
    for call in (plan, release, append, attn):
        rejects(call, -1, status=OFF2)
        if not torch.cuda.is_available():
            assert call() == OK_PAST_CHECKS and call(status=None) == OK_PAST_CHECKS
