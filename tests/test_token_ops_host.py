"""The token path without a GPU: what its calls refuse before launching
anything, the rotary frequencies (a host function) against the oracle, and the
oracle against closed forms."""
import ctypes
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as to

FAKE = ctypes.c_void_p(1 << 20)  # non-null, 256-byte aligned; never dereferenced
ODD = ctypes.c_void_p((1 << 20) + 1)
OFF2 = ctypes.c_void_p((1 << 20) + 2)
OK_PAST_CHECKS = -3  # no GPU here: a call that passes its checks fails at the CUDA runtime


@pytest.fixture(scope="module")
def vx():
    from geometry_routed_block_b200 import build
    build.build()
    from geometry_routed_block_b200 import velox
    return velox


def strides(*s):
    return (ctypes.c_int64 * len(s))(*s)


def spec(vx, **kw):
    a = dict(freqs=1 << 20, rot=64, style=0, axes=1, sections=(32, 0, 0), mscale=1.0, inverse=0, **{})
    a.update(kw)
    return vx._Rope(a["freqs"], a["rot"], a["style"], a["axes"], (ctypes.c_int * 3)(*a["sections"]),
                    a["mscale"], a["inverse"])


def rejects(call, code, **kw):
    assert call(**kw) == code, kw


BAD_SPECS = [
    (dict(freqs=None), -1), (dict(freqs=(1 << 20) + 4), -1), (dict(rot=63), -1), (dict(rot=66), -1),
    (dict(rot=-2), -1), (dict(style=2), -2), (dict(axes=0), -1), (dict(axes=4), -1),
    (dict(sections=(31, 0, 0)), -1), (dict(axes=2, sections=(33, -1, 0)), -1),
    (dict(axes=2, sections=(16, 17, 0)), -1), (dict(axes=3, sections=(2**31 - 1, 2**31 - 1, 34)), -1),
    (dict(mscale=float("nan")), -1), (dict(mscale=float("inf")), -1),
]


def test_rope_rejects(vx):
    ok = dict(x=FAKE, dtype=0, B=1, H=2, N=4, d=64, xs=strides(512, 256, 64), pos=FAKE, pa=4, pb=0,
              rope=spec(vx), y=FAKE, ys=strides(512, 256, 64))

    def call(**kw):
        a = {**ok, **kw}
        ref = ctypes.byref(a["rope"]) if a["rope"] is not None else None
        return vx.lib.velox_rope(a["x"], a["dtype"], a["B"], a["H"], a["N"], a["d"], a["xs"], a["pos"],
                                 a["pa"], a["pb"], ref, a["y"], a["ys"], None)

    for name in ("x", "y", "rope", "xs", "ys", "pos"):
        rejects(call, -1, **{name: None})
    for name in ("B", "H", "N", "d"):
        rejects(call, -1, **{name: 0})
    rejects(call, -1, d=4097)
    rejects(call, -1, B=1 << 16, N=1 << 16)
    rejects(call, -2, dtype=2)
    rejects(call, -1, x=ODD)
    rejects(call, -1, y=OFF2, dtype=1)
    rejects(call, -1, pos=OFF2)
    rejects(call, -1, xs=strides(-1, 256, 64))
    rejects(call, -1, ys=strides(512, 0, 64))   # two heads on one another
    for bad, code in BAD_SPECS:
        rejects(call, code, rope=spec(vx, **bad))
    if not torch.cuda.is_available():
        assert call() == OK_PAST_CHECKS
        assert call(xs=strides(0, 0, 0)) == OK_PAST_CHECKS  # a broadcast input
        assert call(rope=spec(vx, rot=0, sections=(0, 0, 0), freqs=None), pos=None) == OK_PAST_CHECKS


def test_append_rejects(vx):
    ok = dict(q=FAKE, k=FAKE, v=FAKE, dtype=0, N=4, H=4, Hkv=2, d=64, qs=strides(256, 64),
              ks=strides(128, 64), vs=strides(128, 64), slots=FAKE, pos=FAKE, rope=spec(vx), out=FAKE,
              kp=FAKE, vp=FAKE, page=16, num_pages=8)

    def call(**kw):
        a = {**ok, **kw}
        ref = ctypes.byref(a["rope"]) if a["rope"] is not None else None
        return vx.lib.velox_paged_append(a["q"], a["k"], a["v"], a["dtype"], a["N"], a["H"], a["Hkv"],
                                         a["d"], a["qs"], a["ks"], a["vs"], a["slots"], a["pos"], 4, ref,
                                         a["out"], a["kp"], a["vp"], a["page"], a["num_pages"], None, None)

    for name in ("k", "v", "qs", "ks", "vs", "slots", "pos", "out", "kp", "vp", "q"):
        rejects(call, -1, **{name: None})
    for name in ("N", "H", "Hkv", "d", "page", "num_pages"):
        rejects(call, -1, **{name: 0})
    rejects(call, -2, dtype=9)
    rejects(call, -2, page=24)
    rejects(call, -2, page=256)
    rejects(call, -2, d=96)
    rejects(call, -1, num_pages=2**27)          # 2^31 slots
    rejects(call, -1, kp=OFF2)
    rejects(call, -1, out=OFF2)
    rejects(call, -1, k=ODD)
    rejects(call, -1, slots=OFF2)
    rejects(call, -1, ks=strides(-128, 64))
    rejects(call, -1, Hkv=2**30, H=2**30)
    for bad, code in BAD_SPECS:
        rejects(call, code, rope=spec(vx, **bad))
    if not torch.cuda.is_available():
        assert call() == OK_PAST_CHECKS
        assert call(q=None, out=None, qs=None) == OK_PAST_CHECKS
        assert call(rope=None, pos=None) == OK_PAST_CHECKS
        assert call(k=OFF2) == OK_PAST_CHECKS   # aligned to its element


def test_plan_and_release_reject(vx):
    ok = dict(add=FAKE, lens=FAKE, table=FAKE, fl=FAKE, fc=FAKE, R=4, mp=8, page=16, np=32, n_cap=8,
              lo=FAKE, fo=FAKE, cu=FAKE, slots=FAKE)

    def plan(**kw):
        a = {**ok, **kw}
        return vx.lib.velox_paged_plan(a["add"], a["lens"], a["table"], a["fl"], a["fc"], a["R"], a["mp"],
                                       a["page"], a["np"], a["n_cap"], a["lo"], a["fo"], a["cu"],
                                       a["slots"], None, None, None, None)

    def release(**kw):
        a = {**ok, **kw}
        return vx.lib.velox_paged_release(a["add"], a["lens"], a["table"], a["fl"], a["fc"], a["R"],
                                          a["mp"], a["page"], a["np"], a["lo"], a["fo"], None, None)

    for call in (plan, release):
        for name in ("add", "lens", "table", "fl", "fc", "lo", "fo"):
            rejects(call, -1, **{name: None})
            rejects(call, -1, **{name: OFF2})
        for name in ("R", "mp", "page", "np"):
            rejects(call, -1, **{name: 0})
        rejects(call, -1, R=8193)
        rejects(call, -2, page=17)
        rejects(call, -1, mp=2**27)
        rejects(call, -1, np=2**27)
        if not torch.cuda.is_available():
            assert call() == OK_PAST_CHECKS
    rejects(plan, -1, n_cap=-1)
    rejects(plan, -1, cu=None)
    rejects(plan, -1, slots=None)


def test_attn_rejects(vx):
    ok = dict(q=FAKE, kp=FAKE, vp=FAKE, table=FAKE, lens=FAKE, R=2, H=8, Hkv=2, d=64, page=16, np=32,
              mp=300, scale=0.125, o=FAKE, lse=None, ws=FAKE, n=1 << 30)

    def call(**kw):
        a = {**ok, **kw}
        return vx.lib.velox_paged_attn(a["q"], a["kp"], a["vp"], a["table"], a["lens"], a["R"], a["H"],
                                       a["Hkv"], a["d"], a["page"], a["np"], a["mp"], a["scale"], a["o"],
                                       a["lse"], a["ws"], a["n"], None, None)

    for name in ("q", "kp", "vp", "table", "lens", "o", "ws"):
        rejects(call, -1, **{name: None})
        rejects(call, -1, **{name: OFF2})
    rejects(call, -1, lse=OFF2)
    for name in ("R", "H", "Hkv", "d", "page", "np", "mp"):
        rejects(call, -1, **{name: 0})
    rejects(call, -1, R=65536)
    rejects(call, -1, H=7)                      # not a multiple of the key heads
    rejects(call, -1, H=1)
    rejects(call, -2, d=32)
    rejects(call, -2, page=8)
    rejects(call, -1, scale=0.0)
    rejects(call, -1, scale=float("nan"))
    rejects(call, -1, np=2**26)                 # rows of the pool: 2^31
    rejects(call, -1, mp=2**27)
    rejects(call, -1, R=65535, H=2**16)
    need = vx.lib.velox_paged_attn_workspace_size(2, 8, 2, 64)
    assert need > 0
    rejects(call, -1, n=need - 1)
    rejects(call, -1, ws=ctypes.c_void_p((1 << 20) + 16))
    if not torch.cuda.is_available():
        assert call(n=need) == OK_PAST_CHECKS
        # short histories of few rows need no workspace: 512 tokens for each CTA a row can have
        for R, mp in ((2, 256), (16, 256), (17, 128), (32, 128), (33, 64), (64, 64), (65, 32), (128, 32)):
            assert call(mp=mp, R=R, ws=None, n=0) == OK_PAST_CHECKS
    for R, mp in ((2, 257), (16, 257), (17, 129), (32, 129), (33, 65), (64, 65), (65, 33), (128, 33), (129, 1)):
        rejects(call, -1, mp=mp, R=R, ws=None, n=0)
        assert not vx._needs_no_workspace(R * 2, mp * 16)
        assert vx._needs_no_workspace(R * 2, (mp - 1) * 16)
    rejects(call, -1, mp=4, page=128, R=8, H=40 * 17, Hkv=17, ws=None, n=0)  # three tiles of heads
    for bad in ((0, 8, 2, 64), (2, 7, 2, 64), (2, 8, 0, 64), (2, 8, 2, 96), (65536, 8, 2, 64)):
        assert vx.lib.velox_paged_attn_workspace_size(*bad) == 0


def test_freqs_match_the_oracle(vx):
    for rot in (2, 16, 42, 64, 128):
        for scaling, kw in (("plain", {}), ("linear", dict(factor=8.0)), ("base", dict(factor=4.0)),
                            ("bands", dict(factor=16.0, orig_len=4096)),
                            ("bands", dict(factor=2.0, orig_len=7, beta_fast=1.5, beta_slow=0.01))):
            if rot == 2 and scaling == "base":
                continue
            got, m = vx.rope_freqs(rot, 10000.0, scaling, device="cpu", **kw)
            want, wm = to.freqs(rot, 10000.0, scaling, **kw)
            assert got.dtype == torch.float64 and got.shape == (rot // 2,)
            # pow and log of the two libraries: a few units in the last place each
            assert np.allclose(got.numpy(), want, rtol=1e-13, atol=0)
            assert abs(m - wm) <= 2**-23 * wm


def test_freqs_rejects(vx):
    f = (ctypes.c_double * 64)()
    call = lambda rot=64, base=1e4, kind=0, factor=1.0, n=0, bf=32.0, bs=1.0, out=f: (  # noqa: E731
        vx.lib.velox_rope_freqs(rot, base, kind, factor, n, bf, bs, out, None))
    assert call() == 0
    for bad in (dict(rot=0), dict(rot=7), dict(rot=-2), dict(base=1.0), dict(base=float("inf")),
                dict(kind=1, factor=0.5), dict(kind=2, factor=float("nan")), dict(kind=2, rot=2, factor=2.0),
                dict(kind=3, factor=2.0, n=0), dict(kind=3, factor=2.0, n=10, bf=1.0, bs=1.0),
                dict(kind=3, factor=2.0, n=10, bs=0.0), dict(out=None)):
        assert call(**bad) == -1, bad
    assert call(kind=4) == -2
    with pytest.raises(ValueError):
        vx.rope_freqs(64, scaling="other", device="cpu")


def test_binding_refuses_host_tensors_and_wrong_shapes(vx):
    x = torch.zeros(1, 2, 4, 64, dtype=torch.bfloat16)
    pos, fr = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    with pytest.raises(ValueError, match="CUDA"):
        vx.rope(x, pos, fr)
    with pytest.raises(TypeError):
        vx.rope(x.half(), pos, fr)
    with pytest.raises(TypeError):
        vx.rope(x, pos.long(), fr)
    with pytest.raises(TypeError):
        vx.rope(x, pos, fr.float())
    with pytest.raises(ValueError):
        vx.rope(x, pos[:, :3].contiguous(), fr)
    with pytest.raises(ValueError):
        vx.rope(x, pos, fr, sections=(16, 16))      # two axes, positions of one
    with pytest.raises(ValueError):
        vx.rope(x, pos, fr, style="both")
    for bad in ((), (8, 8, 8, 8), (-1, 33), (2**32 + 32,)):
        with pytest.raises(ValueError):
            vx.rope(x, pos, fr, sections=bad)
    with pytest.raises(ValueError, match="dense"):
        vx.rope(torch.zeros(1, 2, 4, 128, dtype=torch.bfloat16)[..., ::2], pos, fr)
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pages = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    k = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        vx.paged_append(k, k, i(3), pages, pages)
    with pytest.raises(ValueError):
        vx.paged_append(k, k[:2], i(3), pages, pages)
    with pytest.raises(ValueError):
        vx.paged_append(k, k, i(2), pages, pages)
    with pytest.raises(ValueError, match="heads"):
        vx.paged_append(k[:, :1], k[:, :1], i(3), pages, pages)
    with pytest.raises(ValueError, match="pos"):
        vx.paged_append(k, k, i(3), pages, pages, freqs=fr)
    with pytest.raises(ValueError, match="out"):
        vx.paged_append(k, k, i(3), pages, pages, out=k)
    with pytest.raises(ValueError, match="CUDA"):
        vx.paged_plan(i(2), i(2), i(2, 4), i(8), i(1), 16, 2)
    with pytest.raises(ValueError):
        vx.paged_plan(i(3), i(2), i(2, 4), i(8), i(1), 16, 2)
    with pytest.raises(ValueError):
        vx.paged_plan(i(2), i(2), i(3, 4), i(8), i(1), 16, 2)
    with pytest.raises(ValueError):
        vx.paged_plan(i(2), i(2), i(2, 4), i(8), i(1), 16, 2**31)
    with pytest.raises(ValueError, match="CUDA"):
        vx.paged_release(i(2), i(2), i(2, 4), i(8), i(1), 16)
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        vx.paged_attn(q, pages, pages, i(2, 4), i(2))
    with pytest.raises(ValueError):
        vx.paged_attn(q, pages, pages, i(3, 4), i(2))
    with pytest.raises(ValueError):
        vx.paged_attn(q, pages, pages[:2], i(2, 4), i(2))
    with pytest.raises(TypeError):
        vx.paged_attn(q.float(), pages, pages, i(2, 4), i(2))
    with pytest.raises(ValueError, match="contiguous"):
        vx.paged_attn(q.transpose(0, 1).contiguous().transpose(0, 1), pages, pages, i(2, 4), i(2))


def test_shared_elements_are_found(vx):
    """_apart against the sets of addresses."""
    buf = torch.zeros(4000, dtype=torch.bfloat16)
    rng = np.random.default_rng(0)

    def addresses(t):
        idx = torch.arange(4000).as_strided(t.shape, t.stride(), t.storage_offset())
        return set(idx.flatten().tolist())

    seen = set()
    for _ in range(400):
        shape = tuple(int(i) for i in rng.integers(1, 4, 2)) + (int(rng.integers(1, 5)), 8)
        s = [int(i) for i in rng.permutation([8, 8 * shape[2] + 8, 8 * shape[2] * shape[1] * 2 + 64])]
        x = buf.as_strided(shape, (*s, 1), int(rng.integers(0, 300)))
        y = buf.as_strided(shape, (*s, 1) if rng.random() < 0.8 else (600, 100, 10, 1),
                           int(rng.integers(0, 300)))
        apart = vx._apart(x, y)
        shared = bool(addresses(x) & addresses(y))
        assert not (apart and shared), (shape, s, x.storage_offset(), y.storage_offset())
        if x.stride() == y.stride():
            assert apart != shared
        seen.add((apart, shared))
    assert (True, False) in seen and (False, True) in seen
    assert vx._apart(buf[:100], buf[100:200]) and not vx._apart(buf[:101], buf[100:201])


# ---------------------------------------------------------------- the oracle itself

def test_oracle_rope_closed_forms():
    x = np.random.default_rng(0).standard_normal((3, 5, 8))
    pos = np.zeros((1, 5), np.int64)
    f, _ = to.freqs(8)
    assert np.allclose(to.rope(x, pos, f, "half", (4,)), x)
    # position p of a pair with frequency pi/2 turns it p quarter turns
    y = to.rope(x, np.full((1, 5), 1), np.full(4, math.pi / 2), "interleaved", (4,))
    assert np.allclose(y[..., 0::2], -x[..., 1::2]) and np.allclose(y[..., 1::2], x[..., 0::2])
    # products of rotated queries and keys depend on the distance alone
    p = lambda n: to.rope(x, np.full((1, 5), n), f, "half", (4,))  # noqa: E731
    assert np.allclose((p(7) * p(3)).sum(-1), (p(104) * p(100)).sum(-1))
    back = to.rope(to.rope(x, np.full((1, 5), 9), f, "half", (4,), 2.0), np.full((1, 5), 9), f, "half",
                   (4,), 0.5, inverse=True)
    assert np.allclose(back, x)


def test_oracle_pages_and_attention():
    table = np.full((3, 4), -1)
    cu, slots, pos, req, lens, table, stack = to.plan([5, 0, 17], [0, 0, 0], table, range(8), 16, 24)
    assert cu == [0, 5, 5, 22] and lens == [5, 0, 17] and stack == [0, 1, 2, 3, 4]
    assert table[0, 0] == 7 and table[2, :2].tolist() == [6, 5]
    assert slots[:5] == [112, 113, 114, 115, 116] and slots[21:] == [80, -1, -1]
    assert pos[20:22] == [15, 16] and req[4:6] == [0, 2]
    assert to.plan([129, 0, 0], [0, 0, 0], np.full((3, 9), -1), range(8), 16, 200) is None
    lens, stack = to.release([0, 1, 1], lens, table, stack, 16)
    assert lens == [5, 0, 0] and stack == [0, 1, 2, 3, 4, 6, 5]
    rng = np.random.default_rng(1)
    kp, vp = rng.standard_normal((2, 8, 2, 16, 8))
    q = rng.standard_normal((2, 4, 8))
    o, lse, _, _ = to.token_attention(q, kp, vp, np.array([[3, 5], [1, -1]]), [20, 0])
    assert (o[1] == 0).all() and np.isneginf(lse[1]).all()
    k = np.concatenate([kp[3], kp[5]], 1)[:, :20]
    s = torch.einsum("hgd,hnd->hgn", torch.tensor(q[0].reshape(2, 2, 8)), torch.tensor(k)) / math.sqrt(8)
    v = torch.tensor(np.concatenate([vp[3], vp[5]], 1)[:, :20])
    assert np.allclose(o[0].reshape(2, 2, 8), (s.softmax(-1) @ v).numpy())
