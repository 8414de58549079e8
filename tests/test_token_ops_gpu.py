"""GPU parity of the token path (rotary positions, paged cache, attention of one
new token) against the fp64 oracle, and its behaviour at the edges.

Tolerances, derived once:
  rotation  the reduced angle is a float32 of at most one half turn: off by 2^-25
            half turns = 9.4e-8 rad; sincospif and mscale add at most 1.8e-7 to the
            factors, two products and a sum 1.2e-7: together under 4e-7 (|a| + |b|)
            mscale; then one rounding to bf16, half a step: 2^-8 of the value.
  attention a score is an fp32 sum of d exact products: off by at most
            (d + 4) 2^-24 scale sum |q||k|; a weight by that (relative), by 2^-16
            (two bf16 and the exponential) and by (n + 64) 2^-24 (sums); an output by
            2 * that * sum p|v|, and by half a step of bf16. lse: the score's error,
            2^-19 absolute for sums and the logarithm, 2^-22 relative.
"""
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as to

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def vx():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from geometry_routed_block_b200 import velox
    return velox


def i32(a):
    return torch.tensor(np.asarray(a), dtype=I32, device="cuda")


def host(t):
    return t.detach().float().cpu().numpy().astype(np.float64) if t.is_floating_point() else t.cpu().numpy()


def flags(vx, status):
    bits = int(status.item())
    status.zero_()
    return bits


# ---------------------------------------------------------------- rotary positions

def freqs_for(sections):
    return np.concatenate([to.freqs(2 * s)[0] if s else np.zeros(0) for s in sections])


def rope_tolerance(x, y, mscale, rot, style, bf16):
    """Per element: (|a| + |b|) of its pair times 4e-7 mscale, and the rounding."""
    h = rot // 2
    mag = np.abs(x)
    tol = np.zeros_like(mag)
    if style == "half":
        pair = mag[..., :h] + mag[..., h:rot]
        tol[..., :h], tol[..., h:rot] = pair, pair
    else:
        pair = mag[..., 0:rot:2] + mag[..., 1:rot:2]
        tol[..., 0:rot:2], tol[..., 1:rot:2] = pair, pair
    return tol * 4e-7 * mscale + (2.0 ** -8 if bf16 else 2.0 ** -24) * np.abs(y)


ROPE_CASES = [
    # B, H, N, d, sections, layout
    (1, 2, 1, 64, (32,), "dense"),
    (2, 3, 17, 128, (64,), "dense"),
    (1, 24, 131, 128, (22, 21, 21), "dense"),
    (2, 5, 33, 64, (8,), "tokens"),          # part of the head; [B,N,H,d] memory
    (1, 4, 50, 128, (16, 8), "slice"),       # slices of a wider projection
    (1, 3, 29, 64, (5, 4, 0), "dense"),      # 18 rotated elements: one at a time
    (1, 2, 19, 80, (20,), "offset"),         # rows off the 16-byte boundaries
    (1, 1, 7, 2, (1,), "dense"),
    (1, 2, 5, 4096, (2048,), "dense"),
    (3, 2, 9, 72, (), "dense"),              # nothing rotated
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("case", ROPE_CASES, ids=lambda c: "-".join(map(str, c)))
def test_rope_matches_oracle(vx, case, style, dtype):
    B, H, N, d, sec, layout = case
    g = torch.Generator(device="cuda").manual_seed(N * d)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    if layout == "dense":
        x = rnd(B, H, N, d)
    elif layout == "tokens":
        x = rnd(B, N, H, d).transpose(1, 2)
    elif layout == "slice":
        x = rnd(B, N, 3 * H, d)[:, :, H:2 * H].transpose(1, 2)
    else:
        x = rnd(B, H, N, d + 3)[..., 1:d + 1]
    axes = max(1, len(sec))
    sec = sec or (0,)
    f = freqs_for(sec)
    rng = np.random.default_rng(d)
    pos = rng.integers(-5000, 300000, size=(axes, B, N))
    pos.flat[0] = 2 ** 31 - 1
    pos.flat[-1] = -2 ** 31
    for shared in (False, True):
        p = pos[:, 0] if shared else pos
        for inverse, mscale in ((False, 1.0), (True, 1.25)):
            y = vx.rope(x, i32(p), torch.tensor(f, device="cuda"), style=style, sections=sec,
                        mscale=mscale, inverse=inverse)
            assert y.shape == x.shape and y.dtype == dtype and y.is_contiguous()
            at = p[:, None, None, :] if shared else p[:, :, None, :]
            want = to.rope(host(x), at, f, style, sec, mscale, inverse)
            err = np.abs(host(y) - want)
            assert (err <= rope_tolerance(host(x), want, mscale, 2 * len(f), style,
                                          dtype == torch.bfloat16)).all(), err.max()
            rest = 2 * len(f)
            assert torch.equal(y[..., rest:], x[..., rest:])


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_in_place_strided_output_and_broadcast_input(vx, style, dtype):
    f = torch.tensor(freqs_for((16, 8)), device="cuda")
    x = torch.randn(2, 6, 37, 64, device="cuda").to(dtype)
    pos = i32(np.random.default_rng(0).integers(0, 9999, size=(2, 37)))
    kw = dict(style=style, sections=(16, 8))
    want = vx.rope(x, pos, f, **kw)
    y = x.clone()
    assert vx.rope(y, pos, f, out=y, **kw) is y and torch.equal(y, want)
    wide = torch.full((2, 37, 8, 64), 7.0, device="cuda").to(dtype)  # out: heads 1..6 of 8
    vx.rope(x, pos, f, out=wide[:, :, 1:7].transpose(1, 2), **kw)
    assert torch.equal(wide[:, :, 1:7].transpose(1, 2), want)
    assert (wide[:, :, 0] == 7).all() and (wide[:, :, 7] == 7).all()
    one = x[:1, :1].expand(2, 6, 37, 64)
    assert torch.equal(vx.rope(one, pos, f, **kw), vx.rope(one.contiguous(), pos, f, **kw))
    with pytest.raises(ValueError):
        vx.rope(x, pos, f, out=x.as_strided(x.shape, (6 * 37 * 64, 64, 6 * 64, 1)), **kw)
    with pytest.raises(vx.VeloxError):
        vx.rope(x, pos, f, out=torch.empty_like(x[:, :1]).expand_as(x), **kw)


def test_rope_back_is_the_gradient(vx):
    """<rope(x), u> = <x, rope back(u)>, and differences of the (linear) forward call."""
    B, H, N, d, sec = 2, 3, 21, 64, (10, 6)
    f = torch.tensor(freqs_for(sec), device="cuda")
    pos = i32(np.random.default_rng(3).integers(0, 5000, size=(2, N)))
    kw = dict(style="interleaved", sections=sec, mscale=1.3)
    x, u = torch.randn(2, B, H, N, d, device="cuda")
    grad = vx.rope(u, pos, f, inverse=True, **kw)
    lhs = (vx.rope(x, pos, f, **kw).double() * u.double()).sum().item()
    rhs = (x.double() * grad.double()).sum().item()
    scale = 1.3 * float(x.double().norm() * u.double().norm())
    assert abs(lhs - rhs) <= 2e-6 * scale
    for at in ((0, 1, 5, 3), (1, 2, 20, 31), (1, 0, 0, 40)):  # the last is not rotated
        e = torch.zeros_like(x)
        e[at] = 1.0
        diff = ((vx.rope(x + e, pos, f, **kw) - vx.rope(x - e, pos, f, **kw)).double() * u.double()).sum() / 2
        # each of the two calls rounds every output (2^-24) and its factors (4e-7), on two elements
        assert abs(diff.item() - grad[at].item()) <= 2e-5


# ---------------------------------------------------------------- block tables, slots, pages back

def plan_state(lens, page, width, spare, seed):
    rng = np.random.default_rng(seed)
    used = [-(-n // page) for n in lens]
    num = sum(used) + spare
    ids = rng.permutation(num)
    table = np.full((len(lens), width), -1)
    at = 0
    for r, u in enumerate(used):
        table[r, :u] = ids[at:at + u]
        at += u
    free = ids[at:].tolist()
    return table, free, num


def run_plan(vx, add, lens, table, free, num, page, n_cap, **kw):
    fl = i32(free + [-7] * (num - len(free)))
    tab, status = i32(table), torch.zeros(1, dtype=I32, device="cuda")
    p = vx.paged_plan(i32(add), i32(lens), tab, fl, i32([len(free)]), page, n_cap, status=status, **kw)
    return p, tab, fl, flags(vx, status)


PLANS = [  # R, page, longest, most added, spare tokens in n_cap
    (1, 16, 0, 1, 0), (1, 128, 500, 4608, 3), (5, 16, 40, 1, 2), (48, 32, 900, 1, 0),
    (300, 64, 2000, 200, 1000), (1025, 16, 50, 3, 1), (8192, 16, 30, 2, 5),
]


@pytest.mark.parametrize("case", PLANS, ids=str)
def test_plan_and_release_match_oracle(vx, case):
    R, page, longest, most, pad = case
    rng = np.random.default_rng(R + page)
    lens = rng.integers(0, longest + 1, R)
    add = rng.integers(0, most + 1, R)
    if R > 3:
        lens[:3], add[:3] = (0, page, page - 1), (0, 0, 2)
    if R == 1:
        add[:] = most
    need = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, add))
    width = max(1, max(-(-(a + b) // page) for a, b in zip(lens, add)))
    table, free, num = plan_state(lens.tolist(), page, width, need + (R % 3), R)
    n_cap = int(add.sum()) + pad
    want = to.plan(add, lens, table, free, page, n_cap)
    p, tab, fl, bits = run_plan(vx, add, lens, table, free, num, page, n_cap)
    assert bits == 0
    for got, exp, name in zip((p.cu, p.slots, p.pos, p.req, p.lens, tab), want, "cu slots pos req lens table".split()):
        assert np.array_equal(got.cpu().numpy(), np.asarray(exp)), name
    assert p.free_count.item() == len(want[6])
    assert fl[:len(want[6])].tolist() == want[6]
    # pages back, in place
    done = rng.integers(0, 2, R)
    lens2, stack2 = to.release(done, want[4], want[5], want[6], page)
    lens_t, count_t, status = p.lens, p.free_count, torch.zeros(1, dtype=I32, device="cuda")
    vx.paged_release(i32(done), lens_t, tab, fl, count_t, page, lens_out=lens_t, free_count_out=count_t,
                     status=status)
    assert flags(vx, status) == 0
    assert lens_t.tolist() == list(map(int, lens2))
    assert count_t.item() == len(stack2) and fl[:len(stack2)].tolist() == stack2
    assert np.array_equal(tab.cpu().numpy(), want[5])


def test_plan_in_place_equals_out_of_place_and_allows_no_tokens(vx):
    lens, add, page = [3, 0, 31, 16], [2, 0, 3, 40], 16
    table, free, num = plan_state(lens, page, 8, 9, 0)
    a, tab_a, _, _ = run_plan(vx, add, lens, table, free, num, page, 64)
    lt, ct, tab = i32(lens), i32([len(free)]), i32(table)
    e = lambda n: torch.empty(n, dtype=I32, device="cuda")  # noqa: E731
    out = vx.PagedPlan(e(5), e(64), e(64), e(64), lt, ct)
    vx.paged_plan(i32(add), lt, tab, i32(free + [0] * (num - len(free))), ct, np.int64(page), np.int64(64),
                  out=out)
    for x, y in zip(a, out):
        assert torch.equal(x, y)
    assert torch.equal(tab, tab_a)
    none, tab_n, _, bits = run_plan(vx, [0] * 4, lens, table, free, num, page, 0)
    assert bits == 0 and none.cu.tolist() == [0] * 5 and none.lens.tolist() == lens
    assert np.array_equal(tab_n.cpu().numpy(), table)


@pytest.mark.parametrize("R,most,pad", [(3, 40, 0), (60, 100, 40), (300, 300, 3), (2000, 90, 77)])
@pytest.mark.parametrize("fits", [True, False])
def test_plan_and_release_in_place_at_every_size(vx, R, most, pad, fits):
    """One CTA, a cluster, and a grid with a second kernel: lengths and count in place, a
    plan that fits and one that does not, then all pages back."""
    page = 16
    rng = np.random.default_rng(R)
    lens, add = rng.integers(0, 200, R), rng.integers(0, most, R)
    need = sum(-(-(a + b) // page) - -(-a // page) for a, b in zip(lens, add))
    width = max(-(-(a + b) // page) for a, b in zip(lens, add))
    table, free, num = plan_state(lens.tolist(), page, width, need - (0 if fits else 1), R)
    n_cap = int(add.sum()) + pad
    want = to.plan(add, lens, table, free, page, n_cap)
    assert (want is not None) == fits
    lt, ct, tab, fl = i32(lens), i32([len(free)]), i32(table), i32(free + [0] * (num - len(free)))
    status = torch.zeros(1, dtype=I32, device="cuda")
    e = lambda n: torch.empty(n, dtype=I32, device="cuda")  # noqa: E731
    out = vx.PagedPlan(e(R + 1), e(n_cap), e(n_cap), e(n_cap), lt, ct)
    vx.paged_plan(i32(add), lt, tab, fl, ct, page, n_cap, out=out, status=status)
    assert flags(vx, status) == (0 if fits else vx.VELOX_STATUS_NO_SPACE)
    if fits:
        for got, exp in zip((*out[:5], tab), want):
            assert np.array_equal(got.cpu().numpy(), np.asarray(exp))
        lens, table, free = want[4], want[5], want[6]
    else:
        assert (out.slots == -1).all() and (out.cu == 0).all()
        assert np.array_equal(tab.cpu().numpy(), table)
    assert lt.tolist() == list(map(int, lens)) and ct.item() == len(free)
    done = rng.integers(0, 2, R)
    lens, free = to.release(done, lens, table, free, page)
    for what, code in ((done, 0), (np.ones(R, int), 0)):
        vx.paged_release(i32(what), lt, tab, fl, ct, page, lens_out=lt, free_count_out=ct, status=status)
        assert flags(vx, status) == code
        assert lt.tolist() == list(map(int, lens)) and ct.item() == len(free)
        assert fl[:len(free)].tolist() == free
        lens, free = to.release(np.ones(R, int), lens, table, free, page)
    assert sorted(free) == list(range(num))     # every page is free once
    ct.fill_(num + 1)
    lt.fill_(page)
    vx.paged_release(i32(done), lt, tab, fl, ct, page, lens_out=lt, free_count_out=ct, status=status)
    assert flags(vx, status) == vx.VELOX_STATUS_BAD_INDEX
    assert (lt == page).all() and ct.item() == num + 1


BAD_PLANS = [
    ("no page left", dict(add=[0, 200, 0]), 4),
    ("more tokens than room", dict(n_cap=4), 4),
    ("row of the table too short", dict(lens=[128, 5, 0], add=[1, 1, 1]), 4),
    ("negative add", dict(add=[1, -1, 2]), 1),
    ("negative length", dict(lens=[3, -1, 0]), 1),
    ("length beyond the row", dict(lens=[129, 5, 0]), 1),
    ("more free pages than pages", dict(count=1000), 1),
    ("fewer than none", dict(count=-1), 1),
    ("huge numbers", dict(add=[2**31 - 1, 2**31 - 1, 2**31 - 1]), 4),
]


@pytest.mark.parametrize("what,change,code", BAD_PLANS, ids=[b[0] for b in BAD_PLANS])
@pytest.mark.parametrize("n_cap", [8, 5000, 20000])
def test_plans_that_do_not_fit_change_nothing(vx, what, change, code, n_cap):
    page, width = 16, 8
    base = [3, 20, 0]
    table, free, num = plan_state(base, page, width, 6, 1)
    lens, add = change.get("lens", base), change.get("add", [2, 1, 2])
    if "n_cap" in change:
        n_cap = change["n_cap"]
    count, tab, fl = i32([change.get("count", len(free))]), i32(table), i32(free + [0] * (num - len(free)))
    lt, status = i32(lens), torch.zeros(1, dtype=I32, device="cuda")
    before = fl.clone()
    p = vx.paged_plan(i32(add), lt, tab, fl, count, page, n_cap, status=status)
    assert flags(vx, status) == code
    assert p.cu.tolist() == [0] * 4 and p.lens.tolist() == lens and p.free_count.item() == count.item()
    for t in (p.slots, p.pos, p.req):
        assert (t == -1).all()
    assert np.array_equal(tab.cpu().numpy(), table) and torch.equal(fl, before)


def test_plan_flags_page_ids_outside_the_pool(vx):
    page = 16
    table, free, num = plan_state([20, 5], page, 4, 3, 2)
    table[0, 1] = num           # the page that token 20 goes to
    free[-1] = -3               # the page that request 1 gets for its tokens 16..
    p, tab, _, bits = run_plan(vx, [1, 13], [20, 5], table, free, num, page, 16)
    assert bits == vx.VELOX_STATUS_BAD_INDEX
    s = p.slots.tolist()
    assert s[0] == -1 and all(x >= 0 for x in s[1:12]) and s[12:14] == [-1, -1] and s[14:] == [-1, -1]
    assert p.lens.tolist() == [21, 18]


def test_release_refuses_pages_given_back_twice(vx):
    page, lens = 16, [40, 33]
    table, free, num = plan_state(lens, page, 4, 2, 3)
    fl, status = i32(free + [0] * (num - len(free))), torch.zeros(1, dtype=I32, device="cuda")
    before = fl.clone()
    for lens_in, count, code in (([40, 33], len(free) + 1, 4), ([40, -1], len(free), 1),
                                 ([65, 33], len(free), 1), ([40, 33], -1, 1), ([40, 33], num + 1, 1)):
        lo, fo = vx.paged_release(i32([1, 1]), i32(lens_in), i32(table), fl, i32([count]), page, status=status)
        assert flags(vx, status) == code
        assert lo.tolist() == lens_in and fo.item() == count and torch.equal(fl, before)


# ---------------------------------------------------------------- append

APPENDS = [  # N, H, Hkv, d, page, sections, layout
    (1, 2, 2, 64, 16, (32,), "dense"),
    (37, 8, 2, 128, 16, (64,), "fused"),
    (130, 24, 24, 128, 64, (22, 21, 21), "heads"),
    (45, 6, 3, 64, 32, (8,), "fused"),
    (33, 4, 1, 128, 128, (5, 4), "dense"),     # 18 rotated elements: one at a time
    (20, 3, 3, 64, 16, (32,), "offset"),
    (9, 5, 1, 128, 32, None, "dense"),         # no rotation
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("case", APPENDS, ids=str)
def test_append_matches_oracle(vx, case, style, dtype):
    N, H, Hkv, d, page, sec, layout = case
    g = torch.Generator(device="cuda").manual_seed(N)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)  # noqa: E731
    if layout == "dense":
        q, k, v = rnd(N, H, d), rnd(N, Hkv, d), rnd(N, Hkv, d)
    elif layout == "fused":
        q, k, v = rnd(N, H + 2 * Hkv, d).split([H, Hkv, Hkv], 1)
    elif layout == "heads":
        q, k, v = (rnd(h, N, d).transpose(0, 1) for h in (H, Hkv, Hkv))
    else:
        q, k, v = (rnd(N, h, d + 1)[..., 1:] for h in (H, Hkv, Hkv))
    num = -(-N // page) + 4
    rng = np.random.default_rng(N + d)
    slots = rng.permutation(num * page)[:N]
    slots[rng.random(N) < 0.2] = -1
    if N > 5:
        slots[3], slots[4] = num * page, 2 ** 31 - 1   # outside: skipped and flagged
    kp, vp = (rnd(num, Hkv, page, d).to(torch.bfloat16) for _ in range(2))
    k0, v0 = kp.clone(), vp.clone()
    kw, pos = {}, None
    if sec:
        f = freqs_for(sec)
        pos = rng.integers(0, 10 ** 6, size=(len(sec), N))
        kw = dict(freqs=torch.tensor(f, device="cuda"), style=style, sections=sec, pos=i32(pos), mscale=1.1)
    status = torch.zeros(1, dtype=I32, device="cuda")
    out = vx.paged_append(k, v, i32(slots), kp, vp, q=q, status=status, **kw)
    assert flags(vx, status) == (vx.VELOX_STATUS_BAD_INDEX if N > 5 else 0)
    turn = lambda x: to.rope(host(x), pos[:, :, None], f, style, sec, 1.1) if sec else host(x)  # noqa: E731
    rot = 2 * sum(sec or ())

    def near(got, x, want):
        err = np.abs(host(got) - want)
        assert (err <= rope_tolerance(host(x), want, 1.1, rot, style, True)).all(), err.max()

    assert out.dtype == torch.bfloat16 and out.shape == (N, H, d)
    near(out, q, turn(q))
    wk, live = turn(k), (slots >= 0) & (slots < num * page)
    at = torch.tensor(slots[live], device="cuda")
    mine = torch.tensor(live, device="cuda")
    near(kp[at // page, :, at % page], k[mine], wk[live])
    assert torch.equal(vp[at // page, :, at % page], v[mine].to(torch.bfloat16))
    k0[at // page, :, at % page] = kp[at // page, :, at % page]
    v0[at // page, :, at % page] = vp[at // page, :, at % page]
    assert torch.equal(kp, k0) and torch.equal(vp, v0)   # nothing else was touched
    # without queries, and with the output given (it may be q itself)
    k1, v1 = kp.clone(), vp.clone()
    assert vx.paged_append(k, v, i32(slots), k1, v1, **kw) is None
    assert torch.equal(k1, kp) and torch.equal(v1, vp)
    qq = q.contiguous().clone()
    if dtype == torch.bfloat16:
        assert vx.paged_append(k, v, i32(slots), k1, v1, q=qq, out=qq, **kw) is qq
        assert torch.equal(qq, out)


# ---------------------------------------------------------------- attention of one new token

def attn_state(R, Hkv, d, page, lens, seed, spare=3, garbage=True):
    """Pages in a shuffled pool; rows behind each last token, and unused pages, hold NaN and inf."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    used = [-(-n // page) for n in lens]
    num = sum(used) + spare
    ids = np.random.default_rng(seed).permutation(num)
    width = max(1, max(used)) + 1
    table = np.full((R, width), -1)
    kp = torch.randn((num, Hkv, page, d), generator=g, device="cuda") + 0.5 * torch.randn(
        (Hkv, 1, d), generator=g, device="cuda")
    vp = torch.randn((num, Hkv, page, d), generator=g, device="cuda")
    at = 0
    fill = (float("nan"), float("inf"), -float("inf"))
    for r, n in enumerate(lens):
        table[r, :used[r]] = ids[at:at + used[r]]
        at += used[r]
        if garbage and n % page:
            last = int(table[r, used[r] - 1])
            kp[last, :, n % page:] = fill[r % 3]
            vp[last, :, n % page:] = fill[(r + 1) % 3]
    if garbage:
        kp[ids[at:].tolist()] = float("nan")
        vp[ids[at:].tolist()] = float("nan")
    return kp.to(torch.bfloat16), vp.to(torch.bfloat16), table, num


def check_attn(o, lse, want, lens, scale, d, label=""):
    wo, wl, pv, qk = want
    n = np.asarray(lens, np.float64)[:, None]
    e_s = (d + 4) * 2.0 ** -24 * qk
    delta = e_s + 2.0 ** -16 + (n + 64) * 2.0 ** -24
    err = np.abs(host(o) - wo)
    assert (err <= 2.0 ** -8 * np.abs(wo) + 2 * delta[..., None] * pv).all(), (label, err.max())
    if lse is not None:
        l = host(lse)
        empty = n[:, 0] == 0
        assert np.isneginf(l[empty]).all() and (host(o)[empty] == 0).all()
        e = np.abs(l[~empty] - wl[~empty])
        assert (e <= (e_s + 2.0 ** -19 + 2.0 ** -22 * np.abs(wl))[~empty]).all(), (label, e.max())


ATTNS = [  # H, Hkv, d, page, lens
    (1, 1, 64, 16, [1]),
    (2, 2, 64, 16, [257]),
    (4, 4, 128, 128, [130, 0, 1, 15, 16, 17]),
    (8, 2, 128, 16, [0, 0, 0]),
    (32, 8, 128, 16, [0, 1, 31, 33, 500, 64, 1000]),
    (8, 1, 64, 32, [700, 3, 0, 2049]),
    (9, 1, 128, 64, [333, 1, 4097]),           # just more than 8 heads to a key head
    (16, 1, 64, 16, [100, 0, 900]),
    (32, 2, 128, 32, [2500, 7]),
    (24, 1, 128, 128, [1, 900]),               # two tiles of query heads
    (40, 1, 64, 64, [513]),                    # three
    (24, 24, 128, 64, [4609]),
    (6, 2, 64, 128, [20000]),                  # one long row over many CTAs
    (2, 1, 128, 16, [5] * 700 + [40]),         # many short ones
]


@pytest.mark.parametrize("wide", [False, True], ids=["narrow", "wide"])
@pytest.mark.parametrize("case", ATTNS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-R{len(c[4])}")
def test_attn_matches_oracle(vx, case, wide):
    """Narrow tables (short histories take a CTA or a cluster per row) and wide ones (rows are
    dealt out by length)."""
    H, Hkv, d, page, lens = case
    R = len(lens)
    kp, vp, table, num = attn_state(R, Hkv, d, page, lens, seed=H * page + d)
    if wide:
        table = np.concatenate([table, np.full((R, 4200 // page + 1), -1)], 1)
    q = torch.randn(R, H, d, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=I32, device="cuda")
    want = to.token_attention(host(q), host(kp), host(vp), table, lens)
    o, lse = vx.paged_attn(q, kp, vp, i32(table), i32(lens), status=status)
    assert flags(vx, status) == 0
    check_attn(o, lse, want, lens, 1 / math.sqrt(d), d)
    o2, none = vx.paged_attn(q, kp, vp, i32(table), i32(lens), want_lse=False)
    assert none is None and torch.equal(o, o2)     # the same from call to call
    o3, l3 = vx.paged_attn(q, kp, vp, i32(table), i32(lens), scale=0.9)
    check_attn(o3, l3, to.token_attention(host(q), host(kp), host(vp), table, lens, 0.9), lens, 0.9, d)


@pytest.mark.parametrize("H,Hkv,d", [(24, 24, 128), (12, 12, 64), (32, 32, 64), (40, 10, 128), (160, 10, 128),
                                     (170, 10, 64)])
@pytest.mark.parametrize("n", [0, 1, 16, 17, 130, 1000, 3001])
def test_attn_of_one_request_by_clusters(vx, H, Hkv, d, n):
    """One request whose key heads (and tiles of query heads) make up a grid of clusters, from no
    token to more than every warp has units; the table is always wide."""
    page = 64
    kp, vp, table, num = attn_state(1, Hkv, d, page, [n], seed=H + n)
    table = np.concatenate([table, np.full((1, 200), -1)], 1)
    q = torch.randn(1, H, d, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=I32, device="cuda")
    want = to.token_attention(host(q), host(kp), host(vp), table, [n])
    o, lse = vx.paged_attn(q, kp, vp, i32(table), i32([n]), status=status)
    assert flags(vx, status) == 0
    check_attn(o, lse, want, [n], 1 / math.sqrt(d), d)
    o2, _ = vx.paged_attn(q, kp, vp, i32(table), i32([n]))
    assert torch.equal(o, o2)
    # as one of two requests the rows are dealt out by length: the same up to rounding
    two = torch.cat([q, q])
    o3, l3 = vx.paged_attn(two, kp, vp, i32(np.repeat(table, 2, 0)), i32([n, n]))
    for r in range(2):
        check_attn(o3[r:r + 1], l3[r:r + 1], want, [n], 1 / math.sqrt(d), d)
    if n == 130:
        t = table.copy()
        t[0, 1] = num
        vx.paged_attn(q, kp, vp, i32(t), i32([n]), status=status)
        assert flags(vx, status) == vx.VELOX_STATUS_BAD_INDEX
        o, lse = vx.paged_attn(q, kp, vp, i32(np.where(table < 0, 0, table)), i32([-3]), status=status)
        assert flags(vx, status) == vx.VELOX_STATUS_BAD_INDEX
        assert (o == 0).all() and torch.isneginf(lse).all()


def test_attn_extreme_scores_and_values(vx):
    """A last key that dwarfs all before it, scores of -inf, an infinite value among the valid."""
    d, page, n = 128, 16, 300
    kp, vp, table, _ = attn_state(1, 1, d, page, [n], seed=5)
    q = torch.ones(1, 4, d, device="cuda").to(torch.bfloat16)
    at = lambda t: (int(table[0, t // page]), 0, t % page)  # noqa: E731
    kp[at(n - 1)] = 60.0           # score 60 * 128 / sqrt(128), far above the rest
    want = to.token_attention(host(q), host(kp), host(vp), table, [n])
    o, lse = vx.paged_attn(q, kp, vp, i32(table), i32([n]))
    check_attn(o, lse, want, [n], 1 / math.sqrt(d), d)
    kp[at(n - 1)] = -float("inf")  # masked by its own score: weight 0
    kp[at(0)] = -float("inf")
    vp[at(7)][5] = float("inf")
    with np.errstate(invalid="ignore"):
        want = to.token_attention(host(q), host(kp), host(vp), table, [n])
    o, lse = vx.paged_attn(q, kp, vp, i32(table), i32([n]))
    assert torch.isposinf(o[:, :, 5]).all()
    fine = [i for i in range(d) if i != 5]
    want = (want[0][..., fine], want[1], want[2][..., fine], np.zeros_like(want[3]) + 200.0)
    check_attn(o[..., fine], lse, want, [n], 1 / math.sqrt(d), d)


def test_attn_all_scores_at_the_lowest_value(vx):
    """Keys of the type's lowest value: equal scores near -3.4e38 / sqrt(d), a plain mean."""
    d, page, n = 64, 16, 50
    kp, vp, table, _ = attn_state(1, 1, d, page, [n], seed=6)
    q = torch.zeros(1, 2, d, device="cuda").to(torch.bfloat16)
    q[..., 0] = 1.0
    kp[..., 0] = torch.finfo(torch.bfloat16).min
    kp[..., 1:] = 0.0
    o, lse = vx.paged_attn(q, kp, vp, i32(table), i32([n]))
    ids = torch.tensor(table[0, :-(-n // page)], device="cuda")
    mean = host(vp[ids, 0].reshape(-1, d)[:n]).mean(0)
    assert np.abs(host(o) - mean).max() <= 2.0 ** -8 * np.abs(mean).max() + 1e-5
    assert torch.isfinite(lse).all()


def test_attn_bad_pages_and_lengths_are_flagged(vx):
    H, Hkv, d, page = 4, 2, 64, 16
    lens = [70, 20, 33]
    kp, vp, table, num = attn_state(3, Hkv, d, page, lens, seed=9, garbage=False)
    q = torch.randn(3, H, d, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=I32, device="cuda")
    for bad, wide in ((num, 0), (-1, 300), (2 ** 31 - 1, 0), (-2 ** 31, 300)):
        t = np.concatenate([table, np.full((3, wide), -1)], 1)
        t[1, 1] = bad
        o, lse = vx.paged_attn(q, kp, vp, i32(t), i32(lens), status=status)
        assert flags(vx, status) == vx.VELOX_STATUS_BAD_INDEX
        t[1, 1] = 0                                   # what it is replaced by
        want = to.token_attention(host(q), host(kp), host(vp), t, lens)
        check_attn(o, lse, want, lens, 0.125, d)
        vx.paged_attn(q, kp, vp, i32(t), i32(lens))   # without a status word
    width = table.shape[1]
    t = np.where(table < 0, 0, table)
    for bad, as_if in ((-5, 0), (width * page + 1, width * page), (2 ** 31 - 1, width * page)):
        o, lse = vx.paged_attn(q, kp, vp, i32(t), i32([bad] + lens[1:]), status=status)
        assert flags(vx, status) == vx.VELOX_STATUS_BAD_INDEX
        now = [as_if] + lens[1:]
        check_attn(o, lse, to.token_attention(host(q), host(kp), host(vp), t, now), now, 0.125, d)


def test_attn_pool_beyond_32_bit_offsets(vx):
    """A pool of 2.2e9 elements a tensor, the pages in use at its end."""
    d, page, Hkv = 128, 128, 2
    num = (2 ** 31 // (page * Hkv * d)) + 3000
    kp, vp = (torch.empty((num, Hkv, page, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    n = 40 * page + 5
    ids = np.arange(num - 41, num)[::-1].copy()
    sel = torch.tensor(ids, device="cuda")
    kp[sel] = torch.randn(41, Hkv, page, d, device="cuda").to(torch.bfloat16)
    slots = i32([int(ids[40]) * page + 4])
    kv = torch.randn(1, Hkv, d, device="cuda").to(torch.bfloat16)
    vp[sel] = torch.randn(41, Hkv, page, d, device="cuda").to(torch.bfloat16)
    vx.paged_append(kv, kv, slots, kp, vp)
    assert torch.equal(kp[int(ids[40]), :, 4], kv[0]) and torch.equal(vp[int(ids[40]), :, 4], kv[0])
    q = torch.randn(1, 4, d, device="cuda").to(torch.bfloat16)
    o, lse = vx.paged_attn(q, kp, vp, i32(ids[None]), i32([n]))
    sub = host(kp[sel]), host(vp[sel])
    want = to.token_attention(host(q), *sub, np.arange(41)[None], [n])
    check_attn(o, lse, want, [n], 1 / math.sqrt(d), d)


def test_outputs_on_inputs_are_refused(vx):
    """What would race on the GPU: an output that shares some elements of an input."""
    R, H, d = 2, 4, 64
    pages = torch.zeros(4, H, 16, d, dtype=torch.bfloat16, device="cuda")
    table, lens = i32(np.zeros((R, 2))), i32([3, 4])
    big = torch.zeros(R + 1, H, d, dtype=torch.bfloat16, device="cuda")
    for out in (big[:R], big[1:]):
        with pytest.raises(ValueError, match="share"):
            vx.paged_attn(big[:R], pages, pages, table, lens, out=out)
    k, v = (torch.zeros(R, H, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for q, out in ((big[:R], big[1:]), (big[:R], k), (big[:R], v), (big[:R].float(), big[:R])):
        if q.dtype == torch.float32:
            continue
        with pytest.raises(ValueError, match="share"):
            vx.paged_append(k, v, i32([0, 1]), pages, pages, q=q, out=out)
    x = torch.zeros(1, 2, 8, d, device="cuda")
    f = torch.tensor(freqs_for((32,)), device="cuda")
    y = torch.zeros(1, 3, 8, d, device="cuda")
    with pytest.raises(ValueError, match="share"):
        vx.rope(y[:, :2], i32(np.arange(8)), f, out=y[:, 1:])
    qkv = torch.randn(1, 8, 4, d, device="cuda").transpose(1, 2)   # heads side by side: allowed
    want = vx.rope(qkv[:, :2], i32(np.arange(8)), f)
    vx.rope(qkv[:, :2], i32(np.arange(8)), f, out=qkv[:, 2:])
    assert torch.equal(qkv[:, 2:], want) and x.sum() == 0


# ---------------------------------------------------------------- together

def test_cache_of_requests_equals_the_block_path(vx):
    """A chunk of 128 tokens and one more token: the pages' attention against the dense
    block attention over the same rotated keys."""
    from geometry_routed_block_b200.paged import PagedCache
    H, d, page, n = 4, 128, 32, 256
    sec = (22, 21, 21)
    f = torch.tensor(freqs_for(sec), device="cuda")
    t = np.arange(n)
    pos = i32(np.stack([t // 64, (t // 8) % 8, t % 8]))
    q, k, v = (torch.randn(1, H, n, d, device="cuda").to(torch.bfloat16) for _ in range(3))
    kw = dict(style="interleaved", sections=sec)
    qr, kr = vx.rope(q, pos, f, **kw), vx.rope(k, pos, f, **kw)
    o_ref, lse_ref = vx.sparse_attn_fwd(qr, kr, v, None, 128)
    c = PagedCache(1, 1, H, d, page, 16, 10, freqs=f, **kw)
    p = c.plan(i32([n]), n)
    rows = lambda x: x[0].transpose(0, 1)  # noqa: E731
    got = c.append(0, p, rows(k), rows(v), q=rows(q), pos=pos)
    assert torch.equal(got, rows(qr))
    at = p.slots.long()
    assert torch.equal(c.k[0][at // page, :, at % page], rows(kr))
    assert torch.equal(c.v[0][at // page, :, at % page], rows(v))
    for i in (0, 100, n - 1):
        o = c.attend(0, got[i:i + 1].contiguous())
        # both are within 2e-2 of the exact result by their own contracts, in practice far nearer
        assert (o[0].float() - o_ref[0, :, i].float()).abs().max() <= 4e-3
    c.check()


def play(cache, vx, steps, seed, R, H, Hkv, d, graph):
    """Several decoding steps with requests that begin and end; returns all outputs and the
    keys and values in order."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda h: torch.randn(R, h, d, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    data = [(rnd(H), rnd(Hkv), rnd(Hkv)) for _ in range(steps)]
    adds = [i32(np.random.default_rng(seed + s).integers(0, 2, R)) for s in range(steps)]
    q, k, v = (torch.empty_like(x) for x in data[0])
    add = torch.empty_like(adds[0])
    plan = cache.new_plan(R)
    qo, o = torch.empty(R, H, d, dtype=torch.bfloat16, device="cuda"), torch.empty(
        R, H, d, dtype=torch.bfloat16, device="cuda")
    back = torch.zeros(R, H, d, dtype=torch.bfloat16, device="cuda")

    def step():
        cache.plan(add, R, out=plan)
        # token i of the plan is request req[i]; padding takes request 0 and is skipped
        r = plan.req.long().clamp(min=0)
        cache.append(0, plan, k[r], v[r], q=q[r], out=qo)
        live = (plan.req >= 0)[:, None, None]
        back.zero_()
        back.index_add_(0, r, torch.where(live, qo, torch.zeros_like(qo)))
        cache.attend(0, back, out=o)

    outs, gr = [], None
    if graph:
        add.zero_()
        q.copy_(data[0][0]), k.copy_(data[0][1]), v.copy_(data[0][2])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()          # no tokens: changes nothing
        torch.cuda.current_stream().wait_stream(s)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
    for i in range(steps):
        q.copy_(data[i][0]), k.copy_(data[i][1]), v.copy_(data[i][2]), add.copy_(adds[i])
        gr.replay() if graph else step()
        outs.append((o.clone(), cache.lens.clone(), plan.pos.clone(), back.clone()))
        if i % 4 == 3:
            done = torch.zeros(R, dtype=I32, device="cuda")
            done[i % R] = 1
            cache.release(done)
    cache.check()
    return data, adds, outs


@pytest.mark.parametrize("graph", [False, True])
def test_decoding_steps_match_oracle(vx, graph):
    from geometry_routed_block_b200.paged import PagedCache
    R, H, Hkv, d, page, steps = 5, 8, 2, 64, 16, 40
    f = torch.tensor(freqs_for((16,)), device="cuda")
    c = PagedCache(1, R, Hkv, d, page, 24, 4, H=H, freqs=f, style="half")
    data, adds, outs = play(c, vx, steps, 11, R, H, Hkv, d, graph)
    hist = [[] for _ in range(R)]
    for i in range(steps):
        o, lens, pos, q_in = outs[i]
        for r in range(R):
            if adds[i][r]:
                kk = to.rope(host(data[i][1][r]), np.full((1, Hkv), len(hist[r])), f.cpu().numpy(), "half", (16,))
                hist[r].append((kk, host(data[i][2][r])))
        assert lens.tolist() == [len(h) for h in hist]
        for r in range(R):
            if not hist[r]:
                assert (o[r] == 0).all()
                continue
            kr = torch.tensor(np.stack([h[0] for h in hist[r]])).to(torch.bfloat16)
            vr = np.stack([h[1] for h in hist[r]])
            want = to.token_attention(host(q_in[r:r + 1]), host(kr).transpose(1, 0, 2)[None],
                                      vr.transpose(1, 0, 2)[None], np.zeros((1, 1), int), [len(hist[r])])
            # the oracle's keys are rounded from fp64, the cache's from fp32: a key element may
            # land on the neighbouring bf16 (2^-7 of it); such flips are rare, and move a
            # score by 2^-7 |q||k| scale at most each: 0.05 covers a few of them
            tol = 2.0 ** -8 * np.abs(want[0]) + 0.05 * want[2]
            assert (np.abs(host(o[r:r + 1]) - want[0]) <= tol).all(), (i, r)
        if i % 4 == 3:
            hist[i % R] = []


def test_two_captured_steps_of_two_caches_and_eager_calls_between(vx):
    """Two graphs, each with its own cache, replayed on two streams at once, equal the
    eager runs."""
    from geometry_routed_block_b200.paged import PagedCache
    R, H, d, page, n = 3, 4, 64, 16, 200
    runs = []
    for seed in (1, 2):
        c = PagedCache(1, R, H, d, page, 64, 20)
        g = torch.Generator(device="cuda").manual_seed(seed)
        p = c.plan(i32([n, 7, 0]), n + 7)
        k, v = (torch.randn(n + 7, H, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        c.append(0, p, k, v)
        q = torch.randn(R, H, d, generator=g, device="cuda").to(torch.bfloat16)
        want = c.attend(0, q)
        out = torch.empty_like(want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            c.attend(0, q, out=out)
        torch.cuda.synchronize()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr, stream=s):
            c.attend(0, q, out=out)
        runs.append((c, q, want, out, s, gr))
    for _ in range(5):
        for c, q, want, out, s, gr in runs:
            with torch.cuda.stream(s):
                out.zero_()
                gr.replay()
        torch.cuda.synchronize()
        for c, q, want, out, s, gr in runs:
            assert torch.equal(out, want)
            assert torch.equal(c.attend(0, q), want)


def test_calls_on_a_given_stream(vx):
    """stream=: the calls run there (after what was queued there) and allocate there."""
    s = torch.cuda.Stream()
    x = torch.randn(1, 4, 64, 64, device="cuda")
    f = torch.tensor(freqs_for((32,)), device="cuda")
    pos = i32(np.arange(64))
    want = vx.rope(x, pos, f)
    y = torch.zeros_like(x)
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        y.copy_(x)
    got = vx.rope(y, pos, f, stream=s)
    s.synchronize()
    assert torch.equal(got, want)


def test_nothing_to_do(vx):
    """No tokens, no requests: empty results, nothing written."""
    f = torch.tensor(freqs_for((32,)), device="cuda")
    e = lambda *s, t=torch.bfloat16: torch.empty(s, dtype=t, device="cuda")  # noqa: E731
    assert vx.rope(e(2, 3, 0, 64), e(1, 0, t=I32), f).shape == (2, 3, 0, 64)
    kp = torch.ones(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda")
    vp = kp.clone()
    q = vx.paged_append(e(0, 2, 64), e(0, 2, 64), e(0, t=I32), kp, vp, q=e(0, 4, 64), pos=e(0, t=I32), freqs=f)
    assert q.shape == (0, 4, 64) and q.dtype == torch.bfloat16
    assert vx.paged_append(e(0, 2, 64), e(0, 2, 64), e(0, t=I32), kp, vp) is None
    o, lse = vx.paged_attn(e(0, 4, 64), kp, vp, e(0, 5, t=I32), e(0, t=I32))
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    assert (kp == 1).all() and (vp == 1).all()
    with pytest.raises(vx.VeloxError):      # a cache without requests is not planned
        vx.paged_plan(e(0, t=I32), e(0, t=I32), e(0, 5, t=I32), i32([0]), i32([1]), 16, 4)


def test_cache_reports_and_recovers(vx):
    from geometry_routed_block_b200.paged import PagedCache
    c = PagedCache(1, 2, 1, 64, 16, 4, 4)
    c.plan(i32([40, 0]), 40)
    c.check()
    c.plan(i32([0, 33]), 40)         # three pages, one is left
    with pytest.raises(vx.VeloxError):
        c.check()
    assert c.lens.tolist() == [40, 0] and c.free_count.item() == 1
    c.check()                        # reported once
    c.release(i32([1, 0]))
    p = c.plan(i32([0, 33]), 40)
    c.check()
    assert c.lens.tolist() == [0, 33] and (p.slots[:33] >= 0).all() and (p.slots[33:] == -1).all()
