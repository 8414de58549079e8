"""Planned steps with idle requests, through the public calls alone: append's rows go to the
attention as they are. Tolerances are those of test_token_ops_gpu.py."""
import math

import numpy as np
import pytest
import torch

from oracle import token_oracle as to
from tests.test_token_ops_gpu import (attn_state, check_attn, flags, freqs_for, host, i32,
                                      rope_tolerance, vx)  # noqa: F401

pytestmark = pytest.mark.gpu
I32 = torch.int32

STEPS = [  # H, Hkv, d, page, lens, new tokens (0: idle), rows behind the last token
    (4, 2, 64, 16, [40, 17], [0, 1], 1),
    (8, 2, 128, 16, [300, 1, 55, 200], [0, 1, 0, 1], 2),
    (8, 2, 128, 16, [300, 1, 55, 200], [1, 0, 3, 0], 0),
    (2, 2, 64, 32, [5], [5], 3),
    (24, 24, 128, 64, [700], [1], 0),
    (16, 1, 64, 16, [100, 5, 900], [0, 2, 1], 1),
    (40, 1, 128, 128, [513, 90], [1, 0], 0),
    (4, 4, 64, 16, [9, 8, 7], [0, 0, 0], 4),
    (2, 1, 128, 16, [30] * 700 + [5000], [i % 3 for i in range(701)], 5),
]


@pytest.mark.parametrize("wide", [False, True], ids=["narrow", "wide"])
@pytest.mark.parametrize("case", STEPS, ids=lambda c: f"{c[0]}-{c[1]}-{c[2]}-{c[3]}-R{len(c[4])}-{sum(c[5])}")
def test_rows_of_a_step_match_oracle(vx, case, wide):  # noqa: F811
    H, Hkv, d, page, lens, add, pad = case
    R, N = len(lens), sum(add) + pad
    kp, vp, table, _ = attn_state(R, Hkv, d, page, lens, seed=H + d + R)
    table = np.concatenate([table, np.full((R, 6000 // page if wide else 0), -1)], 1)
    cu = np.concatenate([[0], np.cumsum(add)])
    rows, live = cu[1:] - 1, np.asarray(add) > 0
    # what an idle request has is not looked at: a length and a table that cannot be
    lens_d, table_d = np.where(live, lens, 2 ** 31 - 1), np.where(live[:, None], table, 10 ** 9)
    q = torch.randn(N, H, d, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=I32, device="cuda")
    out = torch.full((N, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((N, H), 7.0, device="cuda")
    args = (q, kp, vp, i32(table_d), i32(lens_d))
    got = vx.paged_attn(*args, out=out, lse=lse, status=status, cu=i32(cu))
    assert got[0] is out and got[1] is lse and flags(vx, status) == 0
    at = torch.tensor(rows[live], device="cuda")
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[at] = False
    assert (out[rest] == 7).all() and (lse[rest] == 7).all()    # rows of no request: as they were
    if live.any():
        n = np.asarray(lens)[live].tolist()
        want = to.token_attention(host(q[at]), host(kp), host(vp), table[live], n)
        check_attn(out[at], lse[at], want, n, 1 / math.sqrt(d), d)
        # the same work as a call with a row for every request, idle ones of length 0
        by_request = torch.zeros(R, H, d, dtype=torch.bfloat16, device="cuda")
        by_request[torch.tensor(live, device="cuda")] = q[at]
        o2, l2 = vx.paged_attn(by_request, kp, vp, i32(table), i32(np.where(live, lens, 0)))
        mine = torch.tensor(live, device="cuda")
        assert torch.equal(o2[mine], out[at]) and torch.equal(l2[mine], lse[at])
    o3, l3 = vx.paged_attn(*args, cu=i32(cu))
    assert torch.equal(o3[at], out[at]) and (o3[rest] == 0).all() and torch.isneginf(l3[rest]).all()


def test_a_row_without_history_gets_zeros(vx):  # noqa: F811
    kp, vp, table, _ = attn_state(3, 2, 64, 16, [20, 0, 5], seed=1)
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    for wider in (0, 400):
        t = i32(np.concatenate([table, np.full((3, wider), -1)], 1))
        out = torch.full_like(q, 7.0)
        _, lse = vx.paged_attn(q, kp, vp, t, i32([20, 0, 5]), out=out, cu=i32([0, 0, 1, 2]))
        assert (out[0] == 0).all() and torch.isneginf(lse[0]).all() and torch.isfinite(lse[1]).all()


@pytest.mark.parametrize("wider", [0, 400])
@pytest.mark.parametrize("cu,bad", [([0, 1, 2, 3], 2), ([0, 1, 2, 2 ** 31 - 1], 2), ([-1, 1, 2, 2], 0),
                                    ([0, 1, 0, 1], 1), ([-2 ** 31, 1, 2, 2], 0)])
def test_rows_outside_the_step_are_flagged(vx, cu, bad, wider):  # noqa: F811
    H, d, lens = 4, 64, [50, 33, 20]
    kp, vp, table, _ = attn_state(3, 2, d, 16, lens, seed=2)
    table = np.concatenate([table, np.full((3, wider), -1)], 1)
    q = torch.randn(2, H, d, device="cuda").to(torch.bfloat16)
    status = torch.zeros(1, dtype=I32, device="cuda")
    room = torch.full((4, H, d), 7.0, dtype=torch.bfloat16, device="cuda")
    vx.paged_attn(q, kp, vp, i32(table), i32(lens), out=room[1:3], status=status, cu=i32(cu))
    assert flags(vx, status) == vx.VELOX_STATUS_BAD_INDEX
    assert (room[0] == 7).all() and (room[3] == 7).all()
    ends = [cu[r + 1] for r in range(3) if r != bad and cu[r + 1] > cu[r]]
    for r in range(3):      # the other requests have their rows
        # (cu = 0 1 0 1 gives row 0 to requests 0 and 2: one row cannot hold two results)
        if r != bad and cu[r + 1] > cu[r] and ends.count(cu[r + 1]) == 1:
            want = to.token_attention(host(q[cu[r + 1] - 1:cu[r + 1]]), host(kp), host(vp),
                                      table[r:r + 1], lens[r:r + 1])
            check_attn(room[1 + cu[r + 1] - 1:1 + cu[r + 1]], None, want, lens[r:r + 1], 0.125, d)


@pytest.mark.parametrize("style", ["half", "interleaved"])
@pytest.mark.parametrize("graph", [False, True])
def test_plan_append_attend_with_idle_requests(vx, graph, style):  # noqa: F811
    """The documented sequence: requests idle, gain one token or several, end; eager and captured."""
    from geometry_routed_block_b200.paged import PagedCache
    R, H, Hkv, d, page, steps, layers, n_cap = 5, 8, 2, 64, 16, 24, 2, 12
    f = freqs_for((16,))
    c = PagedCache(layers, R, Hkv, d, page, 40, 8, H=H, freqs=torch.tensor(f, device="cuda"), style=style,
                   mscale=1.2)
    g = torch.Generator(device="cuda").manual_seed(7)
    rnd = lambda h: torch.randn(n_cap, h, d, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    add, plan = torch.zeros(R, dtype=I32, device="cuda"), c.new_plan(n_cap)
    q, k, v = rnd(H), rnd(Hkv), rnd(Hkv)
    qo, o = torch.empty_like(q), [torch.empty_like(q) for _ in range(layers)]

    def step():
        c.plan(add, n_cap, out=plan)
        for layer in range(layers):
            c.append(layer, plan, k, v, q, out=qo)
            c.attend(layer, qo, out=o[layer], plan=plan)

    if graph:
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            step()          # no tokens: changes nothing
        torch.cuda.current_stream().wait_stream(s)
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            step()
    rng = np.random.default_rng(3)
    lens = np.zeros(R, int)
    seen = set()
    for i in range(steps):
        new = rng.choice([0, 0, 1, 1, 2], R)
        add.copy_(i32(new))
        for x, h in ((q, H), (k, Hkv), (v, Hkv)):
            x.copy_(rnd(h))
        for x in o:
            x.fill_(7.0)
        gr.replay() if graph else step()
        old, lens = lens.copy(), lens + new
        assert c.lens.tolist() == lens.tolist()
        total = int(new.sum())
        pos, slots, table = plan.pos.cpu().numpy(), plan.slots.long(), c.table.cpu().numpy()
        assert pos[:total].tolist() == [t for r in range(R) for t in range(old[r], lens[r])]
        turn = lambda x: to.rope(host(x), pos[None, :total, None], f, style, (16,), 1.2)  # noqa: E731
        for x, got in ((q, qo[:total]), (k, c.k[0][slots[:total] // page, :, slots[:total] % page])):
            want = turn(x[:total])
            assert (np.abs(host(got) - want) <= rope_tolerance(host(x[:total]), want, 1.2, 32, style, True)).all()
        live, at = new > 0, np.cumsum(new) - 1
        rest = np.setdiff1d(np.arange(n_cap), at[live])
        for layer in range(layers):
            assert (o[layer][rest.tolist()] == 7).all()
            if live.any():
                sel = at[live].tolist()
                want = to.token_attention(host(qo[sel]), host(c.k[layer]), host(c.v[layer]), table[live],
                                          lens[live])
                check_attn(o[layer][sel], None, want, lens[live], 1 / math.sqrt(d), d)
        seen |= set(new.tolist())
        if i % 5 == 4:
            c.release(i32(np.arange(R) == i % R))
            lens[i % R] = 0
    c.check()
    assert seen == {0, 1, 2}
