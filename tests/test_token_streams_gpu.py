"""Token calls across streams: their launches overlap the end of the kernel before them in the
stream, and still wait for what events say; captured with branches that join again; scores of
which none is left."""
import numpy as np
import pytest
import torch

from tests.test_token_ops_gpu import attn_state, freqs_for, i32, vx  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def problem(n=2000, R=3, H=8, Hkv=2, d=128, page=32):
    lens = [n, 0, 700]
    kp, vp, table, num = attn_state(R, Hkv, d, page, lens, seed=n, spare=4)
    return lens, kp, vp, i32(np.concatenate([table, np.full((R, 300), -1)], 1)), num


def test_calls_wait_for_events_between_them(vx):  # noqa: F811
    """A call on one stream, an event of another, then a call that reads what that stream wrote."""
    lens, kp, vp, table, num = problem()
    H, d, R = 8, 128, 3
    n, f = i32(lens), torch.tensor(freqs_for((64,)), device="cuda")
    x, pos = torch.randn(1, H, 512, d, device="cuda").to(BF), i32(np.arange(512))
    qs = [torch.randn(R, H, d, device="cuda").to(BF) for _ in range(3)]
    xs = [torch.randn_like(x) for _ in range(3)]
    want = [(vx.paged_attn(q, kp, vp, table, n)[0], vx.rope(y, pos, f)) for q, y in zip(qs, xs)]
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    q, y, o = torch.zeros_like(qs[0]), torch.zeros_like(x), torch.empty_like(qs[0])
    z = torch.empty_like(x)
    torch.cuda.synchronize()
    for i in range(3):
        written = torch.cuda.Event()
        with torch.cuda.stream(b):
            torch.cuda._sleep(3_000_000)
            q.copy_(qs[i])
            y.copy_(xs[i])
            written.record()
        with torch.cuda.stream(a):
            vx.rope(x, pos, f, out=z)           # lets the next launch of the stream in early
            a.wait_event(written)
            vx.paged_attn(q, kp, vp, table, n, out=o, want_lse=False)
            got_o = o.clone()
            vx.rope(x, pos, f, out=z)
            a.wait_event(written)
            got_y = vx.rope(y, pos, f)
        torch.cuda.synchronize()
        assert torch.equal(got_o, want[i][0]) and torch.equal(got_y, want[i][1])


def test_captured_branches_that_join(vx):  # noqa: F811
    """Queries and keys come from different branches of a captured step, the output goes to two."""
    lens, kp, vp, table, num = problem()
    H, Hkv, d, page, R = 8, 2, 128, 32, 3
    n, f = i32(lens), torch.tensor(freqs_for((64,)), device="cuda")
    pos, slots = i32(np.arange(R)), i32([(num - 1) * page + i for i in range(R)])
    src_q, src_k = torch.randn(R, H, d, device="cuda").to(BF), torch.randn(R, Hkv, d, device="cuda").to(BF)
    q, k, v = torch.zeros_like(src_q), torch.zeros_like(src_k), torch.zeros_like(src_k)
    qo, o = torch.empty_like(q), torch.empty_like(q)
    left, right = torch.empty_like(q), torch.empty_like(q)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    main, side = torch.cuda.Stream(), torch.cuda.Stream()

    def step():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            torch.mul(src_k, 2, out=k)
            vx.rope(src_k.unsqueeze(2), i32_zero, f, out=v.unsqueeze(2))
        torch.mul(src_q, 0.5, out=q)
        main.wait_stream(side)
        vx.paged_append(k, v, slots, kp, vp, q=q, pos=pos, freqs=f, out=qo, status=status)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            vx.rope(qo.unsqueeze(0).transpose(1, 2), pos, f, out=left.unsqueeze(0).transpose(1, 2))
        vx.paged_attn(qo, kp, vp, table, n, out=o, want_lse=False, status=status)
        torch.mul(o, 2, out=right)
        main.wait_stream(side)

    i32_zero = torch.zeros((1, R, 1), dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr, stream=main):
        step()
    for i in range(4):
        src_q.copy_(torch.randn_like(src_q))
        src_k.copy_(torch.randn_like(src_k))
        for t in (q, k, v, qo, o, left, right):
            t.zero_()
        gr.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in (qo, o, left, right, kp[num - 1, :, :R], vp[num - 1, :, :R])]
        assert status.item() == 0
        want_q = vx.paged_append(src_k * 2, src_k, slots, kp, vp, q=src_q * 0.5, pos=pos, freqs=f)
        want_o, _ = vx.paged_attn(want_q, kp, vp, table, n)
        want = [want_q, want_o, vx.rope(want_q.unsqueeze(0).transpose(1, 2), pos, f)[0].transpose(0, 1),
                want_o * 2, kp[num - 1, :, :R], vp[num - 1, :, :R]]
        for g, w in zip(got, want):
            assert torch.equal(g, w)


@pytest.mark.parametrize("wider", [0, 400])
def test_scores_of_which_none_is_left(vx, wider):  # noqa: F811
    """Keys that score -inf throughout: a softmax of nothing, NaN with lse = -inf, as torch's; the
    other requests and heads are not touched by it."""
    lens, d, page = [300, 40, 33], 64, 16
    kp, vp, table, _ = attn_state(3, 2, d, page, lens, seed=4)
    q = torch.ones(3, 4, d, device="cuda").to(BF)
    ids = torch.tensor(table[1][table[1] >= 0], device="cuda")
    kp[ids, 0] = -float("inf")          # request 1, key head 0
    t = i32(np.concatenate([table, np.full((3, wider), -1)], 1))
    o, lse = vx.paged_attn(q, kp, vp, t, i32(lens))
    assert torch.isnan(o[1, :2]).all() and torch.isneginf(lse[1, :2]).all()
    rest = torch.ones(3, 4, dtype=torch.bool, device="cuda")
    rest[1, :2] = False
    assert torch.isfinite(o[rest]).all() and torch.isfinite(lse[rest]).all()
