"""Outputs of the token calls that share elements with what other threads still read or
write: refused before anything is launched. What is documented as allowed goes through."""
import numpy as np
import pytest
import torch

from tests.test_token_ops_gpu import freqs_for, i32, plan_state, vx  # noqa: F401

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def cache_state(R=4, page=16, width=6):
    table, free, num = plan_state([3, 20, 0, 31], page, width, 12, 1)
    return i32([3, 20, 0, 31]), i32(table), i32(free + [0] * (num - len(free))), i32([len(free)]), num


def plan_outputs(vx, R, n_cap, **over):  # noqa: F811
    e = lambda n: torch.empty(n, dtype=torch.int32, device="cuda")  # noqa: E731
    out = dict(cu=e(R + 1), slots=e(n_cap), pos=e(n_cap), req=e(n_cap), lens=e(R), free_count=e(1))
    out.update(over)
    return vx.PagedPlan(**out)


def test_plan_refuses_shared_outputs(vx):  # noqa: F811
    R, page, n_cap = 4, 16, 8
    lens, table, fl, fc, num = cache_state()
    add = i32([1, 2, 0, 3])
    room = torch.zeros(64, dtype=torch.int32, device="cuda")
    lens_room, status = torch.zeros(R + 1, dtype=torch.int32, device="cuda"), i32([0])
    lens_room[:R] = lens
    bad = [  # what is put where
        (lens_room[:R], dict(lens=lens_room[1:])),          # one element further
        (lens_room[1:], dict(lens=lens_room[:R])),
        (lens, dict(free_count=lens[1:2])), (lens, dict(free_count=add[:1])),
        (lens, dict(lens=table.view(-1)[:R])), (lens, dict(lens=fl[:R])),
        (lens, dict(slots=room[:n_cap], pos=room[n_cap - 1:2 * n_cap - 1])),
        (lens, dict(req=room[:n_cap], cu=room[n_cap - 1:n_cap + R])),
        (lens, dict(slots=table.view(-1)[2:2 + n_cap])), (lens, dict(free_count=status)),
        (lens, dict(cu=room[:R + 1], lens=room[R:2 * R])),
    ]
    for src, over in bad:
        with pytest.raises(ValueError, match="share"):
            vx.paged_plan(add, src, table, fl, fc, page, n_cap, out=plan_outputs(vx, R, n_cap, **over),
                          status=status)
    # neighbours, the state itself, and outputs of no elements
    want = vx.paged_plan(add, lens, table, fl, fc, page, n_cap, status=status)
    side = dict(slots=room[:n_cap], pos=room[n_cap:2 * n_cap], req=room[2 * n_cap:3 * n_cap],
                cu=room[3 * n_cap:3 * n_cap + R + 1], lens=lens_room[:R], free_count=lens_room[R:])
    got = vx.paged_plan(add, lens, table, fl, fc, page, n_cap, out=plan_outputs(vx, R, n_cap, **side))
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    vx.paged_plan(i32([0] * R), lens, table, fl, fc, page, 0, out=plan_outputs(vx, R, 0))
    vx.paged_plan(add, lens, table, fl, fc, page, n_cap,
                  out=plan_outputs(vx, R, n_cap, lens=lens, free_count=fc), status=status)
    assert torch.equal(lens, want.lens) and torch.equal(fc, want.free_count) and status.item() == 0


@pytest.mark.parametrize("R,n_cap", [(4, 80), (300, 5000), (2000, 30000)])
def test_the_new_lengths_may_be_the_added_ones(vx, R, n_cap):  # noqa: F811
    """Lengths doubled (add is lens is lens_out), written over add, and all that have tokens given back
    (done is lens): one CTA, a cluster, and a grid with a second kernel."""
    page, width = 16, 3
    old = np.random.default_rng(R).integers(0, 12, R)
    table, free, num = plan_state(old.tolist(), page, width, R, 1)
    for over_add in (False, True):
        lens, tab, fc = i32(old), i32(table), i32([len(free)])
        fl, status = i32(free + [0] * (num - len(free))), i32([0])
        add = lens.clone() if over_add else lens
        want = vx.paged_plan(i32(old), i32(old), i32(table), fl, i32([len(free)]), page, n_cap)
        out = plan_outputs(vx, R, n_cap, lens=add, free_count=fc)
        vx.paged_plan(add, lens, tab, fl, fc, page, n_cap, out=out, status=status)
        for a, b in zip(out, want):
            assert torch.equal(a, b)
        now = add       # done, lens and lens_out at once
        vx.paged_release(now, now, tab, fl, fc, page, lens_out=now, free_count_out=fc, status=status)
        assert (now == 0).all() and fc.item() == num and status.item() == 0
        assert sorted(fl.tolist()) == list(range(num))


def test_release_refuses_shared_outputs(vx):  # noqa: F811
    R, page = 4, 16
    lens, table, fl, fc, num = cache_state()
    done, before = i32([1, 0, 0, 1]), fl.clone()
    lens_room = torch.zeros(R + 1, dtype=torch.int32, device="cuda")
    lens_room[:R] = lens
    for src, kw in ((lens_room[:R], dict(lens_out=lens_room[1:])), (lens_room[1:], dict(lens_out=lens_room[:R])),
                    (lens, dict(lens_out=fl[:R])),
                    (lens, dict(free_count_out=lens[:1])), (lens, dict(free_count_out=fl[-1:])),
                    (lens, dict(lens_out=table.view(-1)[:R])),
                    (lens, dict(lens_out=lens_room[:R], free_count_out=lens_room[1:2]))):
        with pytest.raises(ValueError, match="share"):
            vx.paged_release(done, src, table, fl, fc, page, **kw)
    assert torch.equal(fl, before)
    lo, _ = vx.paged_release(done, lens, table, fl, fc, page, lens_out=lens)
    assert lo is lens and lens.tolist() == [0, 20, 0, 0]


@pytest.mark.parametrize("dtype", [BF, torch.float32])
def test_append_refuses_tensors_in_the_pages(vx, dtype):  # noqa: F811
    N, H, d, page, num = 4, 2, 64, 16, 8
    z = lambda *s, t=dtype: torch.zeros(s, dtype=t, device="cuda")  # noqa: E731
    pool = z(2 * num + 1, H, page, d, t=BF)
    kp, vp = pool[:num], pool[num:2 * num]
    k, v, slots = z(N, H, d), z(N, H, d), i32(np.arange(N))
    inside = kp.view(dtype).view(-1)        # the pages' memory as the inputs' type
    strided = lambda t: t.as_strided((N, H, d), (H * d + 8, d, 1))  # noqa: E731
    before = pool.clone()
    for a, b in ((kp, kp), (kp, pool[1:num + 1]), (pool[1:num + 1], kp)):
        with pytest.raises(ValueError, match="share"):
            vx.paged_append(k, v, slots, a, b)
    dense = inside[64:64 + N * H * d].view(N, H, d)
    for kk, vv, q in ((dense, v, None), (k, dense, None), (k, v, dense), (strided(inside), v, None)):
        with pytest.raises(ValueError, match="share"):
            vx.paged_append(kk, vv, slots, kp, vp, q=q)
    for out in (vp.reshape(-1)[:N * H * d].view(N, H, d), kp.reshape(-1)[-N * H * d:].view(N, H, d)):
        with pytest.raises(ValueError, match="share"):
            vx.paged_append(k, v, slots, kp, vp, q=z(N, H, d), out=out)
    # an output on its own queries' memory in another type
    q = z(N, H, d)
    half = q.view(BF).view(-1)[:N * H * d].view(N, H, d)
    if dtype == torch.float32:
        with pytest.raises(ValueError, match="share"):
            vx.paged_append(k, v, slots, kp, vp, q=q, out=half)
    assert torch.equal(pool, before)
    # side by side with the pages, and between them
    room = z(3 * num, H, page, d, t=BF)
    kp, vp = room[:num], room[2 * num:]
    mid = room[num:2 * num].view(dtype).view(-1)
    mid.copy_(torch.randn(mid.shape, device="cuda"))
    k, v, q = (mid[i * N * H * d:(i + 1) * N * H * d].view(N, H, d) for i in range(3))
    o = vx.paged_append(k, v, slots, kp, vp, q=q)
    assert torch.equal(o, q.to(BF)) and torch.equal(kp[0, :, :N].transpose(0, 1), k.to(BF))
    assert torch.equal(vp[0, :, :N].transpose(0, 1), v.to(BF))


def test_attention_refuses_outputs_in_its_inputs(vx):  # noqa: F811
    R, H, d = 2, 4, 64
    kp, vp = (torch.randn(4, H, 16, d, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(R, H, d, device="cuda").to(BF)
    args = (q, kp, vp, i32(np.zeros((R, 2))), i32([3, 4]))
    for pages in (kp, vp):
        flat = pages.view(-1)
        for out in (flat[:R * H * d], flat[-R * H * d:]):
            with pytest.raises(ValueError, match="share"):
                vx.paged_attn(*args, out=out.view(R, H, d))
        with pytest.raises(ValueError, match="share"):
            vx.paged_attn(*args, lse=pages.view(torch.float32).view(-1)[:R * H].view(R, H))
    out = torch.empty_like(q)
    for t in (q, out):
        with pytest.raises(ValueError, match="share"):
            vx.paged_attn(*args, out=out, lse=t.view(torch.float32).view(-1)[:R * H].view(R, H))
    want, _ = vx.paged_attn(*args)
    assert torch.equal(vx.paged_attn(*args, out=out, lse=torch.empty(R, H, device="cuda"))[0], want)
    vx.paged_attn(q, kp, kp, *args[3:])      # pages that are only read may be the same


def test_rope_refuses_an_output_on_itself(vx):  # noqa: F811
    """Rows of an output that lie on one another: which of them stays would depend on timing."""
    f = torch.tensor(freqs_for((32,)), device="cuda")
    x, pos = torch.randn(1, 3, 8, 64, device="cuda"), i32(np.arange(8))
    room = torch.zeros(4096, device="cuda")
    for strides in ((1536, 512, 32, 1), (1536, 256, 64, 1), (1536, 500, 64, 1)):
        with pytest.raises(ValueError, match="itself"):
            vx.rope(x, pos, f, out=room.as_strided(x.shape, strides))
    for strides in ((0, 512, 64, 1), (1536, 64, 192, 1), (1536, 600, 70, 1)):
        out = room.as_strided(x.shape, strides)
        assert torch.equal(vx.rope(x, pos, f, out=out), vx.rope(x, pos, f))


def test_status_words_have_an_element(vx):  # noqa: F811
    """An empty status tensor has no address: what a call reports would be lost."""
    lens, table = [20, 0, 7], i32(np.zeros((3, 4)))
    kp, vp = (torch.zeros(4, 2, 32, 128, dtype=BF, device="cuda") for _ in range(2))
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    q, k = torch.zeros(3, 8, 128, device="cuda").to(BF), torch.zeros(3, 2, 128, device="cuda").to(BF)
    z = i32([0, 0, 0])
    for call in (lambda: vx.paged_attn(q, kp, vp, table, i32(lens), status=none),
                 lambda: vx.paged_append(k, k, z, kp, vp, status=none),
                 lambda: vx.paged_plan(z, z, table, z, i32([0]), 32, 4, status=none),
                 lambda: vx.paged_release(z, z, table, z, i32([0]), 32, status=none)):
        with pytest.raises(ValueError, match="status"):
            call()
