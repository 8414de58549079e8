"""What is measured of the token operators: rotary positions, the paged KV
cache (block tables and slot maps, append, release) and the attention of one new
token over it.

Each case names its operator in "op":
  rope     rotary positions of x [B,H,N,d] (1 to 3 position axes, both layouts, part
           of the head, backwards)
  plan     pages for the new tokens of R requests: block table, slot map, positions
  release  the pages of finished requests go back to the free list
  append   q, k rotated; k, v written to their slots of the paged cache
  attn     one new token per request against its pages

`run` computes the plain form with elementary torch operations, or with `own`
the calls of this package.
"""
import math
import random

import numpy as np
import torch

own = False

DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ cases

def listed():
    return [
        # a single state token of the small fp32 setup, far into a rollout, rotated back
        # (the direction of the gradient): latency
        dict(name="rope token f32 back", op="rope", B=1, H=2, N=1, d=64, rot=32, style="half",
             sec="16", dtype="f32", far=1000003, mscale=1.1, inverse=True),
        # the queries of one 4608-token chunk (3 frames x 32 x 48) with frame, row and
        # column positions
        dict(name="rope chunk", op="rope", B=1, H=24, N=4608, d=128, rot=128, style="interleaved",
             sec="22,21,21", dtype="bf16", far=0, mscale=1.0, inverse=False),
        # one decoding step of a small batch of rollouts, some of them idle: latency
        dict(name="plan step", op="plan", R=48, page=16, lo=0, hi=8000, add_lo=0, add_hi=1, pad=16,
             lseed=1),
        # many requests arrive at once, up to a chunk each
        dict(name="plan arrivals", op="plan", R=301, page=64, lo=0, hi=20000, add_lo=1, add_hi=4608,
             pad=1000, lseed=2),
        # half of a large batch ends
        dict(name="release half", op="release", R=1000, page=16, lo=1, hi=9000, lseed=3),
        # one decoding step of a batch, four query heads to a key head
        dict(name="append step", op="append", N=48, H=32, Hkv=8, d=128, rot=128, style="half",
             sec="64", dtype="bf16", page=16, heads_first=False, pad=5),
        # a whole chunk of the headline setup goes into the pages, in the layout
        # [H][N][d] that the block-sparse attention takes
        dict(name="append chunk", op="append", N=4608, H=24, Hkv=24, d=128, rot=128,
             style="interleaved", sec="22,21,21", dtype="bf16", page=64, heads_first=True, pad=0),
        # an odd number of fp32 tokens of the small setup, a quarter of the head rotated
        dict(name="append odd f32", op="append", N=301, H=2, Hkv=2, d=64, rot=16, style="half",
             sec="8", dtype="f32", page=32, heads_first=False, pad=3),
        # one token of the small setup against a short, ragged history: latency
        dict(name="attn short", op="attn", R=1, H=2, Hkv=2, d=64, page=16, lo=257, hi=257, lseed=4),
        # a batch of requests of all lengths (an empty and a one-token one among them)
        dict(name="attn ragged", op="attn", R=64, H=32, Hkv=8, d=128, page=16, lo=0, hi=16384, lseed=5),
        # sixteen query heads share a key head, medium lengths
        dict(name="attn shared heads", op="attn", R=16, H=32, Hkv=2, d=128, page=32, lo=512, hi=32768,
             lseed=6),
        # one token against the whole history of chunk 48, 24 heads
        dict(name="attn history", op="attn", R=1, H=24, Hkv=24, d=128, page=128, lo=225793, hi=225793,
             lseed=7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _rotary(rng, d):
    """rot and its sections: the whole head or a part, one axis or three."""
    rot = rng.choice([d, d, d // 2, d // 4])
    if rng.random() < 0.5 or rot < 32:
        return rot, str(rot // 2)
    s = rot // 6
    return rot, "%d,%d,%d" % (rot // 2 - 2 * s, s, s)


def draw(rng):
    op = rng.choice(["rope", "plan", "release", "append", "attn", "attn"])
    if op == "rope":
        d = rng.choice([64, 128])
        rot, sec = _rotary(rng, d)
        B, H, N = rng.choice([1, 1, 2]), rng.randint(1, 24), _log(rng, 1, 2300)
        return dict(op=op, B=B, H=H, N=N, d=d, rot=rot, style=rng.choice(["half", "interleaved"]),
                    sec=sec, dtype=rng.choice(["bf16", "f32"]), far=rng.choice([0, _log(rng, 1000, 2000000)]),
                    mscale=rng.choice([1.0, 1.25]), inverse=rng.random() < 0.3)
    if op == "plan":
        hi = rng.choice([1, 1, _log(rng, 2, 4608)])
        return dict(op=op, R=_log(rng, 1, 300), page=rng.choice([16, 32, 64, 128]), lo=0,
                    hi=_log(rng, 100, 20000), add_lo=0, add_hi=hi, pad=rng.randint(0, 500),
                    lseed=rng.randint(0, 10**6))
    if op == "release":
        return dict(op=op, R=_log(rng, 1, 1000), page=rng.choice([16, 32, 64, 128]), lo=0,
                    hi=_log(rng, 100, 9000), lseed=rng.randint(0, 10**6))
    if op == "append":
        d = rng.choice([64, 128])
        rot, sec = _rotary(rng, d)
        Hkv = rng.choice([1, 2, 4, 6, 8])
        return dict(op=op, N=_log(rng, 1, 4608), H=Hkv * rng.choice([1, 2, 3]), Hkv=Hkv, d=d, rot=rot,
                    style=rng.choice(["half", "interleaved"]), sec=sec, dtype=rng.choice(["bf16", "f32"]),
                    page=rng.choice([16, 32, 64, 128]), heads_first=rng.random() < 0.4,
                    pad=rng.randint(0, 9))
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8, 12, 24])
    G = rng.choice([1, 1, 2, 3, 4, 5, 8, 12, 16])
    R = _log(rng, 1, 96)
    hi = _log(rng, 16, max(32, min(200000, 60000000 // (R * Hkv * d))))
    return dict(op=op, R=R, H=Hkv * G, Hkv=Hkv, d=d, page=rng.choice([16, 32, 64, 128]),
                lo=rng.choice([0, max(1, hi // 4)]), hi=hi, lseed=rng.randint(0, 10**6))


def _lengths(case, lo, hi, salt=0):
    """Lengths of the requests: over their logarithm, the case's extremes among them."""
    rng = random.Random(case["lseed"] * 7 + salt)
    n = [_log(rng, max(lo, 1), max(hi, 1)) for _ in range(case["R"])]
    if case["R"] >= 4:
        n[0], n[1], n[2] = lo, max(lo, 1), hi
        rng.shuffle(n)
    return n


def _added(case):
    if case["add_hi"] == 1:
        rng = random.Random(case["lseed"])
        return [1 if rng.random() < 0.9 else case["add_lo"] for _ in range(case["R"])]
    return _lengths(case, case["add_lo"], case["add_hi"], salt=1)


def _pages(n, page):
    return -(-n // page)


def work(case):
    op, e = case["op"], 4 if case.get("dtype") == "f32" else 2
    if op == "rope":
        n = case["B"] * case["H"] * case["N"]
        return {"bytes": 2 * n * case["d"] * e + 4 * case["N"] * len(case["sec"].split(",")),
                "flops": 3 * n * case["rot"]}
    if op == "plan":
        old, add = _lengths(case, case["lo"], case["hi"]), _added(case)
        new = sum(_pages(a + b, case["page"]) - _pages(a, case["page"]) for a, b in zip(old, add))
        # lengths in and out, offsets, new pages read and entered, three words for each token
        return {"bytes": 4 * (4 * case["R"] + 2 * new + 3 * (sum(add) + case["pad"])), "flops": 0}
    if op == "release":
        done = _done(case)
        gone = sum(_pages(n, case["page"]) for n, x in zip(_lengths(case, case["lo"], case["hi"]), done) if x)
        return {"bytes": 4 * (3 * case["R"] + 2 * gone), "flops": 0}
    if op == "append":
        n = case["N"] - case["pad"] if case["N"] > case["pad"] else case["N"]
        return {"bytes": n * case["d"] * (case["H"] + 2 * case["Hkv"]) * (e + 2) + 8 * case["N"],
                "flops": 3 * n * case["rot"] * (case["H"] + case["Hkv"])}
    t = sum(_lengths(case, case["lo"], case["hi"]))
    return {"bytes": 4 * t * case["Hkv"] * case["d"] + case["R"] * case["H"] * (4 * case["d"] + 4)
            + 4 * sum(_pages(n, case["page"]) for n in _lengths(case, case["lo"], case["hi"])),
            "flops": 4 * t * case["H"] * case["d"]}


def _done(case):
    rng = random.Random(case["lseed"] + 11)
    return [1 if rng.random() < 0.5 else 0 for _ in range(case["R"])]


# ------------------------------------------------------------------ inputs

def _frequencies(sec):
    """Radians per position of each rotated pair: every axis has the powers of its own size."""
    return torch.cat([10000.0 ** (-torch.arange(s, dtype=torch.float64) / s) for s in sec]).to(DEV)


def _positions(N, axes, far, g):
    """[axes][N]: one running position, or frame, row and column of a 32 x 48 grid."""
    t = torch.arange(N, device=DEV)
    if axes == 1:
        start = int(torch.randint(0, 1000, (1,), generator=g, device=DEV)) + far
        return (t + start).to(torch.int32)[None].contiguous()
    return torch.stack([t // 1536 + far, (t // 48) % 32, t % 48])[:axes].to(torch.int32).contiguous()


def _table(lens, page, num_pages, extra, g):
    """A block table over a shuffled pool, -1 behind each request's pages; the pages left."""
    used = torch.tensor([_pages(n, page) for n in lens], device=DEV)
    width = max(1, int(used.max()) + extra)
    perm = torch.randperm(num_pages, generator=g, device=DEV).to(torch.int32)
    at = torch.arange(width, device=DEV)[None]
    first = (used.cumsum(0) - used)[:, None]
    table = torch.where(at < used[:, None], perm[(first + at).clamp(max=num_pages - 1)],
                        torch.full_like(perm[:1], -1))
    return table.contiguous(), perm[int(used.sum()):].contiguous()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device=DEV)  # noqa: E731
    op = case["op"]
    st = dict(case)
    if op in ("rope", "append"):
        sec = tuple(int(s) for s in case["sec"].split(","))
        dt = F32 if case["dtype"] == "f32" else BF
        st["sec"], st["freqs"] = sec, _frequencies(sec)
        st["axis"] = torch.repeat_interleave(torch.arange(len(sec)), torch.tensor(sec)).to(DEV)
        st["pos"] = _positions(case["N"], len(sec), case.get("far", 0), g)
    if op == "rope":
        st["x"] = rnd(case["B"], case["H"], case["N"], case["d"]).to(dt)
    elif op == "append":
        N, page, d = case["N"], case["page"], case["d"]
        if case["heads_first"]:
            q, k, v = (rnd(h, N, d).to(dt).transpose(0, 1) for h in (case["H"], case["Hkv"], case["Hkv"]))
        else:  # slices of one projection's output
            qkv = rnd(N, case["H"] + 2 * case["Hkv"], d).to(dt)
            q, k, v = qkv.split([case["H"], case["Hkv"], case["Hkv"]], dim=1)
        num_pages = _pages(N, page) + 3
        # tokens lie in order in shuffled pages, from inside the first page on
        perm = torch.randperm(num_pages, generator=g, device=DEV)
        t = torch.arange(N, device=DEV) + page // 2
        slots = (perm[t // page] * page + t % page).to(torch.int32)
        if N > case["pad"] > 0:
            slots[N - case["pad"]:] = -1
        st.update(q=q, k=k, v=v, slots=slots,
                  kp=rnd(num_pages, case["Hkv"], page, d).to(BF), vp=rnd(num_pages, case["Hkv"], page, d).to(BF))
    elif op == "plan":
        old, add = _lengths(case, case["lo"], case["hi"]), _added(case)
        both = [a + b for a, b in zip(old, add)]
        pages = sum(_pages(n, case["page"]) for n in both)
        most = max(_pages(n, case["page"]) for n in both)
        extra = most - max(_pages(n, case["page"]) for n in old) + 2
        table, left = _table(old, case["page"], pages + 7, extra, g)
        st.update(lens=torch.tensor(old, dtype=torch.int32, device=DEV),
                  add=torch.tensor(add, dtype=torch.int32, device=DEV), table=table,
                  free_count=torch.tensor([left.numel()], dtype=torch.int32, device=DEV),
                  free_list=torch.cat([left, left.new_zeros(pages + 7 - left.numel())]),
                  n_cap=sum(add) + case["pad"] + 1)
    elif op == "release":
        lens = _lengths(case, case["lo"], case["hi"])
        pages = sum(_pages(n, case["page"]) for n in lens) + 7
        table, left = _table(lens, case["page"], pages, 1, g)
        st.update(lens=torch.tensor(lens, dtype=torch.int32, device=DEV), table=table,
                  done=torch.tensor(_done(case), dtype=torch.int32, device=DEV),
                  free_count=torch.tensor([left.numel()], dtype=torch.int32, device=DEV),
                  free_list=torch.cat([left, left.new_zeros(pages - left.numel())]))
    else:
        lens = _lengths(case, case["lo"], case["hi"])
        num_pages = sum(_pages(n, case["page"]) for n in lens) + 5
        shape = (num_pages, case["Hkv"], case["page"], case["d"])
        table, _ = _table(lens, case["page"], num_pages, 1, g)
        # keys with an offset of each head, as the chunks of the synthetic rollouts have them
        off = 0.5 * rnd(case["Hkv"], 1, case["d"])
        st.update(q=rnd(case["R"], case["H"], case["d"]).to(BF), table=table,
                  kp=(rnd(*shape) + off).to(BF), vp=rnd(*shape).to(BF),
                  lens=torch.tensor(lens, dtype=torch.int32, device=DEV))
    return st


# ------------------------------------------------------------------ plain forms

def _angles(s):
    """cos and sin [N][rot/2] (positions [axes][N]), angles in 64 bits."""
    t = s["pos"][s["axis"]].double().T * s["freqs"]
    return t.cos(), t.sin()


def _rotate(x, cos, sin, style, rot):
    """x [..., d] in 32 bits; cos, sin broadcast over its leading dimensions."""
    if style == "half":
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    return torch.cat([y, x[..., rot:]], dim=-1)


def _plain_rope(s):
    cos, sin = _angles(s)
    m = s["mscale"]
    cos, sin = (cos * m).float(), ((-sin if s["inverse"] else sin) * m).float()
    return _rotate(s["x"].float(), cos, sin, s["style"], s["rot"]).to(s["x"].dtype)


def _plain_append(s):
    cos, sin = (t.float()[:, None] for t in _angles(s))
    q = _rotate(s["q"].float(), cos, sin, s["style"], s["rot"]).to(BF)
    k = _rotate(s["k"].float(), cos, sin, s["style"], s["rot"]).to(BF)
    v = s["v"].float().to(BF)
    page, keep = s["page"], s["slots"] >= 0
    # padding writes the row back that the first token's slot gets anyway
    at = torch.where(keep, s["slots"], s["slots"][:1]).long()
    k, v = torch.where(keep[:, None, None], k, k[:1]), torch.where(keep[:, None, None], v, v[:1])
    s["kp"][at // page, :, at % page] = k
    s["vp"][at // page, :, at % page] = v
    return q, s["kp"], s["vp"]


def _plain_plan(s):
    lens, add, page, table = s["lens"].long(), s["add"].long(), s["page"], s["table"]
    cu = torch.cat([add.new_zeros(1), add.cumsum(0)])
    old, new = (lens + page - 1) // page, (lens + add + page - 1) // page
    first = (new - old).cumsum(0) - (new - old)
    at = torch.arange(table.shape[1], device=DEV)[None]
    fresh = (at >= old[:, None]) & (at < new[:, None])
    take = s["free_count"].long() - 1 - (first[:, None] + at - old[:, None])
    table.copy_(torch.where(fresh, s["free_list"][take.clamp(0, s["free_list"].numel() - 1)], table))
    t = torch.arange(s["n_cap"], device=DEV)
    req = torch.searchsorted(cu[1:], t, right=True)
    real = req < lens.numel()
    r = req.clamp(max=lens.numel() - 1)
    pos = lens[r] + t - cu[r]
    slot = table[r, (pos // page).clamp(0, table.shape[1] - 1)].long() * page + pos % page
    i32 = lambda x: torch.where(real, x, torch.full_like(x, -1)).to(torch.int32)  # noqa: E731
    return (cu.to(torch.int32), i32(slot), i32(pos), i32(req), (lens + add).to(torch.int32), table,
            (s["free_count"].long() - (new - old).sum()).to(torch.int32))


def _plain_release(s):
    lens, page, done = s["lens"].long(), s["page"], s["done"] != 0
    n = torch.where(done, (lens + page - 1) // page, torch.zeros_like(lens))
    at = torch.arange(s["table"].shape[1], device=DEV)[None]
    gone = at < n[:, None]
    size = s["free_list"].numel()
    to = s["free_count"].long() + (n.cumsum(0) - n)[:, None] + at
    # what does not move goes to one place behind the list
    more = torch.cat([s["free_list"], s["free_list"][:1]])
    more[torch.where(gone, to, torch.full_like(to, size)).flatten()] = s["table"].flatten()
    s["free_list"].copy_(more[:size])
    return (torch.where(done, torch.zeros_like(lens), lens).to(torch.int32), s["free_list"],
            (s["free_count"].long() + n.sum()).to(torch.int32))


def _plain_attn(s):
    R, H, d = s["q"].shape
    Hkv, page = s["Hkv"], s["page"]
    k = s["kp"][s["table"].clamp(min=0)].float().transpose(2, 3).reshape(R, -1, Hkv, d)
    v = s["vp"][s["table"].clamp(min=0)].float().transpose(2, 3).reshape(R, -1, Hkv, d)
    q = s["q"].float().reshape(R, Hkv, H // Hkv, d)
    ok = torch.arange(k.shape[1], device=DEV)[None] < s["lens"][:, None]
    sc = torch.matmul(q, k.permute(0, 2, 3, 1)) * (1.0 / math.sqrt(d))
    sc = sc.masked_fill(~ok[:, None, None], -math.inf)
    top = sc.amax(-1, keepdim=True)
    p = torch.exp(sc - torch.where(top == -math.inf, torch.zeros_like(top), top))
    den = p.sum(-1, keepdim=True)
    v = torch.where(ok[:, :, None, None], v, torch.zeros_like(v))
    o = torch.matmul(p, v.transpose(1, 2)) / torch.where(den == 0, torch.ones_like(den), den)
    return o.reshape(R, H, d).to(BF), (top + den.log()).reshape(R, H)


# ------------------------------------------------------------------ one pass

def run(state):
    s = state
    if own:
        from geometry_routed_block_b200 import velox as vx
        if s["op"] == "rope":
            return vx.rope(s["x"], s["pos"], s["freqs"], style=s["style"], sections=s["sec"],
                           mscale=s["mscale"], inverse=s["inverse"])
        if s["op"] == "append":
            q = vx.paged_append(s["k"], s["v"], s["slots"], s["kp"], s["vp"], q=s["q"], pos=s["pos"],
                                freqs=s["freqs"], style=s["style"], sections=s["sec"])
            return q, s["kp"], s["vp"]
        if s["op"] == "plan":
            p = vx.paged_plan(s["add"], s["lens"], s["table"], s["free_list"], s["free_count"], s["page"],
                              s["n_cap"])
            return p.cu, p.slots, p.pos, p.req, p.lens, s["table"], p.free_count
        if s["op"] == "release":
            lens, count = vx.paged_release(s["done"], s["lens"], s["table"], s["free_list"],
                                           s["free_count"], s["page"])
            return lens, s["free_list"], count
        return vx.paged_attn(s["q"], s["kp"], s["vp"], s["table"], s["lens"])
    return {"rope": _plain_rope, "append": _plain_append, "plan": _plain_plan,
            "release": _plain_release, "attn": _plain_attn}[s["op"]](s)


# ------------------------------------------------------------------ from the definitions

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rope", "append"):
        # the rotation of each pair as the product with a unit complex number
        t = s["pos"].double()[s["axis"]].T * s["freqs"]

        def turn(x, back, m):  # x [..., N, d]
            x = x.double()
            rot = s["rot"]
            i = torch.arange(rot // 2, device=DEV)
            re, im = (i, i + rot // 2) if s["style"] == "half" else (2 * i, 2 * i + 1)
            z = torch.complex(x[..., re], x[..., im]) * torch.polar(torch.full_like(t, m), -t if back else t)
            y = x.clone()
            y[..., re], y[..., im] = z.real, z.imag
            return y

        if op == "rope":
            return turn(s["x"], s["inverse"], s["mscale"])
        q, k = (turn(s[n].transpose(0, 1), False, 1.0).transpose(0, 1) for n in ("q", "k"))
        kp, vp = s["kp"].double(), s["vp"].double()
        for i, a in enumerate(s["slots"].tolist()):
            if a >= 0:
                kp[a // s["page"], :, a % s["page"]] = k[i]
                vp[a // s["page"], :, a % s["page"]] = s["v"][i].double()
        return q.contiguous(), kp, vp
    if op in ("plan", "release"):
        # the requests one after the other, pages from and to the end of the list
        page, lens = s["page"], s["lens"].tolist()
        table = s["table"].cpu().numpy().copy()
        stack = s["free_list"].tolist()
        n = int(s["free_count"])
        if op == "release":
            for r, x in enumerate(s["done"].tolist()):
                if x:
                    for i in range(_pages(lens[r], page)):
                        stack[n] = int(table[r, i])
                        n += 1
                    lens[r] = 0
            return np.array(lens, np.int32), np.array(stack, np.int32), np.array([n], np.int32)
        cu, slots, pos, req = [0], [], [], []
        for r, a in enumerate(s["add"].tolist()):
            for i in range(_pages(lens[r], page), _pages(lens[r] + a, page)):
                n -= 1
                table[r, i] = stack[n]
            at = np.arange(lens[r], lens[r] + a)
            slots.append(table[r, at // page].astype(np.int64) * page + at % page)
            pos.append(at)
            req.append(np.full(a, r))
            cu.append(cu[-1] + a)
            lens[r] += a
        fill = [np.full(s["n_cap"] - cu[-1], -1)]
        whole = lambda p: np.concatenate(p + fill).astype(np.int32)  # noqa: E731
        return (np.array(cu, np.int32), whole(slots), whole(pos), whole(req), np.array(lens, np.int32), table,
                np.array([n], np.int32))
    R, H, d = s["q"].shape
    G = H // s["Hkv"]
    o = torch.zeros(R, H, d, dtype=torch.float64, device=DEV)
    lse = torch.full((R, H), -math.inf, dtype=torch.float64, device=DEV)
    for r, n in enumerate(s["lens"].tolist()):
        if n == 0:
            continue
        own_pages = s["table"][r, :_pages(n, s["page"])].long()
        for h in range(s["Hkv"]):
            k = s["kp"][own_pages, h].reshape(-1, d)[:n].double()
            v = s["vp"][own_pages, h].reshape(-1, d)[:n].double()
            x = s["q"][r, h * G:(h + 1) * G].double() @ k.T / math.sqrt(d)
            lse[r, h * G:(h + 1) * G] = torch.logsumexp(x, -1)
            o[r, h * G:(h + 1) * G] = torch.softmax(x, -1) @ v
    return o, lse
