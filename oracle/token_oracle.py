"""fp64 CPU oracle of the token path: rotary positions, the paged KV cache and
the attention of one new token over it. Plain numpy, one request and one pair
at a time where that keeps it plain; shares no code with the CUDA path."""
from __future__ import annotations

import math

import numpy as np


def rope(x, pos, freqs, style, sections, mscale=1.0, inverse=False):
    """x [...,N,d] float64, pos [axes,N] or [axes,...,N] broadcastable to x's leading
    dimensions, freqs [rot/2]."""
    y = np.array(x, np.float64)
    half = len(freqs)
    axis = np.repeat(np.arange(len(sections)), sections)
    for i in range(half):
        a, b = (i, i + half) if style == "half" else (2 * i, 2 * i + 1)
        t = np.asarray(pos[axis[i]], np.float64) * freqs[i]
        c, s = mscale * np.cos(t), mscale * np.sin(t) * (-1.0 if inverse else 1.0)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
    return y


def freqs(rot, base=10000.0, scaling="plain", factor=1.0, orig_len=0, beta_fast=32.0, beta_slow=1.0):
    if scaling == "base":
        base = base * factor ** (rot / (rot - 2))
    f = np.array([base ** (-2.0 * i / rot) for i in range(rot // 2)])
    if scaling == "linear":
        return f / factor, 1.0
    if scaling != "bands":
        return f, 1.0
    turns = lambda n: rot * math.log(orig_len / (n * 2 * math.pi)) / (2 * math.log(base))  # noqa: E731
    lo = min(max(math.floor(turns(beta_fast)), 0), rot - 1)
    hi = min(max(math.ceil(turns(beta_slow)), 0), rot - 1)
    i = np.arange(rot // 2)
    mix = np.clip((i - lo) / (hi - lo), 0, 1) if hi > lo else (i > lo).astype(float)
    return f * (1 - mix) + f / factor * mix, 0.1 * math.log(factor) + 1.0


def _pages(n, page):
    return -(-int(n) // page)


def plan(add, lens, table, stack, page, n_cap):
    """stack: list of free pages. Returns (cu, slots, pos, req, lens, table, stack) or
    None when the step does not fit."""
    R = len(lens)
    lens, table, stack = list(lens), np.array(table), list(stack)
    if sum(add) > n_cap:
        return None
    cu, slots, pos, req = [0], [], [], []
    for r in range(R):
        have, want = _pages(lens[r], page), _pages(lens[r] + add[r], page)
        if want > table.shape[1] or want - have > len(stack):
            return None
        for i in range(have, want):
            table[r, i] = stack.pop()
        for t in range(int(lens[r]), int(lens[r] + add[r])):
            slots.append(int(table[r, t // page]) * page + t % page)
            pos.append(t)
            req.append(r)
        lens[r] += add[r]
        cu.append(cu[-1] + int(add[r]))
    pad = [-1] * (n_cap - len(slots))
    return cu, slots + pad, pos + pad, req + pad, lens, table, stack


def release(done, lens, table, stack, page):
    lens, stack = list(lens), list(stack)
    for r in range(len(lens)):
        if done[r]:
            stack += [int(table[r, i]) for i in range(_pages(lens[r], page))]
            lens[r] = 0
    return lens, stack


def token_attention(q, k_pages, v_pages, table, lens, scale=None):
    """q [R,H,d], pages [num_pages,Hkv,page,d] float64 -> (o [R,H,d], lse [R,H], and for
    error bounds: |p||v| summed [R,H,d], the largest scale * sum |q||k| of a key
    [R,H])."""
    R, H, d = q.shape
    _, Hkv, page, _ = k_pages.shape
    G = H // Hkv
    scale = 1.0 / math.sqrt(d) if scale is None else scale
    o, lse = np.zeros((R, H, d)), np.full((R, H), -np.inf)
    pv, qk = np.zeros((R, H, d)), np.zeros((R, H))
    for r in range(R):
        n = int(lens[r])
        if n == 0:
            continue
        ids = np.asarray(table[r, :_pages(n, page)], np.int64)
        for h in range(Hkv):
            k = k_pages[ids, h].reshape(-1, d)[:n]
            v = v_pages[ids, h].reshape(-1, d)[:n]
            for g in range(h * G, (h + 1) * G):
                s = k @ q[r, g] * scale
                m = s.max()
                e = np.exp(s - m)
                p = e / e.sum()
                o[r, g], lse[r, g] = p @ v, m + np.log(e.sum())
                pv[r, g], qk[r, g] = p @ np.abs(v), (np.abs(k) @ np.abs(q[r, g])).max() * scale
    return o, lse, pv, qk
