"""A paged KV cache of many requests, read by one new token each.

`Rollout` keeps the history of one rollout whose chunks attend in query blocks.
A server of a chunked world model also has requests of different lengths that
gain single tokens (actions, states, captions) or whole chunks of them, begin and
end. `PagedCache` keeps their keys and values in pages of a common pool and orders
the library calls:

- plan(add): pages and slots for the step's new tokens, once per step;
- append(layer, plan, ...): rotary positions, and keys and values into their slots;
- attend(layer, q, plan=plan): the new token of each request against its pages, in the
  plan's rows as append returns them; requests without one are idle and skipped;
- release(done): the pages of finished requests go back.

All state lives on the device and nothing is read back, so a step can be
captured into a CUDA graph and replayed: lengths, table and free list carry on
from replay to replay. What a call on the device cannot do (no page left, a
length out of range) shows in `status`; `check()` reads it. The calls on one cache
follow one another (one stream, or events between streams): they share its state
and one workspace.

Orchestration only: every step runs in libvelox's kernels.
"""
from __future__ import annotations

import torch

from geometry_routed_block_b200 import velox as vx


class PagedCache:
    def __init__(self, layers: int, R: int, Hkv: int, d: int, page: int, num_pages: int,
                 max_pages: int, H: int | None = None, freqs: torch.Tensor | None = None,
                 style: str = "half", sections=None, mscale: float = 1.0, device="cuda"):
        """Room for R requests of up to max_pages pages each out of num_pages of
        `page` tokens, in every layer. H query heads (default Hkv). With freqs
        ([rot/2] float64, see velox.rope) keys and queries get rotary positions
        on their way in."""
        if (num_pages * page >= 2 ** 31) or (max_pages * page >= 2 ** 31):
            raise ValueError("num_pages * page and max_pages * page must stay below 2^31")
        H = Hkv if H is None else H
        i32 = dict(dtype=torch.int32, device=device)
        self.R, self.Hkv, self.H, self.d, self.page = R, Hkv, H, d, page
        self.rope = dict(freqs=freqs, style=style, sections=sections, mscale=mscale)
        pool = lambda: torch.zeros((num_pages, Hkv, page, d), dtype=torch.bfloat16,  # noqa: E731
                                   device=device)
        self.k = [pool() for _ in range(layers)]
        self.v = [pool() for _ in range(layers)]
        self.table = torch.full((R, max_pages), -1, **i32)
        self.lens = torch.zeros(R, **i32)
        self.free_list = torch.arange(num_pages - 1, -1, -1, **i32)
        self.free_count = torch.full((1,), num_pages, **i32)
        self.status = torch.zeros(1, **i32)
        self.ws = vx.paged_attn_workspace(R, H, Hkv, d, device)

    def new_plan(self, n_cap: int) -> vx.PagedPlan:
        """Tensors for a plan of up to n_cap tokens that carries this cache's state on."""
        e = lambda n: torch.empty(n, dtype=torch.int32, device=self.lens.device)  # noqa: E731
        return vx.PagedPlan(e(self.R + 1), e(n_cap), e(n_cap), e(n_cap), self.lens, self.free_count)

    def plan(self, add: torch.Tensor, n_cap: int, out: vx.PagedPlan | None = None) -> vx.PagedPlan:
        """Pages and slots for add [R] int32 new tokens; lengths and free pages move on.
        n_cap bounds the step's tokens; those of request r are cu[r] .. cu[r+1] - 1."""
        out = self.new_plan(n_cap) if out is None else out
        return vx.paged_plan(add, self.lens, self.table, self.free_list, self.free_count, self.page,
                             n_cap, out=out, status=self.status)

    def append(self, layer: int, plan: vx.PagedPlan, k: torch.Tensor, v: torch.Tensor,
               q: torch.Tensor | None = None, pos: torch.Tensor | None = None,
               out: torch.Tensor | None = None) -> torch.Tensor | None:
        """k, v [N,Hkv,d] (and q [N,H,d]) of the plan's tokens into `layer`. Positions are
        the plan's (one axis) unless pos [axes,N] is given. Returns q, rotated."""
        pos = plan.pos if pos is None else pos
        return vx.paged_append(k, v, plan.slots, self.k[layer], self.v[layer], q=q, pos=pos,
                               out=out, status=self.status, **self.rope)

    def attend(self, layer: int, q: torch.Tensor, out: torch.Tensor | None = None,
               plan: vx.PagedPlan | None = None):
        """q bf16 against everything appended so far. With the step's plan, q [N,H,d] has the
        plan's rows (as append returns them), and each request with new tokens attends with
        the last of them; the other rows stay as they were in out (0 without out). Without a
        plan, q [R,H,d] has a row for EVERY request, in their order: append's rows are that
        only in a step in which each request has one new token."""
        return vx.paged_attn(q, self.k[layer], self.v[layer], self.table, self.lens, ws=self.ws,
                             out=out, want_lse=False, status=self.status,
                             cu=None if plan is None else plan.cu)[0]

    def release(self, done: torch.Tensor) -> None:
        """Requests with done [R] int32 != 0 end: their pages are free again."""
        vx.paged_release(done, self.lens, self.table, self.free_list, self.free_count, self.page,
                         lens_out=self.lens, free_count_out=self.free_count, status=self.status)

    def check(self) -> None:
        """Waits for the GPU, calls on all its streams, and raises if one reported something since
        the last check."""
        torch.cuda.synchronize(self.status.device)
        bits = int(self.status.item())
        self.status.zero_()
        if bits & vx.VELOX_STATUS_TIMEOUT:
            raise vx.VeloxError("paged cache", vx.VELOX_ETIMEOUT)
        if bits & vx.VELOX_STATUS_BAD_INDEX:
            raise vx.VeloxError("paged cache", vx.VELOX_EBOUNDS)
        if bits & vx.VELOX_STATUS_NO_SPACE:
            raise vx.VeloxError("paged cache (no page left, or more tokens than the plan has room for)",
                                vx.VELOX_EINVAL)
