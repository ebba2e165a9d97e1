"""Temporal attention over pooled BEV cells: the token operators together.

Each frame's camera features are pooled into bird's-eye-view cells
(bevpool.pool_frame); the cells are tokens with positions (time, y, x).  A
frame's keys are normed, turned and appended to a paged cache beside its
values, and its queries attend over this and the last frames in the cache
(every cell sees every cell).  When the cache is full the oldest frame's pages
are handed to the new one.  `train_step` fits the norms' weights on a frame:
the forward and backward of the norm and rotation.

`PlannedAttention` does the same for several vehicles at once: their frames'
pages are planned on the GPU, and their cache holds E4M3 codes with a scale for
each page and key head.

    python examples/temporal_bev.py            # needs the GPU and the built library
"""
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from depth_weighted_scatter_gb300 import attention, bevpool, workloads  # noqa: E402

PAGE = 64


class TemporalAttention:
    """Projections (random here), norms, rotary frequencies and the frames' cache."""

    def __init__(self, C, Y, X, n_heads=8, n_k_heads=4, head_dim=64, frames=4, cache_dtype=torch.float16, seed=0):
        g = torch.Generator().manual_seed(seed)
        cells = Y * X
        assert cells % PAGE == 0, "a frame fills whole pages here"
        self.H, self.Hk, self.D, self.frames, self.cells = n_heads, n_k_heads, head_dim, frames, cells
        self.project = (torch.randn(C, (n_heads + 2 * n_k_heads) * head_dim, generator=g) / C ** 0.5).half().cuda()
        self.q_weight, self.k_weight = torch.ones(head_dim, device="cuda"), torch.ones(head_dim, device="cuda")
        pairs = head_dim // 2
        self.sections = [pairs // 4, (pairs - pairs // 4) // 2, pairs - pairs // 4 - (pairs - pairs // 4) // 2]
        self.inv_freq = torch.pow(10000.0, -torch.arange(pairs, dtype=torch.float64) / pairs).float().cuda()
        at = torch.arange(cells)
        self.yx = torch.stack([at // X, at % X], dim=1).to(torch.int32).cuda()
        self.pages = cells // PAGE
        shape = (frames * self.pages, n_k_heads, PAGE, head_dim)
        self.k_cache, self.v_cache = torch.zeros(shape, device="cuda").to(cache_dtype), torch.zeros(shape, device="cuda").to(cache_dtype)
        # E4M3 codes stand for code * scale
        self.scales = dict(k_scale=1 / 32.0, v_scale=1 / 32.0) if cache_dtype == torch.float8_e4m3fn else {}
        self.order = []                    # frames' page groups, the newest last
        self.cu_q = torch.tensor([0, cells], dtype=torch.int32, device="cuda")
        self.t = 0

    def qkv(self, bev):
        """[cells, C] -> q, k, v as slices of one projection's output."""
        x = (bev @ self.project).view(self.cells, self.H + 2 * self.Hk, self.D)
        return x[:, :self.H], x[:, self.H:self.H + self.Hk], x[:, self.H + self.Hk:]

    def positions(self):
        return torch.cat([torch.full_like(self.yx[:, :1], self.t), self.yx], dim=1)

    def step(self, bev):
        """One frame: its cells into the cache, and their attention over the frames kept.  -> [cells, heads, head_dim]"""
        q, k, v = self.qkv(bev)
        group = len(self.order) if len(self.order) < self.frames else self.order.pop(0)
        self.order.append(group)
        table = torch.cat([torch.arange(g * self.pages, (g + 1) * self.pages, dtype=torch.int32) for g in self.order])[None].cuda()
        n = len(self.order) * self.cells
        kv_len = torch.tensor([n], dtype=torch.int32, device="cuda")
        q = attention.kv_append(k, v, self.k_cache, self.v_cache, table, kv_len, self.cu_q, self.positions(), self.inv_freq,
                                sections=self.sections, q=q, q_weight=self.q_weight, k_weight=self.k_weight, **self.scales)
        self.t += 1
        return attention.paged_attention(q, self.k_cache, self.v_cache, table, kv_len, self.cu_q, max_q_len=self.cells,
                                         max_kv_len=n, causal=False, **self.scales)

    def train_step(self, bev, target_q, target_k, lr=1e-2):
        """One step of the norms' weights towards given queries and keys; returns the loss (mean squared error)."""
        q, k, _ = self.qkv(bev)
        rot = dict(sections=self.sections, q_weight=self.q_weight, k_weight=self.k_weight)
        yq, yk = attention.qk_norm_rope(q, k, self.positions(), self.inv_freq, **rot)
        eq, ek = yq.float() - target_q.float(), yk.float() - target_k.float()
        _, _, gq, gk = attention.qk_norm_rope_backward(eq.to(q.dtype), ek.to(q.dtype), q, k, self.positions(), self.inv_freq,
                                                       **rot)
        self.q_weight -= lr * gq / (self.cells * self.H)
        self.k_weight -= lr * gk / (self.cells * self.Hk)
        return float(eq.square().mean() + ek.square().mean())


class PlannedAttention(TemporalAttention):
    """A batch of vehicles, each with its own frames, over one pool of pages."""

    def __init__(self, C, Y, X, vehicles, frames=4, **more):
        super().__init__(C, Y, X, frames=frames, cache_dtype=torch.float8_e4m3fn, **more)
        i32 = dict(dtype=torch.int32, device="cuda")
        pool, width = (vehicles * (frames + 1)) * self.pages, (frames + 1) * self.pages
        shape = (pool, self.Hk, PAGE, self.D)
        self.k_cache, self.v_cache = (torch.zeros(shape, device="cuda").to(torch.float8_e4m3fn) for _ in range(2))
        self.k_scales, self.v_scales = (torch.ones(pool, self.Hk, device="cuda") for _ in range(2))
        # lengths, positions of the first tokens kept, tables and free pages: all on the GPU, from one plan to the next
        self.state = [torch.zeros(vehicles, **i32), torch.zeros(vehicles, **i32), torch.full((vehicles, width), -1, **i32),
                      torch.arange(pool, **i32), torch.tensor([pool], **i32)]
        self.vehicles = vehicles

    def step(self, bevs, drive):
        """A frame of the vehicles that drive (a truth value each; bevs: their cells, one after the other).
        -> [cells of those that drive, heads, head_dim]"""
        if len(bevs) != sum(map(bool, drive)) * self.cells:
            raise ValueError(f"{len(bevs)} cells for {sum(map(bool, drive))} vehicles of {self.cells}")
        q, k, v = (bevs @ self.project).view(-1, self.H + 2 * self.Hk, self.D).split([self.H, self.Hk, self.Hk], dim=1)
        on = torch.tensor([bool(x) for x in drive], dtype=torch.int32, device="cuda")
        # a vehicle whose cache is full gives its oldest frame's pages back first
        drop = on * (self.state[0] >= self.frames * self.cells).to(torch.int32) * self.pages
        plan = attention.plan_pages(on * self.cells, *self.state, page_size=PAGE, n_tokens=len(bevs), drop=drop)
        # a plan that does not fit changes nothing and names no tokens: nothing would be attended
        missing = plan.missing.item()
        if missing:
            raise RuntimeError(f"{missing} pages too few for this frame" if missing > 0 else "a vehicle's frames do not fit its pages")
        self.state = [plan.kv_len, plan.first, plan.block_table, plan.free_pages, plan.n_free]
        # token i of a vehicle is cell i % cells of frame i // cells
        at = plan.positions
        positions = torch.stack([at // self.cells, self.yx[at % self.cells, 0], self.yx[at % self.cells, 1]], dim=1).to(torch.int32)
        pages = (self.k_cache, self.v_cache, self.k_scales, self.v_scales, plan.block_table, plan.kv_len, plan.cu_q)
        q = attention.kv_append_scaled(k, v, *pages, positions, self.inv_freq, sections=self.sections, q=q, q_weight=self.q_weight,
                                       k_weight=self.k_weight)
        return attention.paged_attention_scaled(q, *pages, max_q_len=self.cells, max_kv_len=self.frames * self.cells, causal=False)


def pooled_frame(seed, C=64, Y=32, X=40):
    """BEV cells [Y * X, C] (fp16) of one synthetic frame."""
    NC, D, H, W = 2, 10, 8, 16
    cells = np.random.default_rng(seed).integers(-1, Y * X, NC * D * H * W).astype(np.int32)
    wl = workloads.custom(NC, D, H, W, C, Y * X, cells, seed=seed, name=f"frame_{seed}")
    up = lambda a, view: torch.from_numpy(np.ascontiguousarray(a).reshape(-1).view(view).copy()).cuda()  # noqa: E731
    out, _ = bevpool.pool_frame(up(wl.cell_ids, np.int32), up(wl.depth, np.uint16), up(wl.feat, np.uint16), *wl.dims(),
                                wl.n_cells, wl.C)
    return out


def main():
    model = TemporalAttention(64, 32, 40)
    for t in range(6):
        bev = pooled_frame(t)
        y = model.step(bev)
        print(f"frame {t}: {len(model.order)} frames in the cache, output {tuple(y.shape)}, "
              f"mean magnitude {y.float().abs().mean().item():.4f}")
    fleet = PlannedAttention(64, 32, 40, vehicles=3)
    for t in range(6):
        drive = [True, t % 2 == 0, t > 2]
        y = fleet.step(torch.cat([pooled_frame(10 * i + t) for i, on in enumerate(drive) if on]), drive)
        print(f"fleet, frame {t}: {[n // fleet.cells for n in fleet.state[0].tolist()]} frames in the cache, output {tuple(y.shape)}")
    bev = pooled_frame(0)
    q, k, _ = model.qkv(bev)
    target = attention.qk_norm_rope(q, k, model.positions(), model.inv_freq, sections=model.sections,
                                    q_weight=2 * model.q_weight, k_weight=0.5 * model.k_weight)
    for i in range(5):
        print(f"training step {i}: loss {model.train_step(bev, *target, lr=0.5):.5f}")


if __name__ == "__main__":
    main()
