"""A block that routes rows to experts, with adapters beside its shared projection.

    h   = ReLU(x W + scale_i (x A_i^T) B_i)          one adapter i per row
    u_e = ReLU(h_rows-of-e up_e),  y_e = u_e down_e   top-k experts e per row
    y   = sum of its experts' y_e, weighted by the router

Serving runs ``forward``; ``backward`` gives the gradients of the experts'
weights and of h for a training step.  The products are the library's; the
routing (top-k, sort, gather, weighted sum) is plain torch on the same stream,
and no step reads a size back to the host.

    python examples/expert_block.py [--rows 4096] [--steps 10]
"""
from __future__ import annotations

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import tiled_dense_gemm_gb300 as fw  # noqa: E402


class ExpertBlock:
    """Weights of one block: a shared projection (d, d) with R adapters of the
    given rank, a router over E experts, and the experts' two products."""

    def __init__(self, d: int, hidden: int, experts: int, top_k: int, adapters: int, rank: int,
                 dtype=torch.bfloat16, device="cuda", seed: int = 0):
        gen = torch.Generator(device=device).manual_seed(seed)

        def normal(*shape, scale):
            return (torch.randn(shape, generator=gen, device=device) * scale).to(dtype)

        self.experts, self.top_k = experts, top_k
        self.w = normal(d, d, scale=d ** -0.5)
        self.a, self.b = normal(adapters, rank, d, scale=d ** -0.5), normal(adapters, rank, d, scale=rank ** -0.5)
        self.scale = torch.rand(adapters, generator=gen, device=device) + 0.5
        self.router = normal(d, experts, scale=d ** -0.5)
        self.up = normal(experts, d, hidden, scale=d ** -0.5)
        self.down = normal(experts, hidden, d, scale=hidden ** -0.5)

    def route(self, h):
        """The rows' experts: their order by expert, the experts' offsets, and
        the weight of each routed row."""
        weight, expert = torch.softmax(h.float() @ self.router.float(), dim=1).topk(self.top_k, dim=1)
        order = expert.flatten().argsort(stable=True)
        counts = torch.zeros(self.experts, dtype=torch.int32, device=h.device)
        counts.scatter_add_(0, expert.flatten(), torch.ones_like(expert.flatten(), dtype=torch.int32))
        offsets = torch.zeros(self.experts + 1, dtype=torch.int32, device=h.device)
        offsets[1:] = counts.cumsum(0)
        return order // self.top_k, offsets, weight.flatten()[order]

    def forward(self, x, ids):
        """(y, what backward needs)."""
        h = fw.gemm_relu_adapters(x, self.w, self.a, self.b, ids, self.scale)
        row, offsets, weight = self.route(h)
        rows = h[row]
        u = fw.gemm_relu_grouped(rows, self.up, offsets)
        z = fw.gemm_relu_grouped(u, self.down, offsets, apply_relu=False)
        y = torch.zeros(h.shape, dtype=torch.float32, device=h.device).index_add_(0, row, z.float() * weight[:, None])
        return y.to(h.dtype), (row, offsets, weight, rows, u, h.shape)

    def backward(self, dy, kept):
        """Gradients of (h, up, down); the router's weights are taken as given."""
        row, offsets, weight, rows, u, shape = kept
        dz = (dy[row].float() * weight[:, None]).to(dy.dtype)
        d_down = fw.gemm_relu_grouped_dw(u, dz, offsets)
        du = fw.gemm_relu_grouped_dx(dz, self.down, offsets, act=u)  # before up's ReLU
        d_up = fw.gemm_relu_grouped_dw(rows, du, offsets)
        d_rows = fw.gemm_relu_grouped_dx(du, self.up, offsets)
        dh = torch.zeros(shape, dtype=torch.float32, device=dy.device).index_add_(0, row, d_rows.float())
        return dh.to(dy.dtype), d_up, d_down


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--rows", type=int, default=4096)
    p.add_argument("--steps", type=int, default=10)
    p.add_argument("--width", type=int, default=2048)
    p.add_argument("--hidden", type=int, default=4096)
    p.add_argument("--experts", type=int, default=32)
    p.add_argument("--top-k", type=int, default=2)
    p.add_argument("--adapters", type=int, default=16)
    p.add_argument("--rank", type=int, default=16)
    a = p.parse_args()
    block = ExpertBlock(a.width, a.hidden, a.experts, a.top_k, a.adapters, a.rank)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(a.rows, a.width, generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn(a.rows, a.width, generator=gen, device="cuda").to(torch.bfloat16)
    ids = torch.randint(-1, a.adapters, (a.rows,), generator=gen, device="cuda", dtype=torch.int32)
    for name, step in (("forward", lambda: block.forward(x, ids)),
                       ("forward + backward", lambda: block.backward(dy, block.forward(x, ids)[1]))):
        for _ in range(3):
            step()
        begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        begin.record()
        for _ in range(a.steps):
            step()
        end.record()
        torch.cuda.synchronize()
        print(f"{name}: {begin.elapsed_time(end) / a.steps * 1e3:.0f} us for {a.rows} rows")
    fw.check_device_error()


if __name__ == "__main__":
    main()
