"""A mixture-of-experts layer on one GPU, out of the library's operators.

  decode_step   router -> rows sorted by expert (the maps alone) -> 4-bit gate/up
                products with SwiGLU, reading the tokens through the maps -> 4-bit
                down products -> weighted way back.  Nothing is read on the host.
  MoeLayer      the same layer in training, with bf16 experts: router, sort and
                unsort as autograd functions over the library's gradients.

    python examples/moe_layer.py
"""
from __future__ import annotations

import os
import sys
import time
from dataclasses import dataclass

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from combine_moedc_layout_gb300 import moedc  # noqa: E402

FLAGS = moedc.GATE_SOFTMAX | moedc.GATE_NORMALIZE


# ------------------------------------------------------------------ serving


@dataclass
class Int4Experts:
    """E experts: gate and up rows [E, 2I, H/2], down rows [E, H, I/2], with scales."""
    gate_up: torch.Tensor
    gate_up_scales: torch.Tensor
    down: torch.Tensor
    down_scales: torch.Tensor


def quantize_int4(w: torch.Tensor, group: int):
    """Symmetric 4-bit weights of w [..., N, K]: (uint8 [..., N, K/2], scales [..., N, K/group])."""
    g = w.float().reshape(*w.shape[:-1], -1, group)
    s = (g.abs().amax(-1) / 7.0).clamp(min=1e-8).to(torch.bfloat16)
    q = (g / s.float()[..., None]).round().clamp(-8, 7).to(torch.int32) + 8
    q = q.reshape(*w.shape[:-1], -1, 2)
    return (q[..., 0] | q[..., 1] << 4).to(torch.uint8).contiguous(), s.contiguous()


def decode_step(x: torch.Tensor, logits: torch.Tensor, experts: Int4Experts, K: int,
                status: torch.Tensor) -> torch.Tensor:
    """y [T, H] of the tokens x [T, H] with the router's logits [T, E]."""
    E = logits.shape[1]
    idx, w = moedc.gate(logits, K, flags=FLAGS)
    m = moedc.sort(None, idx, E, status=status)          # maps alone: the products gather
    h = moedc.matvec_int4(x, experts.gate_up, experts.gate_up_scales, offsets=m.offsets,
                          counts=m.counts, src=m.src, top_k=K, swiglu=True, status=status)
    out = moedc.matvec_int4(h, experts.down, experts.down_scales, offsets=m.offsets,
                            counts=m.counts, status=status)
    return moedc.unsort(out, m.row, w)


# ----------------------------------------------------------------- training


class Gate(torch.autograd.Function):
    """(topk_idx, topk_weights) of logits."""

    @staticmethod
    def forward(ctx, logits, K):
        idx, w = moedc.gate(logits, K, flags=FLAGS)
        ctx.save_for_backward(logits, idx)
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    def backward(ctx, _, dw):
        logits, idx = ctx.saved_tensors
        return moedc.gate_grad(logits, idx, dw.contiguous(), flags=FLAGS), None


class Sort(torch.autograd.Function):
    """Packed rows of x, with the maps m of moedc.sort(None, ...)."""

    @staticmethod
    def forward(ctx, x, idx, E, align):
        m = moedc.sort(x, idx, E, align=align)
        ctx.save_for_backward(m.row)
        ctx.mark_non_differentiable(m.row, m.src, m.offsets, m.counts)
        return m.rows, m.row, m.src, m.offsets, m.counts

    @staticmethod
    def backward(ctx, drows, *_):
        return moedc.sort_grad(drows.contiguous(), ctx.saved_tensors[0]), None, None, None


class Unsort(torch.autograd.Function):
    """y of the experts' packed rows and the weights."""

    @staticmethod
    def forward(ctx, rows, w, row, src):
        ctx.save_for_backward(rows, w, row, src)
        return moedc.unsort(rows, row, w)

    @staticmethod
    def backward(ctx, dy):
        rows, w, row, src = ctx.saved_tensors
        drows, dw = moedc.unsort_grad(dy.contiguous(), rows, row, src, w)
        return drows, dw, None, None


class MoeLayer(torch.nn.Module):
    """E SwiGLU experts of width I over H channels, K to a token."""

    def __init__(self, H: int, I: int, E: int, K: int, align: int = 16,
                 dtype: torch.dtype = torch.bfloat16, device: str = "cuda"):
        super().__init__()
        self.K, self.E, self.align = K, E, align

        def init(*shape):
            return torch.nn.Parameter(torch.randn(*shape, device=device, dtype=dtype)
                                      * shape[-1] ** -0.5)

        self.router = init(E, H)
        self.gate_up = init(E, 2 * I, H)
        self.down = init(E, H, I)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        idx, w = Gate.apply((x @ self.router.T).float(), self.K)
        rows, row, src, offsets, _ = Sort.apply(x, idx, self.E, self.align)
        # the experts' products, group by group: the group sizes are the one thing read on
        # the host (a grouped GEMM takes `offsets` on the device instead)
        out, edges = [], offsets.tolist()
        for e in range(self.E):
            a, b = (rows[edges[e]:edges[e + 1]] @ self.gate_up[e].T).chunk(2, dim=1)
            out.append((torch.nn.functional.silu(a) * b) @ self.down[e].T)
        tail = rows.shape[0] - edges[-1]
        out.append(rows.new_zeros(tail, rows.shape[1]))
        return Unsort.apply(torch.cat(out), w, row, src)


def main() -> None:
    torch.manual_seed(0)
    H, I, E, K = 2048, 1024, 32, 4
    x = torch.randn(16, H, device="cuda", dtype=torch.bfloat16)
    logits = torch.randn(16, E, device="cuda")
    up = torch.randn(E, 2 * I, H, device="cuda") * H ** -0.5
    down = torch.randn(E, H, I, device="cuda") * I ** -0.5
    experts = Int4Experts(*quantize_int4(up, 128), *quantize_int4(down, 128))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def timed(name, run, n=200):
        for _ in range(20):
            run()
        torch.cuda.synchronize()
        t = time.perf_counter()
        for _ in range(n):
            run()
        torch.cuda.synchronize()
        print(f"decode step, 16 tokens, {E} experts of {H} x {I}, {name}: "
              f"{(time.perf_counter() - t) / n * 1e6:.1f} us")

    timed("call by call", lambda: decode_step(x, logits, experts, K, status))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = decode_step(x, logits, experts, K, status)
    timed("as a CUDA graph", graph.replay)
    assert int(status) == 0 and torch.isfinite(y).all()

    layer = MoeLayer(512, 256, 8, 2)
    opt = torch.optim.SGD(layer.parameters(), lr=0.05)
    data = torch.randn(256, 512, device="cuda", dtype=torch.bfloat16)
    target = torch.randn(256, 512, device="cuda", dtype=torch.bfloat16)
    for step in range(20):
        loss = torch.nn.functional.mse_loss(layer(data).float(), target.float())
        opt.zero_grad()
        loss.backward()
        opt.step()
        if step % 5 == 0 or step == 19:
            print(f"training step {step}: loss {loss.item():.4f}")


if __name__ == "__main__":
    main()
