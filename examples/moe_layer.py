"""A mixture-of-experts layer on one GPU, out of the library's operators.

  decode_step   router -> rows sorted by expert (the maps alone) -> gate/up products
                with SwiGLU, reading the tokens through the maps -> down products
                -> weighted way back.  4-bit experts, or e4m3 ones with a scale for
                each 128 x 128 block, which take the tokens and the rows between the
                products in e4m3 too.  Nothing is read on the host.
  slots_step    e4m3 experts behind dispatch and before combine: the products read
                the receive buffer.
  MoeLayer      the same layer in training, with 16-bit experts: router, sort, gated
                block, down products and unsort as autograd functions over the
                library's gradients.  Nothing is read on the host.

    python examples/moe_layer.py
"""
from __future__ import annotations

import functools
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


@dataclass
class E4m3Experts:
    """E experts: gate and up rows [E, 2I, H], down rows [E, H, I], with scales by 128 x 128
    block (I and H multiples of 128)."""
    gate_up: torch.Tensor
    gate_up_scales: torch.Tensor
    down: torch.Tensor
    down_scales: torch.Tensor

    @staticmethod
    def of(gate_up: torch.Tensor, down: torch.Tensor) -> "E4m3Experts":
        return E4m3Experts(*moedc.quant_e4m3(gate_up, block_rows=128),
                           *moedc.quant_e4m3(down, block_rows=128))


def decode_step(x: torch.Tensor, logits: torch.Tensor, experts: Int4Experts | E4m3Experts, K: int,
                status: torch.Tensor) -> torch.Tensor:
    """y [T, H] of the tokens x [T, H] with the router's logits [T, E]."""
    E = logits.shape[1]
    idx, w = moedc.gate(logits, K, flags=FLAGS)
    m = moedc.sort(None, idx, E, status=status)          # maps alone: the products gather
    maps = dict(offsets=m.offsets, counts=m.counts, status=status)
    if isinstance(experts, E4m3Experts):
        h = moedc.matmul_e4m3(*moedc.quant_e4m3(x), experts.gate_up, experts.gate_up_scales,
                              src=m.src, top_k=K, swiglu=True, out_dtype=moedc.FP8_E4M3, **maps)
        return moedc.unsort(moedc.matmul_e4m3(*h, experts.down, experts.down_scales, **maps), m.row, w)
    h = moedc.matvec_int4(x, experts.gate_up, experts.gate_up_scales, offsets=m.offsets,
                          counts=m.counts, src=m.src, top_k=K, swiglu=True, status=status)
    out = moedc.matvec_int4(h, experts.down, experts.down_scales, offsets=m.offsets,
                            counts=m.counts, status=status)
    return moedc.unsort(out, m.row, w)


def slots_step(x: torch.Tensor, topk_idx: torch.Tensor, topk_weights: torch.Tensor, E: int, R: int,
               cap: int, experts: E4m3Experts) -> torch.Tensor:
    """y [T, H] through dispatch's receive buffer of cap slots an expert."""
    lay, recv, scales, _ = moedc.layout_dispatch(x, topk_idx, E, R, cap, moedc.FP8_E4M3)
    slots = dict(counts=lay.num_tokens_per_expert, status=lay.status)
    h = moedc.matmul_e4m3(recv, scales, experts.gate_up, experts.gate_up_scales, swiglu=True,
                          out_dtype=moedc.FP8_E4M3, **slots)
    out = moedc.matmul_e4m3(*h, experts.down, experts.down_scales, **slots)
    return moedc.combine(out, topk_idx, lay.slot, topk_weights, status=lay.status)


# ----------------------------------------------------------------- training


class _Refused(torch.autograd.Function):
    """A gradient that has none itself with respect to what it was computed from."""

    @staticmethod
    def forward(ctx, grad, *of):
        return grad.view_as(grad)

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("the layer's operators are differentiable once")


def _once(backward):
    """A backward that refuses second derivatives, of the gradients that it takes and of the tensors
    that its forward saved (torch's once_differentiable looks at the former alone: under a loss that
    is linear in the outputs it leaves the others out)."""
    @functools.wraps(backward)
    def run(ctx, *grads):
        with torch.no_grad():
            out = backward(ctx, *grads)
        if not torch.is_grad_enabled():
            return out
        return tuple(g if g is None else _Refused.apply(g, *grads, *ctx.saved_tensors)
                     for g in (out if isinstance(out, tuple) else (out,)))
    return run


class Gate(torch.autograd.Function):
    """(topk_idx, topk_weights) of logits."""

    @staticmethod
    def forward(ctx, logits, K):
        idx, w = moedc.gate(logits, K, flags=FLAGS)
        ctx.save_for_backward(logits, idx)
        ctx.mark_non_differentiable(idx)
        return idx, w

    @staticmethod
    @_once
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
    @_once
    def backward(ctx, drows, *_):
        return moedc.sort_grad(drows.contiguous(), ctx.saved_tensors[0]), None, None, None


class Unsort(torch.autograd.Function):
    """y of the experts' packed rows and the weights."""

    @staticmethod
    def forward(ctx, rows, w, row, src):
        ctx.save_for_backward(rows, w, row, src)
        return moedc.unsort(rows, row, w)

    @staticmethod
    @_once
    def backward(ctx, dy):
        rows, w, row, src = ctx.saved_tensors
        drows, dw = moedc.unsort_grad(dy.contiguous(), rows if ctx.needs_input_grad[1] else None, row, src, w)
        return drows, dw, None, None


def _rows(like, n):
    """Rows for an output of the experts' products, which leave the padding rows as they are: zeros
    there, as hooks, norms and anomaly detection see them."""
    return torch.zeros((like.shape[0], n), dtype=like.dtype, device=like.device)


def _grad(ctx, dout, rows, w, offsets, counts):
    """(drows, dw) of the experts' products, those that are asked for (a frozen expert's are half of the work)."""
    want_rows, want_w = ctx.needs_input_grad[:2]
    out = _rows(dout, w.shape[2]) if want_rows else None, torch.empty_like(w) if want_w else None
    return moedc.matmul_grad(dout, rows if want_w else None, w if want_rows else None, offsets=offsets,
                             counts=counts, status=ctx.status, out=out)


class Block(torch.autograd.Function):
    """silu(rows Wg^T) * (rows Wu^T) of each expert's rows."""

    @staticmethod
    def forward(ctx, rows, gate_up, offsets, counts, status):
        out = _rows(rows, gate_up.shape[1] // 2), rows.new_empty((rows.shape[0], gate_up.shape[1]))
        h, products = moedc.matmul(rows, gate_up, offsets=offsets, counts=counts, swiglu=True,
                                   keep=True, status=status, out=out)
        ctx.save_for_backward(rows, gate_up, products, offsets, counts)
        ctx.status = status
        return h

    @staticmethod
    @_once
    def backward(ctx, dh):
        rows, gate_up, products, offsets, counts = ctx.saved_tensors
        d = moedc.swiglu_grad(dh.contiguous(), products)
        return *_grad(ctx, d, rows, gate_up, offsets, counts), None, None, None


class Product(torch.autograd.Function):
    """rows W^T of each expert's rows."""

    @staticmethod
    def forward(ctx, rows, w, offsets, counts, status):
        ctx.save_for_backward(rows, w, offsets, counts)
        ctx.status = status
        return moedc.matmul(rows, w, offsets=offsets, counts=counts, status=status,
                            out=_rows(rows, w.shape[1]))

    @staticmethod
    @_once
    def backward(ctx, dout):
        return *_grad(ctx, dout.contiguous(), *ctx.saved_tensors), None, None, None


class MoeLayer(torch.nn.Module):
    """E SwiGLU experts of width I over H channels, K to a token.  `status` collects what
    the experts' products report."""

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
        self.register_buffer("status", torch.zeros(1, dtype=torch.int32, device=device), persistent=False)

    def forward(self, x: torch.Tensor) -> torch.Tensor:
        idx, w = Gate.apply((x @ self.router.T).float(), self.K)
        rows, row, src, offsets, counts = Sort.apply(x, idx, self.E, self.align)
        if x.dtype != torch.float32 and not (self.down.shape[1] % 8 or self.down.shape[2] % 8):
            h = Block.apply(rows, self.gate_up, offsets, counts, self.status)
            return Unsort.apply(Product.apply(h, self.down, offsets, counts, self.status), w, row, src)
        # binary32 and odd widths: the experts' products group by group, the group sizes read
        # on the host
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

    for kind, experts in (("4 bits", experts),
                          ("e4m3", E4m3Experts.of(up.to(torch.bfloat16), down.to(torch.bfloat16)))):
        timed(f"{kind}, call by call", lambda: decode_step(x, logits, experts, K, status))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            y = decode_step(x, logits, experts, K, status)
        timed(f"{kind}, as a CUDA graph", graph.replay)
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
