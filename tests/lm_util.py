"""Plain 64-bit forms of the language-model operators (router, sorted rows,
4-bit products) on the CPU, and the bounds that binary32 arithmetic gives."""
from __future__ import annotations

import torch

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U32 = 2.0 ** -24                      # half an ulp, relative: 2^-p for p significant bits
ROUND = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: U32}
# half the subnormal spacing (f16 is the one whose results reach it here)
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}


def rounding(ref: torch.Tensor, dtype: torch.dtype) -> torch.Tensor:
    """Error of rounding `ref` once to `dtype`."""
    return ref.abs() * ROUND[dtype] + TINY[dtype]


def assert_within(got: torch.Tensor, ref: torch.Tensor, bound) -> None:
    got = got.detach().to(ref.device).double()
    assert got.shape == ref.shape
    assert not torch.isnan(got).any()
    over = (got - ref).abs() - bound
    assert (over <= 0).all(), (over.max().item(), (over > 0).sum().item())


# ------------------------------------------------------------------- router


def gate_ref(logits, K, bias=None, sigmoid=False, normalize=True, scale=1.0):
    """(idx int32, w f64) by picking the best remaining expert K times."""
    l32 = logits.cpu().float()
    key = l32 + (bias.cpu().float() if bias is not None else 0.0)
    fmax = torch.finfo(torch.float32).max
    l = l32.double().clamp(max=fmax)
    T, E = l.shape
    idx = torch.full((T, K), -1, dtype=torch.int32)
    w = torch.zeros((T, K), dtype=torch.float64)
    for t in range(T):
        ok = [e for e in range(E) if l32[t, e] > -float("inf") and key[t, e] > -float("inf")]
        order = sorted(ok, key=lambda e: (-float(key[t, e]), e))[:K]
        if not order:
            continue
        idx[t, :len(order)] = torch.tensor(order, dtype=torch.int32)
        w[t, :len(order)] = _weights(l[t], order, ok, sigmoid, normalize) * scale
    return idx, w


def _weights(l, order, ok, sigmoid, normalize):
    c = l[order]
    if sigmoid:
        # as in binary32, a sigmoid below the smallest binary32 number is 0
        s = torch.sigmoid(c)
        s = torch.where(s < 2.0 ** -150, torch.zeros_like(s), s)
        if not normalize:
            return s
        return s / s.sum() if s.sum() > 0 else torch.zeros_like(s)
    over = c if normalize else l[ok]
    m = over.max()
    return torch.exp(c - m) / torch.exp(over - m).sum()


def gate_grad_ref(logits, idx, dw, bias=None, sigmoid=False, normalize=True, scale=1.0):
    """dlogits in 64 bits by automatic differentiation of the weights."""
    l32 = logits.cpu().float()
    key = l32 + (bias.cpu().float() if bias is not None else 0.0)
    T, E = l32.shape
    out = torch.zeros((T, E), dtype=torch.float64)
    for t in range(T):
        live = [k for k in range(idx.shape[1]) if idx[t, k] >= 0]
        if not live:
            continue
        order = [int(idx[t, k]) for k in live]
        ok = [e for e in range(E) if l32[t, e] > -float("inf") and key[t, e] > -float("inf")]
        l = l32[t].double().clone().requires_grad_(True)
        w = _weights(l, order, ok, sigmoid, normalize) * scale
        (w * dw[t, live].cpu().double()).sum().backward()
        out[t] = torch.nan_to_num(l.grad)
    return out


# -------------------------------------------------------------- sorted rows


def sort_ref(topk_idx, E, align, rows):
    """(row, src, offsets, counts) by walking the entries; entries past `rows` dropped."""
    T, K = topk_idx.shape
    flat = topk_idx.cpu().reshape(-1).tolist()
    groups = [[i for i, e in enumerate(flat) if e == x] for x in range(E)]
    row = torch.full((T * K,), -1, dtype=torch.int32)
    src = torch.full((rows,), -1, dtype=torch.int32)
    offsets = [0]
    for g in groups:
        for s, i in enumerate(g):
            r = offsets[-1] + s
            if r < rows:
                row[i] = r
                src[r] = i
        offsets.append(offsets[-1] + -(-len(g) // align) * align)
    offsets = torch.tensor([min(o, rows) for o in offsets], dtype=torch.int32)
    return row.reshape(T, K), src, offsets, torch.tensor([len(g) for g in groups],
                                                         dtype=torch.int32)


def unsort_ref(sorted_, row, w):
    """(y, sum of magnitudes) in 64 bits."""
    T, K = row.shape
    H = sorted_.shape[1]
    s = sorted_.cpu().double()
    y, mag = torch.zeros(T, H, dtype=torch.float64), torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            r = int(row[t, k])
            if 0 <= r < s.shape[0]:
                v = s[r] * (1.0 if w is None else w[t, k].cpu().double())
                y[t] += v
                mag[t] += v.abs()
    return y, mag


# ------------------------------------------------------------ 4-bit weights


def int4_weights(wq, scales, zeros, group):
    """f64 [.., N, Kd] of the packed form, where wq is."""
    q = wq
    w = torch.empty(*q.shape[:-1], 2 * q.shape[-1], dtype=torch.float64, device=q.device)
    w[..., 0::2] = (q % 16).double()
    w[..., 1::2] = (q // 16).double()
    w -= 8.0 if zeros is None else zeros.double().repeat_interleave(group, -1)
    w *= scales.double().repeat_interleave(group, -1)
    return w


def matvec_ref(x_rows, w, swiglu):
    """(out, bound on the binary32 sums' error) of x_rows [r, Kd] with w [n, Kd].
    A sum of Kd products in some 8 parallel chains, their join and the group
    scales: (Kd / 8 + 64) roundings of at most half an ulp of the magnitudes."""
    x = x_rows.to(w.device).double()
    v, mag = x @ w.T, x.abs() @ w.abs().T
    err = (x.shape[1] / 8 + 64) * U32 * mag
    if not swiglu:
        return v, err
    n = w.shape[0] // 2
    a, b, ea, eb = v[:, :n], v[:, n:], err[:, :n], err[:, n:]
    silu = a * torch.sigmoid(a)
    # |silu'| <= 1.1; eight more roundings of the result in the epilogue
    return silu * b, 1.1 * ea * (b.abs() + eb) + silu.abs() * eb + 16 * U32 * (silu * b).abs()
