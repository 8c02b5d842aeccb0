"""The experts' dense layers as workloads: rows and weights to e4m3 with block
scales, products of e4m3 rows and weights, the gated feed-forward block in
bf16 or f16 and its gradients.

`listed()` names the measured cases, `draw()` gives more of the same ranges,
`prepare()` makes a case's inputs on the GPU from a seed, `run()` computes one
pass: through the library where `own` is true, as elementary torch operations
in 32 bits where it is not.  `exact()` gives the same outputs in 64 bits.
"""
from __future__ import annotations

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4, "e4m3": 1}
E4M3 = torch.float8_e4m3fn

# multiplications and weights of the largest listed cases: no drawn case has more
MOST_MACS = 32768 * 4096 * 7168
MOST_E4M3_WEIGHTS = 256 * 4096 * 7168
MOST_WEIGHTS = 64 * 2048 * 7168


def listed():
    return [
        # a serving step's hidden states on their way to 8-bit products: latency
        dict(name="quant 16 tok", kind="quant", E=1, T=16, Kd=7168, block=1, dtype="bf16"),
        # 8 experts' gate and up weights brought to 128 x 128 blocks, the last block not whole
        dict(name="quant weights", kind="quant", E=8, T=4100, Kd=7168, block=128, dtype="bf16"),
        # one token through one linear layer
        dict(name="e4m3 1 tok", kind="e4m3", T=1, E=1, K=1, N=7168, Kd=7168, swiglu=False,
             out="bf16", form="packed"),
        # gate/up products of a serving step with a handful of tokens, e4m3 rows for the down products
        dict(name="e4m3 16 tok swiglu", kind="e4m3", T=16, E=128, K=8, N=1024, Kd=6144,
             swiglu=True, out="e4m3", form="gather"),
        # the low-latency workload's down products over the receive buffer of dispatch
        dict(name="e4m3 128 tok slots", kind="e4m3", T=128, E=288, K=8, N=7168, Kd=2048,
             swiglu=False, out="bf16", form="slots"),
        # the throughput workload's gate/up products
        dict(name="e4m3 4096 tok swiglu", kind="e4m3", T=4096, E=256, K=8, N=2048, Kd=7168,
             swiglu=True, out="e4m3", form="gather"),
        # the gated block over a small batch: the weights' stream
        dict(name="block 64 tok", kind="block", T=64, E=32, K=4, N=1024, Kd=2048, swiglu=True,
             keep=False, align=1, mask=0.0, dtype="bf16", grad=False, dw="bf16"),
        # a training step's gated block, forward, with what its gradient needs
        dict(name="block train", kind="block", T=4096, E=32, K=4, N=2048, Kd=4096, swiglu=True,
             keep=True, align=16, mask=0.0, dtype="bf16", grad=False, dw="bf16"),
        # one dense layer over a long batch, sizes that fill no tile, f16
        dict(name="block dense odd f16", kind="block", T=8191, E=1, K=1, N=4088, Kd=4104,
             swiglu=False, keep=False, align=1, mask=0.0, dtype="f16", grad=False, dw="f16"),
        # the gated block's gradients in small: ragged groups, masked entries, f16
        dict(name="block grad odd f16", kind="block", T=1009, E=60, K=3, N=520, Kd=1032,
             swiglu=True, keep=True, align=1, mask=0.1, dtype="f16", grad=True, dw="f16"),
        # the gradients of the training step above
        dict(name="block grad train", kind="block", T=4096, E=32, K=4, N=2048, Kd=4096,
             swiglu=True, keep=True, align=16, mask=0.0, dtype="bf16", grad=True, dw="bf16"),
        # a down layer's gradients, the weights' in binary32
        dict(name="block grad down", kind="block", T=4096, E=64, K=8, N=7168, Kd=2048,
             swiglu=False, keep=False, align=16, mask=0.0, dtype="bf16", grad=True, dw="f32"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    kind = rng.choice(["quant", "e4m3", "e4m3", "block", "block"])
    if kind == "quant":
        Kd = 128 * _log(rng, 1, 56)
        E = rng.choice([1, 1, 8, 32])
        return dict(kind="quant", E=E, T=_log(rng, 1, min(8192, 8 * 4100 * 7168 // (2 * E * Kd))), Kd=Kd,
                    block=rng.choice([1, 128]), dtype=rng.choice(["bf16", "bf16", "f16", "f32"]))
    if kind == "e4m3":
        E = rng.choice([1, 8, 32, 60, 64, 128, 256, 288])
        K = min(E, rng.choice([1, 2, 4, 6, 8]))
        Kd = 128 * _log(rng, 2, 56)
        swiglu = rng.random() < 0.5
        out = rng.choice(["bf16", "bf16", "f16", "e4m3"])
        form = rng.choice(["packed", "gather", "slots"]) if E > 1 else "packed"
        n = 2 if swiglu else 1
        N = max(128, min(_log(rng, 128, 7168), MOST_E4M3_WEIGHTS // (E * Kd * n)))
        N = N // 128 * 128 if out == "e4m3" else N
        T = _log(rng, 1, max(1, min(4096, MOST_MACS // (K * N * n * Kd), 65536 // E if form == "slots" else 4096)))
        return dict(kind="e4m3", T=T, E=E, K=K, N=N, Kd=Kd, swiglu=swiglu, out=out, form=form)
    E = rng.choice([1, 8, 32, 60, 64])
    K = min(E, rng.choice([1, 2, 4, 8]))
    Kd = 8 * _log(rng, 16, 512)
    swiglu = rng.random() < 0.6
    grad = rng.random() < 0.5
    n = 2 if swiglu else 1
    N = 8 * max(1, min(_log(rng, 16, 896), MOST_WEIGHTS // (8 * E * Kd * n)))
    dtype = rng.choice(["bf16", "bf16", "f16"])
    T = _log(rng, 1, max(1, min(8192, MOST_MACS // (2 * K * N * n * Kd))))
    return dict(kind="block", T=T, E=E, K=K, N=N, Kd=Kd, swiglu=swiglu,
                keep=swiglu and (grad or rng.random() < 0.5), align=rng.choice([1, 1, 8, 16]),
                mask=rng.choice([0.0, 0.0, 0.1]) if E > 1 else 0.0, dtype=dtype, grad=grad,
                dw=rng.choice([dtype, "f32"]) if grad else dtype)


def _rows(c):
    """Rows of the packed buffer: every entry, and the padding of each expert's group."""
    return c["T"] * c["K"] + min(c["E"], c["T"] * c["K"]) * (c.get("align", 1) - 1)


def _active(c):
    """Experts that some token goes to, expected (uniform distinct choices)."""
    return c["E"] * (1.0 - (1.0 - c["K"] / c["E"]) ** c["T"])


def work(case):
    c = case
    if c["kind"] == "quant":
        n = c["E"] * c["T"] * c["Kd"]
        scales = c["E"] * -(-c["T"] // c["block"]) * (c["Kd"] // 128)
        return {"bytes": n * (SIZES[c["dtype"]] + 1) + 4 * scales, "flops": 2.0 * n}
    n = c["N"] * (2 if c["swiglu"] else 1)
    live = c["T"] * c["K"] * (1.0 - c.get("mask", 0.0))
    if c["kind"] == "e4m3":
        groups = c["Kd"] // 128
        blocks = (2 if c["swiglu"] else 1) * -(-c["N"] // 128)
        rows_in = c["T"] if c["form"] == "gather" else live
        b = _active(c) * (n * c["Kd"] + 4 * blocks * groups) + rows_in * (c["Kd"] + 4 * groups)
        b += live * (c["N"] + c["N"] // 32 if c["out"] == "e4m3" else 2 * c["N"])
        return {"bytes": b, "flops": 2.0 * live * n * c["Kd"]}
    weights = c["E"] * n * c["Kd"]
    if not c["grad"]:
        b = 2 * _active(c) * n * c["Kd"] + 2 * live * (c["Kd"] + c["N"] + (n if c["keep"] else 0))
        return {"bytes": b, "flops": 2.0 * live * n * c["Kd"]}
    b = 2 * _active(c) * n * c["Kd"] + weights * SIZES[c["dw"]] + 2 * live * 2 * c["Kd"]
    b += 2 * live * (c["N"] + 2 * n if c["swiglu"] else n)
    return {"bytes": b, "flops": 4.0 * live * n * c["Kd"]}


# ------------------------------------------------------------------ inputs


def _routing(c, g):
    """Distinct experts per token, some more popular than others; -1 where masked."""
    T, E, K = c["T"], c["E"], c["K"]
    z = torch.randn(E, generator=g, device="cuda") * 0.5
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    idx = (z - torch.log(-torch.log(u))).topk(K, dim=1).indices
    if c.get("mask"):
        idx = idx.masked_fill(torch.rand(T, K, generator=g, device="cuda") < c["mask"], -1)
    return idx.cpu()


def _groups(c, idx):
    """(offsets, counts, src) of the packed rows, as lists: entries by expert, then by token."""
    T, E, K = c["T"], c["E"], c["K"]
    flat = idx.reshape(-1).tolist()
    groups = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if e >= 0:
            groups[e].append(i)
    align = c.get("align", 1)
    offsets, src = [0], [-1] * _rows(c)
    for group in groups:
        src[offsets[-1]:offsets[-1] + len(group)] = group
        offsets.append(offsets[-1] + -(-len(group) // align) * align)
    return offsets, [len(group) for group in groups], src


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _randn(g, dt, *shape):
    """Normal values, made part by part."""
    out = torch.empty(*shape, dtype=dt, device="cuda")
    for part in (out if out.dim() == 3 else out[None]):
        part.copy_(torch.randn(*part.shape, generator=g, device="cuda"))
    return out


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    s = {"case": dict(c), "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "out": None}

    if c["kind"] == "quant":
        s["x"] = _randn(g, DTYPES[c["dtype"]], c["E"], c["T"], c["Kd"])
        # outlier rows
        s["x"][torch.rand(c["E"], c["T"], generator=g, device="cuda") < 0.01] *= 100.0
        if c["block"] == 1:
            s["x"] = s["x"].reshape(-1, c["Kd"])
        return s

    T, E, K, N, Kd = (c[k] for k in ("T", "E", "K", "N", "Kd"))
    n = N * (2 if c["swiglu"] else 1)
    offsets, counts, src = _groups(c, _routing(c, g))
    rows = len(src)
    s["counts"] = _i32(counts)
    if c["kind"] == "e4m3":
        G = Kd // 128
        blocks = (2 if c["swiglu"] else 1) * -(-N // 128)
        s["w"] = _randn(g, E4M3, E, n, Kd)
        s["ws"] = (0.5 + torch.rand(E, blocks, G, generator=g, device="cuda")) / Kd ** 0.5
        x_rows = T if c["form"] == "gather" else rows
        if c["form"] == "slots":        # the receive buffer: rows behind an expert's count are old ones
            cap = s["cap"] = T
            x_rows = E * cap
            offsets = [e * cap for e in range(E + 1)]
        s["x"] = _randn(g, E4M3, x_rows, Kd)
        s["xs"] = torch.rand(x_rows, G, generator=g, device="cuda") * 0.5 + 0.5
        if c["form"] == "gather":
            s["src"] = _i32(src)
            s["token"] = (s["src"].long() // K)
            x_rows = rows
        # rows that belong to no expert are not written
        if c["out"] == "e4m3":
            s["out"] = (torch.zeros(x_rows, N, dtype=E4M3, device="cuda"),
                        torch.zeros(x_rows, N // 128, device="cuda"))
        else:
            s["out"] = torch.zeros(x_rows, N, dtype=DTYPES[c["out"]], device="cuda")
    else:
        dt = DTYPES[c["dtype"]]
        s["w"] = _randn(g, dt, E, n, Kd).mul_(Kd ** -0.5)
        s["x"] = _randn(g, dt, rows, Kd)
        if c["grad"]:
            s["dout"] = _randn(g, dt, rows, N)
            if c["swiglu"]:
                s["gu"] = _randn(g, dt, rows, n)
            s["dgu"] = torch.zeros(rows, n, dtype=dt, device="cuda") if c["swiglu"] else s["dout"]
            s["out"] = (torch.zeros(rows, Kd, dtype=dt, device="cuda"),
                        torch.empty(E, n, Kd, dtype=DTYPES[c["dw"]], device="cuda"))
        else:
            s["out"] = torch.zeros(rows, N, dtype=dt, device="cuda")
            if c["keep"]:
                s["out"] = (s["out"], torch.zeros(rows, n, dtype=dt, device="cuda"))
    s["offsets"] = _i32(offsets)
    # a plan that the program keeps: the groups by number, for products group by group
    s["groups"] = [(e, offsets[e], offsets[e] + counts[e]) for e in range(E) if counts[e]]
    return s


# --------------------------------------------------------------- plain form


def _to_e4m3(v, scale):
    return (v / scale).clamp(-448.0, 448.0).to(E4M3)


def _plain_quant(s):
    c, x = s["case"], s["x"]
    G = c["Kd"] // 128
    if c["block"] == 1:
        v = x.float().reshape(x.shape[0], G, 128)
        scale = v.abs().amax(2).clamp(min=1e-4) / 448.0
        return _to_e4m3(v, scale[..., None]).reshape(x.shape), scale
    E, N, Kd = x.shape
    codes, scales = torch.empty(E, N, Kd, dtype=E4M3, device=x.device), []
    for e in range(E):
        v = torch.zeros(-(-N // 128) * 128, Kd, device=x.device)
        v[:N] = x[e].float()
        v = v.reshape(-1, 128, G, 128)
        scale = v.abs().amax((1, 3)).clamp(min=1e-4) / 448.0
        codes[e] = _to_e4m3(v, scale[:, None, :, None]).reshape(-1, Kd)[:N]
        scales.append(scale)
    return codes, torch.stack(scales)


def _silu_mul(a, N):
    g, u = a[:, :N], a[:, N:]
    return g * torch.sigmoid(g) * u


def _plain_e4m3(s):
    c = s["case"]
    N, Kd = c["N"], c["Kd"]
    G, parts = Kd // 128, 2 if c["swiglu"] else 1
    rows_of_block = torch.arange(N, device=s["x"].device) // 128
    blocks = -(-N // 128)
    at = torch.cat([rows_of_block + p * blocks for p in range(parts)])
    out = s["out"]
    for e, a, b in s["groups"]:
        pick = s["token"][a:b] if c["form"] == "gather" else slice(a, b)
        x = (s["x"][pick].float().reshape(-1, G, 128) * s["xs"][pick][..., None]).reshape(-1, Kd)
        w = (s["w"][e].float().reshape(-1, G, 128) * s["ws"][e][at][..., None]).reshape(-1, Kd)
        v = x @ w.T
        if c["swiglu"]:
            v = _silu_mul(v, N)
        if c["out"] != "e4m3":
            out[a:b] = v.to(out.dtype)
            continue
        v = v.reshape(b - a, N // 128, 128)
        scale = v.abs().amax(2).clamp(min=1e-4) / 448.0
        out[0][a:b] = _to_e4m3(v, scale[..., None]).reshape(b - a, N)
        out[1][a:b] = scale
    return out


def _plain_block(s):
    c = s["case"]
    N = c["N"]
    if not c["grad"]:
        h = s["out"][0] if c["keep"] else s["out"]
        for e, a, b in s["groups"]:
            v = s["x"][a:b].float() @ s["w"][e].float().T
            if c["keep"]:
                s["out"][1][a:b] = v.to(h.dtype)
            h[a:b] = (_silu_mul(v, N) if c["swiglu"] else v).to(h.dtype)
        return s["out"]
    d = s["dgu"]
    if c["swiglu"]:
        g, u, dh = s["gu"][:, :N].float(), s["gu"][:, N:].float(), s["dout"].float()
        sig = torch.sigmoid(g)
        d.copy_(torch.cat([dh * u * sig * (1.0 + g * (1.0 - sig)), dh * g * sig], 1))
    dx, dw = s["out"]
    dw.zero_()
    for e, a, b in s["groups"]:
        v = d[a:b].float()
        dx[a:b] = (v @ s["w"][e].float()).to(dx.dtype)
        dw[e] = (v.T @ s["x"][a:b].float()).to(dw.dtype)
    return (d, dx, dw) if c["swiglu"] else (dx, dw)


# -------------------------------------------------------------------- runs


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"quant": _plain_quant, "e4m3": _plain_e4m3, "block": _plain_block}[c["kind"]](s)
    from combine_moedc_layout_gb300 import moedc
    if c["kind"] == "quant":
        s["out"] = moedc.quant_e4m3(s["x"], block_rows=c["block"], out=s["out"])
        return s["out"]
    if c["kind"] == "e4m3":
        out_dtype = moedc.FP8_E4M3 if c["out"] == "e4m3" else moedc.F16 if c["out"] == "f16" else moedc.BF16
        x, xs, out, maps = s["x"], s["xs"], s["out"], {"offsets": s["offsets"]}
        if c["form"] == "gather":
            maps.update(src=s["src"], top_k=c["K"])
        if c["form"] == "slots":
            slots = (c["E"], s["cap"], -1)
            x, xs, maps = x.view(slots), xs.view(slots), {}
            out = tuple(o.view(slots) for o in out) if c["out"] == "e4m3" else out.view(slots)
        moedc.matmul_e4m3(x, xs, s["w"], s["ws"], counts=s["counts"], swiglu=c["swiglu"],
                          out_dtype=out_dtype, status=s["status"], out=out, **maps)
        return s["out"]
    maps = dict(offsets=s["offsets"], counts=s["counts"], status=s["status"])
    if not c["grad"]:
        return moedc.matmul(s["x"], s["w"], swiglu=c["swiglu"], keep=c["keep"], out=s["out"], **maps)
    if not c["swiglu"]:
        return moedc.matmul_grad(s["dout"], s["x"], s["w"], out=s["out"], **maps)
    moedc.swiglu_grad(s["dout"], s["gu"], out=s["dgu"])
    return s["dgu"], *moedc.matmul_grad(s["dgu"], s["x"], s["w"], out=s["out"], **maps)


# -------------------------------------------------------------- 64-bit form


def _e4m3_nearest(q):
    """Nearest e4m3 value of q, ties to the even one: three fraction bits, exponents from -6."""
    power = torch.clamp(torch.floor(torch.log2(q.abs().clamp(min=2.0 ** -60))), min=-6.0)
    step = torch.exp2(power - 3.0)
    return (torch.round(q / step) * step).clamp(-448.0, 448.0)


def _exact_quant(s):
    """The scale and the quotient are binary32 by definition; the code is the nearest to the quotient."""
    c = s["case"]
    x = s["x"] if s["x"].dim() == 3 else s["x"][None]
    codes, scales = [], []
    for part in x:
        R, B = part.shape[0], c["block"]
        scale = torch.empty(-(-R // B), c["Kd"] // 128, device=x.device)
        for i in range(0, c["Kd"], 128):
            peak = part[:, i:i + 128].double().abs().max(1).values
            peak = torch.cat([peak, peak.new_zeros(-R % B)]).reshape(-1, B).max(1).values
            scale[:, i // 128] = torch.maximum(peak, torch.full_like(peak, 1e-4)).float() / 448.0
        wide = scale.repeat_interleave(B, 0)[:R].repeat_interleave(128, 1)
        codes.append(_e4m3_nearest((part.float() / wide).double()))
        scales.append(scale.double())
    codes, scales = torch.stack(codes), torch.stack(scales)
    return (codes, scales) if s["x"].dim() == 3 else (codes[0], scales[0])


def _silu64(a):
    return a / (1.0 + torch.exp(-a))


def _exact_e4m3(s):
    c = s["case"]
    N, Kd = c["N"], c["Kd"]
    outs = s["out"] if c["out"] == "e4m3" else (s["out"],)
    v = torch.zeros(outs[0].shape, dtype=torch.float64, device=s["x"].device)
    for e, a, b in s["groups"]:
        rows = s["src"][a:b].long() // c["K"] if c["form"] == "gather" else torch.arange(a, b, device=v.device)
        x = s["x"][rows].double() * s["xs"][rows].double().repeat_interleave(128, 1)

        def product(first, first_block):
            blocks = -(-N // 128)
            scale = s["ws"][e, first_block:first_block + blocks].double()
            scale = scale.repeat_interleave(128, 0)[:N].repeat_interleave(128, 1)
            return x @ (s["w"][e, first:first + N].double() * scale).T

        p = product(0, 0)
        v[a:b] = _silu64(p) * product(N, -(-N // 128)) if c["swiglu"] else p
    if c["out"] != "e4m3":
        return v
    # the quotients themselves: a code is within half a step of its own
    scale = torch.zeros(outs[1].shape, dtype=torch.float64, device=v.device)
    for _, a, b in s["groups"]:
        peak = v[a:b].reshape(b - a, -1, 128).abs().max(2).values
        scale[a:b] = torch.maximum(peak, torch.full_like(peak, 1e-4)) / 448.0
        v[a:b] /= scale[a:b].repeat_interleave(128, 1)
    return v, scale


def _exact_block(s):
    c = s["case"]
    N, n = c["N"], s["w"].shape[1]
    rows, Kd = s["x"].shape
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device=s["x"].device)  # noqa: E731
    if not c["grad"]:
        h, kept = zeros(rows, N), zeros(rows, n) if c["keep"] else None
        for e, a, b in s["groups"]:
            v = torch.einsum("rk,nk->rn", s["x"][a:b].double(), s["w"][e].double())
            if c["keep"]:
                kept[a:b] = v
            h[a:b] = _silu64(v[:, :N]) * v[:, N:] if c["swiglu"] else v
        return (h, kept) if c["keep"] else h
    if c["swiglu"]:
        g, u = (t.double() for t in s["gu"].split(N, dim=1))
        d = s["dout"].double()
        decay = torch.exp(-g)
        slope = (1.0 + decay + g * decay) / (1.0 + decay) ** 2
        d = torch.cat([d * u * slope, d * _silu64(g)], 1)
    else:
        d = s["dout"].double()
    dx, dw = zeros(rows, Kd), zeros(c["E"], n, Kd)
    for e, a, b in s["groups"]:
        v = d[a:b].to(s["x"].dtype).double()         # of the rounded gradient before the activation
        dx[a:b] = torch.einsum("rn,nk->rk", v, s["w"][e].double())
        dw[e] = torch.einsum("rn,rk->nk", v, s["x"][a:b].double())
    return (d, dx, dw) if c["swiglu"] else (dx, dw)


def exact(case, seed):
    macs = case["T"] * case["K"] * case["N"] * case["Kd"] * (2 if case["swiglu"] else 1) if "N" in case else 0
    if macs * (2 if case.get("grad") else 1) > 4 * MOST_MACS or not math.isfinite(macs):
        return None
    return {"quant": _exact_quant, "e4m3": _exact_e4m3, "block": _exact_block}[case["kind"]](prepare(case, seed))
