"""The library's language-model operators as workloads: top-k router, rows
sorted by expert and back (forward and gradient), expert products with 4-bit
weights.

`listed()` names the measured cases, `draw()` gives more of the same ranges,
`prepare()` makes a case's inputs on the GPU from a seed, `run()` computes one
pass: through the library where `own` is true, as elementary torch operations
in 32 bits where it is not.  `exact()` gives the same outputs in 64 bits.
"""
from __future__ import annotations

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
SIZES = {"bf16": 2, "f16": 2, "f32": 4}

# 4096 tokens x top-8 x 7168 channels: the throughput workload's rows
MOST_ROW_VALUES = 4096 * 8 * 7168
# 288 experts x 2048 outputs x 7168 channels
MOST_WEIGHTS = 288 * 2048 * 7168


def listed():
    return [
        # router of a serving step with a handful of tokens: one launch, latency
        dict(name="gate 16 tok", kind="gate", T=16, E=128, K=8, score="softmax", normalize=True,
             bias=False, mask=0.0, dtype="f32", grad=False),
        # serving step with the balance bias, bf16 logits (many ties), an odd token count,
        # masked experts and tokens whose mask leaves nothing
        dict(name="gate 1021 tok bias", kind="gate", T=1021, E=288, K=8, score="sigmoid",
             normalize=True, bias=True, mask=0.05, dtype="bf16", grad=False),
        # router of a training step over a long batch, with the gradient to the logits
        dict(name="gate train 32768 tok", kind="gate", T=32768, E=256, K=8, score="softmax",
             normalize=False, bias=False, mask=0.0, dtype="f32", grad=True),
        # sorted and back in a serving step: latency
        dict(name="sort 16 tok", kind="sort", T=16, H=6144, K=8, E=128, align=1, mask=0.0,
             dtype="bf16", grad=False),
        # the throughput workload, packed, forward
        dict(name="sort 4096 tok", kind="sort", T=4096, H=7168, K=8, E=256, align=1, mask=0.0,
             dtype="bf16", grad=False),
        # its gradients
        dict(name="sort grad 4096 tok", kind="sort", T=4096, H=7168, K=8, E=256, align=1,
             mask=0.0, dtype="bf16", grad=True),
        # masked entries, groups padded to a grouped GEMM's tile of 128 rows
        dict(name="sort 2048 tok padded", kind="sort", T=2048, H=4096, K=4, E=32, align=128,
             mask=0.1, dtype="bf16", grad=False),
        # binary32 training with an odd width (no 16-byte rows) and an odd token count
        dict(name="sort grad odd f32", kind="sort", T=1009, H=2047, K=3, E=60, align=16,
             mask=0.1, dtype="f32", grad=True),
        # one token through one 4-bit linear layer
        dict(name="int4 1 tok", kind="int4", T=1, E=1, K=1, N=7168, Kd=7168, group=128,
             swiglu=False, zeros=False, dtype="bf16"),
        # gate/up products of a serving step with a handful of tokens
        dict(name="int4 16 tok swiglu", kind="int4", T=16, E=128, K=8, N=1024, Kd=6144, group=128,
             swiglu=True, zeros=False, dtype="bf16"),
        # the low-latency workload: 128 tokens over 288 experts, asymmetric groups of 64
        dict(name="int4 128 tok zeros", kind="int4", T=128, E=288, K=8, N=2048, Kd=7168, group=64,
             swiglu=False, zeros=True, dtype="bf16"),
        # a larger batch over few experts, some 32 rows each; f16, odd output count, groups of 32
        dict(name="int4 255 tok f16", kind="int4", T=255, E=32, K=4, N=2050, Kd=2048, group=32,
             swiglu=False, zeros=False, dtype="f16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, round(lo * (hi / lo) ** rng.random())))


def draw(rng):
    kind = rng.choice(["gate", "sort", "sort", "int4", "int4"])
    if kind == "gate":
        E = rng.choice([32, 60, 64, 100, 128, 160, 256, 288])
        return dict(kind="gate", T=_log(rng, 1, 32768), E=E, K=rng.choice([1, 2, 4, 6, 8]),
                    score=rng.choice(["softmax", "sigmoid"]), normalize=rng.random() < 0.6,
                    bias=rng.random() < 0.5, mask=rng.choice([0.0, 0.05]),
                    dtype=rng.choice(["f32", "bf16", "f16"]), grad=rng.random() < 0.5)
    if kind == "sort":
        dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
        K = rng.choice([1, 2, 3, 4, 6, 8])
        # odd widths, odd multiples of 8 (16-byte rows) and of 128
        H = rng.choice([_log(rng, 64, 7168) | 1, 8 * (_log(rng, 16, 895) | 1), 128 * (_log(rng, 1, 55) | 1)])
        most = min(4096, MOST_ROW_VALUES * 2 // (SIZES[dtype] * K * H))
        return dict(kind="sort", T=_log(rng, 1, most), H=H, K=K,
                    E=rng.choice([8, 32, 60, 64, 128, 256, 288]),
                    align=rng.choice([1, 1, 8, 16, 32]), mask=rng.choice([0.0, 0.0, 0.1]),
                    dtype=dtype, grad=rng.random() < 0.5)
    group = rng.choice([32, 64, 128])
    E = rng.choice([1, 8, 32, 60, 64, 128, 256])
    swiglu = rng.random() < 0.4
    Kd = group * (_log(rng, 512 // group, 7168 // group - 1) | 1)     # an odd number of groups
    N = min(_log(rng, 128, 2048), MOST_WEIGHTS // (E * Kd * (2 if swiglu else 1)))
    return dict(kind="int4", T=_log(rng, 1, 256), E=E, K=min(E, rng.choice([1, 2, 4, 6, 8])),
                N=N, Kd=Kd, group=group, swiglu=swiglu, zeros=rng.random() < 0.4,
                dtype=rng.choice(["bf16", "bf16", "f16"]))


def _rows(c):
    """Rows of the packed buffer: every entry, and the padding of each expert's group."""
    return c["T"] * c["K"] + min(c["E"], c["T"] * c["K"]) * (c.get("align", 1) - 1)


def _active(c):
    """Experts that some token goes to, expected (uniform distinct choices)."""
    return c["E"] * (1.0 - (1.0 - c["K"] / c["E"]) ** c["T"])


def work(case):
    c = case
    if c["kind"] == "gate":
        s = SIZES[c["dtype"]]
        T, E, K = c["T"], c["E"], c["K"]
        b = T * E * s + 8 * T * K
        if c["grad"]:
            # the gradient needs every logit only where the softmax ran over all of them
            again = E if c["score"] == "softmax" and not c["normalize"] else K
            b += T * again * s + 8 * T * K + T * E * s
        return {"bytes": b, "flops": 4.0 * T * E}
    if c["kind"] == "sort":
        s = SIZES[c["dtype"]]
        T, H, K = c["T"], c["H"], c["K"]
        live, rows = T * K * (1.0 - c["mask"]), _rows(c)
        if c["grad"]:
            # dy and the experts' rows in, drows and dw out; drows in, dx out
            b = T * H * s + live * H * s + rows * H * s + 12 * T * K + 4 * rows
            b += live * H * s + T * H * s + 4 * T * K
            return {"bytes": b, "flops": live * H * 4.0}
        # x in, rows out with their maps; the experts' rows in, y out
        b = T * H * s + rows * H * s + 8 * T * K + 4 * rows
        b += live * H * s + T * H * s + 8 * T * K
        return {"bytes": b, "flops": live * H * 2.0}
    n = c["N"] * (2 if c["swiglu"] else 1)
    groups = c["Kd"] // c["group"]
    per = n * (c["Kd"] / 2 + groups * (3 if c["zeros"] else 2))
    rows = c["T"] * c["K"]
    return {"bytes": _active(c) * per + 2 * c["T"] * c["Kd"] + 2 * rows * c["N"],
            "flops": 2.0 * rows * n * c["Kd"]}


# ------------------------------------------------------------------ inputs


def _routing(c, g):
    """Distinct experts per token, some more popular than others; -1 where masked."""
    T, E, K = c["T"], c["E"], c["K"]
    z = torch.randn(E, generator=g, device="cuda") * 0.5
    u = torch.rand(T, E, generator=g, device="cuda").clamp_(1e-6, 1 - 1e-6)
    idx = (z - torch.log(-torch.log(u))).topk(K, dim=1).indices.to(torch.int32)
    if c.get("mask"):
        idx = idx.masked_fill(torch.rand(T, K, generator=g, device="cuda") < c["mask"], -1)
    w = torch.softmax(torch.randn(T, K, generator=g, device="cuda"), dim=1)
    return idx.contiguous(), w.contiguous()


def _maps(idx, E, align, rows):
    """(row, src, offsets, counts) of the rows sorted by expert, from a stable sort."""
    T, K = idx.shape
    key = torch.where(idx < 0, E, idx).reshape(-1)
    skey, order = torch.sort(key, stable=True)
    edges = torch.arange(E + 1, device=idx.device, dtype=skey.dtype)
    start = torch.searchsorted(skey, edges)
    counts = start[1:] - start[:-1]
    padded = (counts + align - 1) // align * align
    offsets = torch.cat([padded.new_zeros(1), padded.cumsum(0)])
    live = skey < E
    e = torch.where(live, skey, 0).long()
    at = offsets[e] + torch.arange(T * K, device=idx.device) - start[e]
    row = torch.empty(T * K, dtype=torch.int64, device=idx.device)
    row[order] = torch.where(live, at, -1)
    src = torch.full((rows + 1,), -1, dtype=torch.int64, device=idx.device)
    src[torch.where(live, at, rows)] = torch.where(live, order, -1)
    i32 = torch.int32
    return (row.reshape(T, K).to(i32), src[:rows].to(i32).contiguous(), offsets.to(i32),
            counts.to(i32))


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    dt = DTYPES[c["dtype"]]

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dt)

    s = {"case": dict(c), "status": torch.zeros(1, dtype=torch.int32, device="cuda"), "out": {}}
    if c["kind"] == "gate":
        T, E = c["T"], c["E"]
        z = torch.randn(T, E, generator=g, device="cuda") * 1.5
        z += torch.randn(E, generator=g, device="cuda") * 0.5
        if c["mask"]:
            z.masked_fill_(torch.rand(T, E, generator=g, device="cuda") < c["mask"], float("-inf"))
            z.masked_fill_(torch.rand(T, 1, generator=g, device="cuda") < 0.01, float("-inf"))
        s["logits"] = z.to(dt)
        s["bias"] = torch.randn(E, generator=g, device="cuda") * 0.3 if c["bias"] else None
        s["dw"] = torch.randn(T, c["K"], generator=g, device="cuda")
        return s
    s["idx"], s["w"] = _routing(c, g)
    rows = _rows(c)
    s["rows"] = rows
    s["row"], s["src"], s["offsets"], s["counts"] = _maps(s["idx"], c["E"], c.get("align", 1), rows)
    if c["kind"] == "sort":
        s["x"] = randn(c["T"], c["H"])            # hidden states, or dy
        s["expert_out"] = randn(rows, c["H"])
        return s
    n = c["N"] * (2 if c["swiglu"] else 1)
    groups = c["Kd"] // c["group"]
    s["x"] = randn(c["T"], c["Kd"])
    s["wq"] = torch.randint(0, 256, (c["E"], n, c["Kd"] // 2), dtype=torch.uint8, generator=g,
                            device="cuda")
    u = torch.rand(c["E"], n, groups, generator=g, device="cuda")
    s["scales"] = ((0.5 + u) * (0.2 / c["Kd"] ** 0.5)).to(dt)
    s["zeros"] = (torch.randint(0, 16, (c["E"], n, groups), dtype=torch.uint8, generator=g,
                                device="cuda") if c["zeros"] else None)
    return s


# --------------------------------------------------------------- plain form


def _plain_gate(s):
    c = s["case"]
    l32 = s["logits"].float()
    key = l32 + s["bias"] if c["bias"] else l32 + 0.0
    ok = (l32 > float("-inf")) & (key > float("-inf"))
    order = torch.sort(torch.where(ok, key, float("-inf")), dim=1, descending=True, stable=True)
    idx = order.indices[:, :c["K"]]
    live = ok.gather(1, idx)
    zero = torch.zeros((), device=l32.device)
    chosen = l32.gather(1, idx)
    if c["score"] == "sigmoid":
        sig = torch.where(live, torch.sigmoid(chosen), zero)
        total = sig.sum(1, keepdim=True) if c["normalize"] else None
        w = torch.where(total > 0, sig / total, zero) if c["normalize"] else sig
    else:
        over, on = (chosen, live) if c["normalize"] else (l32, ok)
        top = torch.where(on, over, float("-inf")).amax(1, keepdim=True)
        top = torch.where(top > float("-inf"), top, zero)
        den = torch.where(on, torch.exp(over - top), zero).sum(1, keepdim=True)
        w = torch.where(live, torch.exp(chosen - top) / den, zero)
    idx32 = torch.where(live, idx, -1).to(torch.int32)
    if not c["grad"]:
        return idx32, w
    d = torch.where(live, s["dw"], zero)
    safe = torch.where(live, idx, 0)
    if c["score"] == "sigmoid":
        slope = sig * torch.sigmoid(-chosen)
        if c["normalize"]:
            dot = (w * d).sum(1, keepdim=True)
            dc = torch.where(total > 0, slope / total * (d - dot), zero)
        else:
            dc = slope * d
        dl = torch.zeros_like(l32).scatter_add_(1, safe, torch.where(live, dc, zero))
    else:
        dot = (w * d).sum(1, keepdim=True)
        if c["normalize"]:
            dl = torch.zeros_like(l32).scatter_add_(1, safe, torch.where(live, w * (d - dot), zero))
        else:
            p = torch.where(ok, torch.exp(l32 - top) / den, zero)
            dl = -p * dot
            dl = dl.scatter_add_(1, safe, torch.where(live, w * d, zero))
    return idx32, w, dl.to(s["logits"].dtype)


def _plain_back(rows, row, w):
    """sum over k of w * rows[row], in binary32."""
    live = (row >= 0)[..., None]
    got = torch.where(live, rows[row.clamp(min=0).long()].float(), 0.0)
    return (got if w is None else got * w[..., None]).sum(1), got


def _plain_sort(s):
    c = s["case"]
    x, K = s["x"], c["K"]
    if not c["grad"]:
        row, src, offsets, counts = _maps(s["idx"], c["E"], c["align"], s["rows"])
        live = (src >= 0)[:, None]
        rows = torch.where(live, x[src.clamp(min=0).long() // K], torch.zeros((), dtype=x.dtype, device=x.device))
        y, _ = _plain_back(s["expert_out"], row, s["w"])
        return rows, row, src, offsets, counts, y.to(x.dtype)
    dy = x.float()
    _, got = _plain_back(s["expert_out"], s["row"], None)
    dw = (got * dy[:, None, :]).sum(2)
    live = (s["src"] >= 0)[:, None]
    entry = s["src"].clamp(min=0).long()
    drows = torch.where(live, s["w"].reshape(-1)[entry][:, None] * dy[entry // K], 0.0).to(x.dtype)
    dx, _ = _plain_back(drows, s["row"], None)
    return drows, dw, dx.to(x.dtype)


def _plain_int4(s):
    c = s["case"]
    q = s["wq"]
    E, n, _ = q.shape
    w = torch.stack([q & 15, q >> 4], dim=-1).reshape(E, n, c["Kd"] // c["group"], c["group"]).float()
    w -= 8.0 if s["zeros"] is None else s["zeros"].float()[..., None]
    w *= s["scales"].float()[..., None]
    src = s["src"].long()
    r = torch.arange(s["rows"], device=q.device)
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    slot = r - s["offsets"].long()[e]
    xp = torch.zeros(E, c["T"], c["Kd"], device=q.device)
    xp[e, slot] = s["x"][src // c["K"]].float()
    out = torch.bmm(xp, w.reshape(E, n, c["Kd"]).transpose(1, 2))[e, slot]
    if c["swiglu"]:
        a, b = out[:, :c["N"]], out[:, c["N"]:]
        out = a * torch.sigmoid(a) * b
    return out.to(s["x"].dtype)


# -------------------------------------------------------------------- runs


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"gate": _plain_gate, "sort": _plain_sort, "int4": _plain_int4}[c["kind"]](s)
    from combine_moedc_layout_gb300 import moedc
    out = s["out"]
    if c["kind"] == "gate":
        flags = moedc.GATE_SIGMOID if c["score"] == "sigmoid" else moedc.GATE_SOFTMAX
        if c["normalize"]:
            flags |= moedc.GATE_NORMALIZE
        out["gate"] = moedc.gate(s["logits"], c["K"], bias=s["bias"], flags=flags, out=out.get("gate"))
        if not c["grad"]:
            return out["gate"]
        out["dl"] = moedc.gate_grad(s["logits"], out["gate"][0], s["dw"], bias=s["bias"],
                                    flags=flags, out=out.get("dl"))
        return *out["gate"], out["dl"]
    if c["kind"] == "sort":
        if not c["grad"]:
            out["sort"] = m = moedc.sort(s["x"], s["idx"], c["E"], align=c["align"],
                                         status=s["status"], out=out.get("sort"))
            out["y"] = moedc.unsort(s["expert_out"], m.row, s["w"], out=out.get("y"))
            return m.rows, m.row, m.src, m.offsets, m.counts, out["y"]
        out["drows"] = moedc.unsort_grad(s["x"], s["expert_out"], s["row"], s["src"], s["w"],
                                         out=out.get("drows"))
        drows, dw = out["drows"]
        out["dx"] = moedc.sort_grad(drows, s["row"], out=out.get("dx"))
        return drows, dw, out["dx"]
    out["mv"] = moedc.matvec_int4(s["x"], s["wq"], s["scales"], zeros=s["zeros"],
                                  offsets=s["offsets"], counts=s["counts"], src=s["src"],
                                  top_k=c["K"], swiglu=c["swiglu"], status=s["status"],
                                  out=out.get("mv"))
    return out["mv"]


# -------------------------------------------------------------- 64-bit form


def _exact_gate(s):
    c = s["case"]
    K = c["K"]
    logits = s["logits"].double()
    key = (s["logits"].float() + (s["bias"] if c["bias"] else 0.0)).double()   # one 32-bit sum
    can = ~(torch.isneginf(logits) | torch.isnan(logits))
    left = torch.where(can, key, torch.full_like(key, -float("inf")))
    picks, alive = [], []
    columns = torch.arange(c["E"], device=key.device)
    for _ in range(K):
        best = left.amax(1, keepdim=True)
        pick = torch.where(left == best, columns, c["E"]).amin(1, keepdim=True)
        alive.append(best > -float("inf"))
        picks.append(pick)
        left = left.masked_fill(columns == pick, -float("inf"))
    idx, live = torch.cat(picks, 1), torch.cat(alive, 1)
    chosen = logits.gather(1, idx)
    hit = torch.zeros_like(logits).scatter_add_(1, idx, live.double()) > 0     # chosen experts
    if c["score"] == "sigmoid":
        f = 1.0 / (1.0 + torch.exp(-logits))
        f = torch.where(can, f, 0.0)
        norm = torch.where(hit, f, 0.0).sum(1, keepdim=True) if c["normalize"] else torch.ones_like(f[:, :1])
    else:
        field = hit if c["normalize"] else can
        shift = torch.where(can, logits, -1e300).amax(1, keepdim=True)
        f = torch.where(can, torch.exp(logits - shift), 0.0)
        norm = torch.where(field, f, 0.0).sum(1, keepdim=True)
    p = torch.where(norm > 0, f / norm.clamp(min=1e-300), 0.0)
    w = torch.where(live, p.gather(1, idx), 0.0)
    if not c["grad"]:
        return None, w
    d = torch.zeros_like(logits).scatter_add_(1, idx, torch.where(live, s["dw"].double(), 0.0))
    mean = (torch.where(hit, p, 0.0) * d).sum(1, keepdim=True)
    if c["score"] == "sigmoid":
        slope = torch.where(hit, f * (1.0 - f), 0.0)
        dl = torch.where(norm > 0, slope / norm * (d - mean), 0.0) if c["normalize"] else slope * d
    else:
        dl = torch.where(field, p * (d - mean), 0.0)
    return None, w, dl


def _exact_sort(s):
    c = s["case"]
    T, K = c["T"], c["K"]
    eo, x, w = s["expert_out"].double(), s["x"].double(), s["w"].double()
    if not c["grad"]:
        rows = torch.zeros(s["rows"], c["H"], dtype=torch.float64, device=x.device)
        y = torch.zeros_like(x)
        e = s["idx"].cpu().reshape(-1).tolist()
        groups = [[] for _ in range(c["E"])]
        for i, v in enumerate(e):
            if v >= 0:
                groups[v].append(i)
        at, entries = [], []
        base = 0
        for group in groups:
            entries += group
            at += range(base, base + len(group))
            base += -(-len(group) // c["align"]) * c["align"]
        entries = torch.tensor(entries, dtype=torch.int64, device=x.device)
        at = torch.tensor(at, dtype=torch.int64, device=x.device)
        rows[at] = x[entries // K]
        y.index_add_(0, entries // K, eo[at] * w.reshape(-1)[entries][:, None])
        return rows, None, None, None, None, y
    drows = torch.zeros(s["rows"], c["H"], dtype=torch.float64, device=x.device)
    dw = torch.zeros(T, K, dtype=torch.float64, device=x.device)
    dx = torch.zeros_like(x)
    for k in range(K):
        t = (s["row"][:, k] >= 0).nonzero()[:, 0]
        at = s["row"][t, k].long()
        drows[at] = w[t, k][:, None] * x[t]
        dw[t, k] = (eo[at] * x[t]).sum(1)
        dx[t] += (w[t, k][:, None] * x[t]).to(s["x"].dtype).double()   # of the rounded drows
    return drows, dw, dx


def _exact_int4(s):
    c = s["case"]
    Kd, g = c["Kd"], c["group"]
    if c["T"] * c["K"] * c["N"] * (2 if c["swiglu"] else 1) * Kd > 4e10:
        return None
    x = s["x"].double()
    out = torch.zeros(s["rows"], c["N"], dtype=torch.float64, device=x.device)
    starts, counts = s["offsets"].tolist(), s["counts"].tolist()
    for e in range(c["E"]):
        if not counts[e]:
            continue
        here = slice(starts[e], starts[e] + counts[e])
        q = s["wq"][e].long()
        w = torch.empty(q.shape[0], Kd, dtype=torch.float64, device=x.device)
        w[:, 0::2] = (q % 16).double()
        w[:, 1::2] = (q // 16).double()
        zero = 8.0 if s["zeros"] is None else s["zeros"][e].double().repeat_interleave(g, 1)
        w = (w - zero) * s["scales"][e].double().repeat_interleave(g, 1)
        v = x[s["src"][here].long() // c["K"]] @ w.T
        if c["swiglu"]:
            v = v[:, :c["N"]] / (1.0 + torch.exp(-v[:, :c["N"]])) * v[:, c["N"]:]
        out[here] = v
    return out


def exact(case, seed):
    s = prepare(case, seed)
    return {"gate": _exact_gate, "sort": _exact_sort, "int4": _exact_int4}[case["kind"]](s)
