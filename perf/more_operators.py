"""The operators of a gated channel mixer, as measurable cases.

Three groups of operators:

* root-mean-square norm with the residual's addition: forward (``rms_fwd``),
  forward with an output in 8 bits and a scale for each row (``rms_q8``),
  backward (``rms_bwd``);
* the gated product act(x Wg^T) * (x Wu^T): forward (``gated_fwd``), forward
  on 8-bit operands (``gated_q8``), backward (``gated_bwd``);
* the global norm of many gradients, and clipping by it (``clip``).

``own = False`` computes them in their plain form (elementary torch operations
in float32, rounded once at the end); ``own = True`` calls the framework's
operators.  ``exact`` evaluates the definitions in float64.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-6
CLIP_EPS = 1e-6
E4M3_MOST = 448.0


def rms(op, M, C, dtype, residual=True):
    return {"op": op, "M": M, "C": C, "dtype": dtype, "residual": residual}


def gated(op, M, C, H, dtype, act):
    return {"op": op, "M": M, "C": C, "H": H, "dtype": dtype, "act": act}


def clip(blocks, C, H, dtype, clips):
    return {"op": "clip", "blocks": blocks, "C": C, "H": H, "dtype": dtype, "clips": clips}


def listed():
    return [
        # one image of 37 x 53 pixels and 90 channels: a call's latency, rows that no vector access divides evenly
        dict(rms("rms_fwd", 1961, 90, "f32"), name="rms_fwd one image"),
        # the first stage's training batch, 64 images of 56 x 56: short rows, many of them
        dict(rms("rms_fwd", 200704, 96, "bf16"), name="rms_fwd stage 1"),
        # 8-bit inference of a wide mixer, the norm in front of the matrices
        dict(rms("rms_q8", 16384, 2048, "f16"), name="rms_q8 wide"),
        # the second stage's training batch at twice the resolution
        dict(rms("rms_bwd", 200704, 192, "bf16"), name="rms_bwd 56x56"),
        # one pixel's channels (a pooled image): bound by reading the weights
        dict(gated("gated_fwd", 1, 768, 2048, "f16", "silu"), name="gated_fwd one row"),
        # the first stage's training batch: a short contraction, bound by memory
        dict(gated("gated_fwd", 200704, 96, 256, "bf16", "gelu"), name="gated_fwd stage 1"),
        # 37 x 49 pixels, widths that no tile divides, in float32
        dict(gated("gated_fwd", 1813, 90, 237, "f32", "silu"), name="gated_fwd odd sizes"),
        # 8-bit inference of a wide mixer, bound by the matrix products
        dict(gated("gated_q8", 8192, 2048, 5632, "bf16", "silu"), name="gated_q8 wide"),
        # the third stage's training batch, 128 images of 14 x 14
        dict(gated("gated_bwd", 25088, 384, 1024, "bf16", "gelu"), name="gated_bwd stage 3"),
        # a wide mixer in training: bound by the matrix products
        dict(gated("gated_bwd", 8192, 2048, 5632, "bf16", "silu"), name="gated_bwd wide"),
        # the gradients of nine blocks of the third stage: many tensors, most of them small
        dict(clip(9, 384, 1024, "f32", True), name="clip stage 3"),
        # four wide blocks at a step that stays below the limit: the norm alone
        dict(clip(4, 2048, 5632, "bf16", False), name="clip wide"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rms_fwd", "rms_q8", "rms_bwd", "gated_fwd", "gated_fwd", "gated_q8", "gated_bwd", "gated_bwd", "clip"))
    dtype = rng.choice(("f32", "f16", "bf16"))
    if op.startswith("rms"):
        C = _log(rng, 24, 6000)
        M = max(1, min(_log(rng, 1, 300_000), 48_000_000 // C))
        return rms(op, M, C, dtype, residual=rng.random() < 0.7)
    if op == "clip":
        C = _log(rng, 32, 2000)
        H = int(C * rng.uniform(1.5, 4.0))
        blocks = max(1, min(_log(rng, 1, 40), 150_000_000 // (3 * C * H + 300 * C)))
        return clip(blocks, C, H, dtype, rng.random() < 0.6)
    C, H = _log(rng, 32, 3000), _log(rng, 48, 6000)
    if op == "gated_q8":
        C, dtype = max(32, C // 16 * 16), rng.choice(("f16", "bf16"))
    # products of at most those of the widest listed case; six of them stand in the place of one of float32
    most = 94_000_000_000 // (6 if dtype == "f32" else 1)
    M = max(1, min(_log(rng, 1, 250_000), most // (C * H), 300_000_000 // (C + 2 * H)))
    return gated(op, M, C, H, dtype, rng.choice(("none", "silu", "gelu")))


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _quantised(x):
    """e4m3 values of the rows, and each row's scale."""
    amax = x.abs().amax(dim=-1).clamp_min(1e-30)
    return (x * (E4M3_MOST / amax)[..., None]).clamp(-E4M3_MOST, E4M3_MOST).to(torch.float8_e4m3fn), amax / E4M3_MOST


def _block_shapes(C, H, k=5, levels=3):
    """A block's parameters: the wavelet layer's, the norm's, the three matrices."""
    return [(C, k, k), (C,), (C,), (levels, 4 * C, k, k), (levels, 4 * C), (C,), (H, C), (H, C), (C, H)]


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    s = dict(case)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    if case["op"].startswith("rms"):
        M, C = case["M"], case["C"]
        # a residual stream whose channels have a size of their own, and rows too
        size = torch.exp(0.5 * randn(C)) * torch.exp(0.3 * randn(M, 1))
        s["weight"] = 1.0 + 0.1 * randn(C)
        if case["op"] == "rms_bwd":
            s["total"] = (randn(M, C) * size).to(dtype)
            s["rstd"] = torch.rsqrt(s["total"].float().square().mean(dim=1) + EPS)
            s["dy"] = randn(M, C).to(dtype)
            s["dtotal"] = randn(M, C).to(dtype) if case["residual"] else None
            return s
        s["x"] = (randn(M, C) * size).to(dtype)
        s["r"] = randn(M, C).to(dtype) if case["residual"] else None
        return s
    if case["op"] == "clip":
        shapes = _block_shapes(case["C"], case["H"]) * case["blocks"]
        sizes = [math.prod(q) for q in shapes]
        s["flat"] = randn(sum(sizes)) * 1e-2
        at = 0
        for n in sizes:  # each parameter's gradient has a size of its own
            s["flat"][at:at + n] *= 0.25 + (at % 7) / 4
            at += n
        s["flat"] = s["flat"].to(dtype)
        s["grads"] = [t.view(q) for t, q in zip(s["flat"].split(sizes), shapes)]
        # limits far below the norm, or above it, as most steps of a training have it
        s["limit"] = 0.5 if case["clips"] else 1e4
        return s
    M, C, H = case["M"], case["C"], case["H"]
    x = randn(M, C)
    gate, up = randn(H, C) * (1.5 / math.sqrt(C)), randn(H, C) * (1.0 / math.sqrt(C))
    if case["op"] == "gated_q8":
        s["x"], s["x_scale"] = _quantised(x)
        s["gate"], s["gate_scale"] = _quantised(gate)
        s["up"], s["up_scale"] = _quantised(up)
        return s
    s["x"], s["gate"], s["up"] = x.to(dtype), gate.to(dtype), up.to(dtype)
    if case["op"] == "gated_bwd":
        s["dh"] = randn(M, H).to(dtype)
    return s


_ops = None


def _framework():
    global _ops
    if _ops is None:
        from memory_bound_cnn_wtconv2d_gb300 import mixerops
        _ops = mixerops
    return _ops


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    f = _framework()
    op = s["op"]
    if op == "rms_fwd":
        y, total, rstd = f.wtconv_rms_norm_fwd(s["x"], s["weight"], residual=s["r"], eps=EPS)
        return {"y": y, "total": total, "rstd": rstd}
    if op == "rms_q8":
        q, scale, total = f.wtconv_rms_norm_q8(s["x"], s["weight"], residual=s["r"], eps=EPS)
        return {"q": q, "scale": scale, "total": total}
    if op == "rms_bwd":
        dx, dweight = f.wtconv_rms_norm_bwd(s["dy"], s["total"], s["rstd"], s["weight"], dtotal=s["dtotal"])
        return {"dx": dx, "dweight": dweight}
    if op == "gated_fwd":
        return {"h": f.wtconv_gated_fwd(s["x"], s["gate"], s["up"], activation=s["act"])}
    if op == "gated_q8":
        return {"h": f.wtconv_gated_q8(s["x"], s["x_scale"], s["gate"], s["gate_scale"], s["up"], s["up_scale"],
                                       activation=s["act"], dtype=DTYPES[s["dtype"]])}
    if op == "gated_bwd":
        dx, dgate, dup = f.wtconv_gated_bwd(s["dh"], s["x"], s["gate"], s["up"], activation=s["act"])
        return {"dx": dx, "dgate": dgate, "dup": dup}
    limit = _limit(s)
    norm = f.wtconv_clip_grads(s["grads"], limit, eps=CLIP_EPS)
    return {"norm": norm, "flat": s["flat"]}


def _limit(s):
    """This pass's limit: a clipping pass lowers it a little, so that the next one clips as well."""
    limit = s["limit"]
    if s["clips"]:
        s["limit"] = limit * 0.9999
    return limit


def _plain_act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    return z


def _plain_act_grad(z, act):
    if act == "silu":
        sig = 1 / (1 + torch.exp(-z))
        return sig * (1 + z * (1 - sig))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    return torch.ones_like(z)


def _run_plain(s):
    op = s["op"]
    if op in ("rms_fwd", "rms_q8"):
        t = s["x"].float()
        if s["r"] is not None:
            t = t + s["r"].float()
        rstd = 1 / torch.sqrt(t.square().mean(dim=1) + EPS)
        y = t * rstd[:, None] * s["weight"]
        total = t.to(s["x"].dtype)
        if op == "rms_fwd":
            return {"y": y.to(s["x"].dtype), "total": total, "rstd": rstd}
        q, scale = _quantised(y)
        return {"q": q, "scale": scale, "total": total}
    if op == "rms_bwd":
        xhat = s["total"].float() * s["rstd"][:, None]
        dy = s["dy"].float()
        dweight = (dy * xhat).sum(dim=0)
        dxhat = dy * s["weight"]
        dx = s["rstd"][:, None] * (dxhat - xhat * (dxhat * xhat).mean(dim=1, keepdim=True))
        if s["dtotal"] is not None:
            dx = dx + s["dtotal"].float()
        return {"dx": dx.to(s["dy"].dtype), "dweight": dweight}
    if op == "clip":
        limit = _limit(s)
        norm = torch.stack([t.float().square().sum() for t in s["grads"]]).sum().sqrt()
        factor = torch.clamp(limit / (norm + CLIP_EPS), max=1.0)
        s["flat"].copy_(s["flat"].float() * factor)
        return {"norm": norm, "flat": s["flat"]}
    x, gate, up = s["x"].float(), s["gate"].float(), s["up"].float()
    if op == "gated_q8":
        x, gate, up = x * s["x_scale"][:, None], gate * s["gate_scale"][:, None], up * s["up_scale"][:, None]
    g, u = x @ gate.T, x @ up.T
    if op != "gated_bwd":
        return {"h": (_plain_act(g, s["act"]) * u).to(DTYPES[s["dtype"]])}
    dh = s["dh"].float()
    dg, du = dh * u * _plain_act_grad(g, s["act"]), dh * _plain_act(g, s["act"])
    dtype = s["x"].dtype
    return {"dx": (dg @ gate + du @ up).to(dtype), "dgate": (dg.T @ x).to(dtype), "dup": (du.T @ x).to(dtype)}


def work(case):
    e = ESIZE[case["dtype"]]
    if case["op"].startswith("rms"):
        M, C = case["M"], case["C"]
        inputs = 2 if case["residual"] else 1
        if case["op"] == "rms_bwd":  # dy, total and dtotal read, dx written; rstd and the weight read, its gradient written
            return {"bytes": (inputs + 2) * M * C * e + 4 * (M + 2 * C), "flops": 12 * M * C}
        # x and the residual read, their sum written; y written, in 8 bits with a scale a row or with rstd
        out = M * C * ((e if case["op"] == "rms_fwd" else 1) + (e if case["residual"] else 0)) + 4 * M
        return {"bytes": inputs * M * C * e + out + 4 * C, "flops": 6 * M * C}
    if case["op"] == "clip":
        n = case["blocks"] * sum(math.prod(q) for q in _block_shapes(case["C"], case["H"]))
        return {"bytes": n * e * (2 if case["clips"] else 1) + 4, "flops": 3 * n}
    M, C, H = case["M"], case["C"], case["H"]
    if case["op"] == "gated_fwd":  # x and both matrices read, h written
        return {"bytes": (M * C + 2 * H * C + M * H) * e, "flops": 4 * M * H * C + 8 * M * H}
    if case["op"] == "gated_q8":
        return {"bytes": M * C + 2 * H * C + M * H * e + 4 * (M + 2 * H), "flops": 4 * M * H * C + 8 * M * H}
    # dh, x and both matrices read, their three gradients written; g and u are made again from x
    return {"bytes": (M * H + 2 * M * C + 4 * H * C) * e, "flops": 12 * M * H * C + 20 * M * H}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rms_fwd", "rms_q8"):
        t = s["x"].double() + (0 if s["r"] is None else s["r"].double())
        rstd = (torch.linalg.vector_norm(t, dim=1) ** 2 / case["C"] + EPS) ** -0.5
        y = torch.einsum("mc,m,c->mc", t, rstd, s["weight"].double())
        if op == "rms_fwd":
            return {"y": y, "total": t, "rstd": rstd}
        scale = y.abs().max(dim=1).values / E4M3_MOST
        return {"q": y / scale[:, None], "scale": scale, "total": t}
    if op == "rms_bwd":
        t, dy, w = s["total"].double(), s["dy"].double(), s["weight"].double()
        rstd = s["rstd"].double()
        along = torch.einsum("mc,mc,c,m->m", dy, t, w, rstd) / case["C"]
        dx = rstd[:, None] * (dy * w) - (rstd ** 2 * along)[:, None] * t
        if s["dtotal"] is not None:
            dx += s["dtotal"].double()
        return {"dx": dx, "dweight": torch.einsum("mc,mc,m->c", dy, t, rstd)}
    if op == "clip":
        flat = s["flat"].double()
        norm = torch.linalg.vector_norm(flat)
        return {"norm": norm, "flat": flat * min(1.0, s["limit"] / (float(norm) + CLIP_EPS))}
    x, gate, up = s["x"].double(), s["gate"].double(), s["up"].double()
    if op == "gated_q8":
        x *= s["x_scale"].double()[:, None]
        gate *= s["gate_scale"].double()[:, None]
        up *= s["up_scale"].double()[:, None]
    F = torch.nn.functional
    act = {"none": lambda z: z, "silu": F.silu, "gelu": F.gelu}[case["act"]]
    if op != "gated_bwd":
        return {"h": act(F.linear(x, gate)) * F.linear(x, up)}
    # the products' gradients by torch's own derivation, in float64
    leaves = [t.requires_grad_() for t in (x, gate, up)]
    h = act(F.linear(x, gate)) * F.linear(x, up)
    dx, dgate, dup = torch.autograd.grad(h, leaves, s["dh"].double())
    return {"dx": dx, "dgate": dgate, "dup": dup}
