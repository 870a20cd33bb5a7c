"""The training operators around the wavelet layer, as measurable cases.

Two groups of operators, four entry points:

* group norm with an activation on channels-last activations, forward and
  backward (``gn_fwd``, ``gn_bwd``);
* the orthogonalisation of a matrix update by Newton-Schulz products
  (``orth``) and the optimiser step built on it (``muon``).

``own = False`` computes them in their plain form (elementary torch operations
in float32, rounded once at the end); ``own = True`` calls the framework's
operators.  ``exact`` evaluates the definitions in float64.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ESIZE = {"f32": 4, "f16": 2, "bf16": 2}
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
GN_EPS = 1e-5
NS_EPS = 1e-7
LR, MOMENTUM, DECAY = 0.02, 0.95, 0.01


def gn(op, N, H, W, C, G, dtype, act):
    return {"op": op, "N": N, "H": H, "W": W, "C": C, "G": G, "dtype": dtype, "act": act}


def matrix(op, count, m, n, dtype):
    return {"op": op, "count": count, "m": m, "n": n, "dtype": dtype}


def listed():
    return [
        # one image at the last stage's resolution (inference of one picture): a call's latency
        dict(gn("gn_fwd", 1, 7, 7, 768, 32, "bf16", "silu"), name="gn_fwd one image 7x7"),
        # the first stage's training batch; groups of three channels, narrower than any vector load
        dict(gn("gn_fwd", 64, 56, 56, 96, 32, "bf16", "gelu"), name="gn_fwd stage 1"),
        # the stem resolution of a 224 x 224 image in float32: samples that no group of SMs holds
        dict(gn("gn_fwd", 16, 224, 224, 64, 8, "f32", "silu"), name="gn_fwd 224x224"),
        # odd image sides, channels and groups that no power of two divides
        dict(gn("gn_bwd", 5, 37, 53, 90, 6, "f32", "gelu"), name="gn_bwd odd sizes"),
        # the third stage's training batch: many small samples
        dict(gn("gn_bwd", 128, 14, 14, 384, 32, "f16", "gelu"), name="gn_bwd stage 3"),
        # large maps in training
        dict(gn("gn_bwd", 32, 128, 128, 96, 16, "bf16", "silu"), name="gn_bwd 128x128"),
        # the first stage's three expanding pointwise matrices: the smallest update
        dict(matrix("orth", 3, 384, 96, "bf16"), name="orth stage 1"),
        # the third stage's nine blocks at once
        dict(matrix("orth", 9, 1536, 384, "bf16"), name="orth stage 3"),
        # sizes that no tile divides, in float32
        dict(matrix("orth", 2, 333, 1201, "f32"), name="orth odd sizes"),
        # one large square matrix: bound by the matrix products
        dict(matrix("orth", 1, 4096, 4096, "bf16"), name="orth 4096"),
        # the optimiser's step on the second stage's contracting matrices, float32 parameters
        dict(matrix("muon", 3, 192, 768, "f32"), name="muon stage 2"),
        # the optimiser's step on wide layers
        dict(matrix("muon", 4, 2048, 1024, "f32"), name="muon 2048x1024"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("gn_fwd", "gn_bwd", "orth", "muon"))
    if op in ("gn_fwd", "gn_bwd"):
        G = rng.choice((1, 2, 3, 4, 6, 8, 16, 32))
        C = G * max(1, _log(rng, 32, 768) // G)
        H, W = _log(rng, 5, 224), _log(rng, 5, 224)
        N = max(1, min(_log(rng, 1, 128), 48_000_000 // (H * W * C)))
        return gn(op, N, H, W, C, G, rng.choice(("f32", "f16", "bf16")), rng.choice(("none", "silu", "gelu")))
    m, n = _log(rng, 48, 4000), _log(rng, 48, 4000)
    m, n = m + (m == 3072), n + (n == 3072)
    # the products of a drawn stack cost no more than those of a 2048 x 1024 stack of four
    each = min(m, n) ** 2 * max(m, n)
    count = max(1, min(rng.randint(1, 12), 12_000_000_000 // each))
    return matrix(op, count, m, n, rng.choice(("f32", "f16", "bf16")))


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _update(g, count, m, n, dtype):
    """Gradient-like matrices: a decaying spectrum of a few strong directions over noise."""
    k = max(1, min(m, n) // 8)
    decay = torch.logspace(0, -2, k, device="cuda")
    u = torch.randn(count, m, k, generator=g, device="cuda") * decay
    v = torch.randn(count, k, n, generator=g, device="cuda")
    noise = torch.randn(count, m, n, generator=g, device="cuda")
    return ((torch.bmm(u, v) + 0.5 * noise) * 1e-3).to(dtype)


def prepare(case, seed):
    g = _generator(seed)
    dtype = DTYPES[case["dtype"]]
    s = dict(case)
    if case["op"] in ("gn_fwd", "gn_bwd"):
        N, H, W, C, G = (case[k] for k in ("N", "H", "W", "C", "G"))
        # activations with a mean and a spread of their own for each channel, as a convolution leaves them
        shift = 0.5 * torch.randn(C, generator=g, device="cuda") + 0.25
        spread = 0.5 + torch.rand(C, generator=g, device="cuda")
        s["x"] = (torch.randn(N, H, W, C, generator=g, device="cuda") * spread + shift).to(dtype)
        s["weight"] = 1.0 + 0.1 * torch.randn(C, generator=g, device="cuda")
        s["bias"] = 0.1 * torch.randn(C, generator=g, device="cuda")
        if case["op"] == "gn_bwd":
            s["dy"] = torch.randn(N, H, W, C, generator=g, device="cuda").to(dtype)
            # what the forward pass kept
            xg = s["x"].float().view(N, H * W, G, C // G)
            s["mean"] = xg.mean(dim=(1, 3))
            s["rstd"] = torch.rsqrt((xg - s["mean"][:, None, :, None]).square().mean(dim=(1, 3)) + GN_EPS)
        return s
    count, m, n = case["count"], case["m"], case["n"]
    s["grad"] = _update(g, count, m, n, dtype)
    if case["op"] == "muon":
        s["weight"] = (torch.randn(count, m, n, generator=g, device="cuda") / math.sqrt(n)).to(dtype)
        s["momentum"] = 0.5 * s["grad"].float() + 0.5 * _update(g, count, m, n, torch.float32)
        s["scale"] = math.sqrt(max(1.0, m / n))
    return s


_ops = None


def _framework():
    global _ops
    if _ops is None:
        from memory_bound_cnn_wtconv2d_gb300 import blockops
        _ops = blockops
    return _ops


def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    f = _framework()
    op = s["op"]
    if op == "gn_fwd":
        y, mean, rstd = f.wtconv_gn_act_fwd(s["x"], s["G"], s["weight"], s["bias"], eps=GN_EPS, activation=s["act"])
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "gn_bwd":
        dx, dweight, dbias = f.wtconv_gn_act_bwd(s["dy"], s["x"], s["mean"], s["rstd"], s["G"], s["weight"],
                                                 s["bias"], activation=s["act"])
        return {"dx": dx, "dweight": dweight, "dbias": dbias}
    if op == "orth":
        return {"out": f.wtconv_orthogonalize(s["grad"], steps=STEPS, coefficients=COEFFICIENTS, eps=NS_EPS)}
    f.wtconv_muon_step(s["weight"], s["grad"], s["momentum"], lr=LR, momentum=MOMENTUM, nesterov=True,
                       weight_decay=DECAY, scale=s["scale"], steps=STEPS, coefficients=COEFFICIENTS, eps=NS_EPS)
    return {"weight": s["weight"], "momentum": s["momentum"]}


def _plain_newton_schulz(g):
    """a X + (b A + c A A) X with A = X X^T, five times, on the wide orientation."""
    a, b, c = COEFFICIENTS
    x = g / (g.square().sum(dim=(1, 2), keepdim=True).sqrt() + NS_EPS)
    tall = x.shape[1] > x.shape[2]
    if tall:
        x = x.transpose(1, 2)
    for _ in range(STEPS):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return x.transpose(1, 2) if tall else x


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
    if op in ("gn_fwd", "gn_bwd"):
        N, H, W, C, G = (s[k] for k in ("N", "H", "W", "C", "G"))
        xg = s["x"].float().view(N, H * W, G, C // G)
        w, b = s["weight"].view(G, C // G), s["bias"].view(G, C // G)
    if op == "gn_fwd":
        mean = xg.mean(dim=(1, 3), keepdim=True)
        centred = xg - mean
        rstd = 1 / torch.sqrt(centred.square().mean(dim=(1, 3), keepdim=True) + GN_EPS)
        y = _plain_act(centred * rstd * w + b, s["act"])
        return {"y": y.to(s["x"].dtype).view(N, H, W, C), "mean": mean.view(N, G), "rstd": rstd.view(N, G)}
    if op == "gn_bwd":
        rstd = s["rstd"][:, None, :, None]
        xhat = (xg - s["mean"][:, None, :, None]) * rstd
        dz = s["dy"].float().view(N, H * W, G, C // G) * _plain_act_grad(xhat * w + b, s["act"])
        dweight, dbias = (dz * xhat).sum(dim=(0, 1)), dz.sum(dim=(0, 1))
        dxhat = dz * w
        dx = rstd * (dxhat - dxhat.mean(dim=(1, 3), keepdim=True) - xhat * (dxhat * xhat).mean(dim=(1, 3), keepdim=True))
        return {"dx": dx.to(s["x"].dtype).view(N, H, W, C), "dweight": dweight.view(C), "dbias": dbias.view(C)}
    grad = s["grad"].float()
    if op == "orth":
        return {"out": _plain_newton_schulz(grad).to(s["grad"].dtype).contiguous()}
    s["momentum"].mul_(MOMENTUM).add_(grad, alpha=1 - MOMENTUM)
    direction = _plain_newton_schulz(MOMENTUM * s["momentum"] + (1 - MOMENTUM) * grad)
    s["weight"].copy_((1 - LR * DECAY) * s["weight"].float() - LR * s["scale"] * direction)
    return {"weight": s["weight"], "momentum": s["momentum"]}


def work(case):
    e = ESIZE[case["dtype"]]
    if case["op"] in ("gn_fwd", "gn_bwd"):
        N, C, G = case["N"], case["C"], case["G"]
        numel = N * case["H"] * case["W"] * C
        if case["op"] == "gn_fwd":  # x read, y written; weight and bias read; mean and rstd written
            return {"bytes": 2 * numel * e + 4 * (2 * C + 2 * N * G), "flops": 12 * numel}
        # x and dy read, dx written; weight, bias, mean, rstd read; two gradients written
        return {"bytes": 3 * numel * e + 4 * (4 * C + 2 * N * G), "flops": 30 * numel}
    count, r, c = case["count"], min(case["m"], case["n"]), max(case["m"], case["n"])
    # the symmetric products X X^T and A A need one triangle each
    flops = count * STEPS * (r * (r + 1) * c + r * (r + 1) * r + 2 * r * r * c)
    if case["op"] == "orth":  # the matrix read, the result written
        return {"bytes": 2 * count * r * c * e, "flops": flops}
    return {"bytes": count * r * c * (3 * e + 8), "flops": flops}  # weight and momentum read and written, gradient read


def _exact_orthogonal(g):
    """The same polynomial through the Gram matrix alone: X_k = Q_k X_0 with Q_k a polynomial of X_0 X_0^T."""
    a, b, c = COEFFICIENTS
    x = g / (torch.linalg.matrix_norm(g)[:, None, None] + NS_EPS)
    wide = x.shape[2] >= x.shape[1]
    s = x @ x.mT if wide else x.mT @ x
    eye = torch.eye(s.shape[1], dtype=torch.float64, device=s.device)
    q = eye.expand_as(s)
    for _ in range(STEPS):
        p = a * eye + s @ (b * eye + c * s)
        q = p @ q
        s = p @ s @ p
    return q @ x if wide else x @ q


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("gn_fwd", "gn_bwd"):
        N, H, W, C, G = (case[k] for k in ("N", "H", "W", "C", "G"))
        x = s["x"].double().reshape(N, H * W, C)
        w, b = s["weight"].double(), s["bias"].double()
        over = lambda t: t.view(N, G, 1).expand(N, G, C // G).reshape(N, 1, C)  # noqa: E731
        if op == "gn_fwd":
            flat = x.view(N, H * W, G, C // G).transpose(1, 2).reshape(N, G, -1)
            var, mean = torch.var_mean(flat, dim=2, correction=0)
            del flat
            rstd = (var + GN_EPS) ** -0.5
        else:
            mean, rstd = s["mean"].double(), s["rstd"].double()
        xhat = (x - over(mean)) * over(rstd)
        z = torch.addcmul(b, xhat, w)
        if op == "gn_fwd":
            y = {"none": lambda t: t, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[case["act"]](z)
            return {"y": y.view(N, H, W, C), "mean": mean, "rstd": rstd}
        dz = s["dy"].double().view(N, H * W, C)
        if case["act"] == "silu":
            sig = torch.sigmoid(z)
            dz = dz * (sig + z * sig * torch.sigmoid(-z))
        elif case["act"] == "gelu":
            dz = dz * (torch.special.ndtr(z) + z * torch.exp(-0.5 * z ** 2) / math.sqrt(2 * math.pi))
        per_channel = torch.stack((dz.sum(1), (dz * xhat).sum(1)))  # [2, N, C]
        sums = (per_channel * w).view(2, N, G, C // G).sum(3) / (H * W * (C // G))
        dx = over(rstd) * (dz * w - over(sums[0].contiguous()) - xhat * over(sums[1].contiguous()))
        return {"dx": dx.view(N, H, W, C), "dweight": per_channel[1].sum(0), "dbias": per_channel[0].sum(0)}
    grad = s["grad"].double()
    if op == "orth":
        return {"out": _exact_orthogonal(grad)}
    momentum = s["momentum"].double() * MOMENTUM + grad * (1 - MOMENTUM)
    direction = _exact_orthogonal(momentum * MOMENTUM + grad * (1 - MOMENTUM))
    return {"weight": s["weight"].double() * (1 - LR * DECAY) - direction * (LR * s["scale"]), "momentum": momentum}
