"""What is measured of the operators on either side of the head: the root-mean-square norm with the
residual's addition, forward, backward and with its output in 8 bits, and the orthogonalising of
updates by Newton-Schulz products.

Each operator has two forms. The plain one is written in elementary torch operations, in 32 bits;
the other is the package's own. `run` takes the one that `own` names.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-6
# one triple a step of x <- a x + (b (x x^T) + c (x x^T)^2) x: it lifts small singular values
# quickly and leaves all of them near 1
STEPS = ((3.4445, -4.7750, 2.0315),) * 5


def _package():
    import linear_cross_entropy_vocab_gb300 as package
    return package


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the norm before the head in one decoding step of four beams, where only latency counts
        {"name": "norm_step_bf16", "op": "norm", "n": 4, "h": 4096, "dtype": "bf16", "residual": "same", "weight": True},
        # the same for a batch of prompts
        {"name": "norm_prompt_f16", "op": "norm", "n": 16384, "h": 3584, "dtype": "f16", "residual": "same", "weight": True},
        # a training step's norm over the long batch: both directions, gradients of the input, the residual and the weight
        {"name": "norm_train_bf16", "op": "train", "n": 32768, "h": 4096, "dtype": "bf16", "residual": "same", "weight": True},
        # a residual stream that is kept in 32 bits beside 16-bit layers
        {"name": "norm_train_wide_bf16", "op": "train", "n": 4096, "h": 2048, "dtype": "bf16", "residual": "f32", "weight": True},
        # a model without powers of two: odd rows, nothing aligned, no residual
        {"name": "norm_train_odd_f32", "op": "train", "n": 4099, "h": 2049, "dtype": "f32", "residual": "none", "weight": True},
        # what the 8-bit head reads in a decoding step of eight beams
        {"name": "quant_step_bf16", "op": "quant", "n": 8, "h": 4096, "dtype": "bf16", "residual": "same", "weight": True},
        # the same where every position of a batch of prompts is scored
        {"name": "quant_prompt_bf16", "op": "quant", "n": 8192, "h": 4096, "dtype": "bf16", "residual": "same", "weight": True},
        # one matrix of a small test model, from 32-bit momentum: latency alone
        {"name": "ortho_small_f32", "op": "ortho", "batch": 1, "rows": 128, "cols": 256, "dtype": "f32"},
        # the key projections of eight layers, taken together
        {"name": "ortho_batch_bf16", "op": "ortho", "batch": 8, "rows": 1024, "cols": 4096, "dtype": "bf16"},
        # a square projection
        {"name": "ortho_square_bf16", "op": "ortho", "batch": 1, "rows": 4096, "cols": 4096, "dtype": "bf16"},
        # matrices whose sizes fit no tile, taller than wide
        {"name": "ortho_odd_f16", "op": "ortho", "batch": 3, "rows": 2049, "cols": 1365, "dtype": "f16"},
        # the feed-forward matrix, taller than wide: the longest products
        {"name": "ortho_ffn_bf16", "op": "ortho", "batch": 1, "rows": 14336, "cols": 4096, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "train", "train", "quant", "ortho", "ortho", "ortho"])
    if op == "ortho":
        m, n = _log_int(rng, 32, 4096), _log_int(rng, 32, 8192)
        if rng.random() < 0.6:  # most models' sizes are multiples of 64
            m, n = (m + 63) // 64 * 64, (n + 63) // 64 * 64
        rows, cols = (m, n) if rng.random() < 0.5 else (n, m)
        most = int(1.3e11 // (min(m, n) ** 2 * max(m, n)))
        return {"op": op, "batch": max(1, min(most, rng.choice([1, 1, 2, 3, 8]))), "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "bf16", "f16", "f32"])}
    n, h = _log_int(rng, 1, 32768), _log_int(rng, 64, 8192)
    if rng.random() < 0.6:
        h = (h + 63) // 64 * 64
    n = min(n, (1 << 27) // h)
    dtype = rng.choice(["bf16", "bf16", "f16"] if op == "quant" else ["bf16", "bf16", "f16", "f32"])
    residual = rng.choice(["same", "same", "none", "f32"])
    if "f32" in (dtype, residual):
        n = max(1, n // 2)
    return {"op": op, "n": n, "h": h, "dtype": dtype, "residual": "same" if residual == dtype else residual, "weight": rng.random() < 0.8}


# ----------------------------------------------------------------- inputs
def prepare(case, seed):
    c, t = case, TYPES[case["dtype"]]
    g = torch.Generator(DEV).manual_seed(int(seed))
    if c["op"] == "ortho":
        # a momentum: what many examples have in common, of some rank, under their noise
        x = torch.randn(c["batch"], c["rows"], c["cols"], generator=g, device=DEV)
        rank = max(1, min(c["rows"], c["cols"]) // 32)
        u = torch.randn(c["batch"], c["rows"], rank, generator=g, device=DEV)
        v = torch.randn(c["batch"], rank, c["cols"], generator=g, device=DEV)
        x.baddbmm_(u, v, alpha=2.0 * rank ** -0.5).mul_(1e-4)
        return {"case": c, "x": x.to(t)}
    train = c["op"] == "train"
    s = {"case": c, "x": torch.randn(c["n"], c["h"], generator=g, device=DEV).to(t).requires_grad_(train), "residual": None, "weight": None}
    wide = torch.float32 if c["residual"] == "f32" else t
    if c["residual"] != "none":
        # the stream: each layer so far has added to it, to some of its columns more
        r = torch.randn(c["n"], c["h"], generator=g, device=DEV)
        s["residual"] = r.mul_(3.0 + 9.0 * (torch.rand(c["h"], generator=g, device=DEV) < 0.01)).to(wide).requires_grad_(train)
    if c["weight"]:
        s["weight"] = (1.0 + 0.3 * torch.randn(c["h"], generator=g, device=DEV)).to(t).requires_grad_(train)
    if train:
        s["grad_y"] = torch.randn(c["n"], c["h"], generator=g, device=DEV).mul_(0.02).to(t)
        if c["residual"] != "none":
            s["grad_sum"] = torch.randn(c["n"], c["h"], generator=g, device=DEV).mul_(0.02).to(wide)
    if c["op"] == "quant":
        s["values"] = torch.empty(c["n"], c["h"], dtype=t, device=DEV)
    return s


# ------------------------------------------------------------ plain forms
@torch.no_grad()
def _plain_norm(s):
    total = s["x"].float() if s["residual"] is None else s["x"].float() + s["residual"].float()
    inverse = ((total * total).mean(1, keepdim=True) + EPS).rsqrt()
    y = total * inverse
    if s["weight"] is not None:
        y = y * s["weight"].float()
    return total, inverse, y


@torch.no_grad()
def _plain_train(s):
    total, inverse, y = _plain_norm(s)
    t = s["x"].dtype
    unit = total * inverse
    upstream = s["grad_y"].float()
    inner = upstream if s["weight"] is None else upstream * s["weight"].float()
    grad = inverse * (inner - unit * (inner * unit).mean(1, keepdim=True))
    out = {"y": y.to(t)}
    if s["residual"] is not None:
        wide = s["residual"].dtype
        grad = grad + s["grad_sum"].float()
        out["sum"], out["grad_residual"] = total.to(wide), grad.to(wide)
    out["grad_x"] = grad.to(t)
    if s["weight"] is not None:
        out["grad_weight"] = (upstream * unit).sum(0).to(t)
    return out


def _plain_quant(s):
    total, _, y = _plain_norm(s)
    scale = y.abs().amax(1) / 127.0
    q = torch.where(scale.unsqueeze(1) > 0, y / scale.unsqueeze(1), 0.0).round().clamp(-127, 127)
    out = {"values": (q * scale.unsqueeze(1)).to(s["x"].dtype), "scale": scale}
    if s["residual"] is not None:
        out["sum"] = total.to(s["residual"].dtype)
    return out


def _plain_ortho(g):
    x = g.float()
    if x.shape[1] > x.shape[2]:
        x = x.transpose(1, 2)
    x = x / ((x * x).sum((1, 2), keepdim=True, dtype=torch.float64).sqrt().float() + 1e-7)
    for a, b, c in STEPS:
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    if g.shape[1] > g.shape[2]:
        x = x.transpose(1, 2)
    return x.contiguous().to(torch.bfloat16 if g.dtype == torch.float32 else g.dtype)


# -------------------------------------------------------------- the passes
def run(state):
    s, c = state, state["case"]
    if own:
        package = _package()
        if c["op"] == "ortho":
            return package.orthogonalize(s["x"], coefficients=STEPS)
        if c["op"] == "quant":
            q, scale, *total = package.rms_norm_quantize(s["x"], s["weight"], EPS, residual=s["residual"])
            # 8-bit integers are shown as the values that they stand for
            out = {"values": torch.mul(q, scale.unsqueeze(1), out=s["values"]), "scale": scale}
            return {**out, "sum": total[0]} if total else out
        got = package.rms_norm(s["x"], s["weight"], EPS, residual=s["residual"])
        y, total = got if s["residual"] is not None else (got, None)
        out = {"y": y} if total is None else {"y": y, "sum": total}
        if c["op"] == "norm":
            return out
        names = [k for k in ("residual", "x", "weight") if s[k] is not None]
        grads = torch.autograd.grad([y] if total is None else [y, total], [s[k] for k in names], [s["grad_y"]] if total is None else [s["grad_y"], s["grad_sum"]])
        return {**{k: v.detach() for k, v in out.items()}, **{"grad_" + k: v for k, v in zip(names, grads)}}
    if c["op"] == "ortho":
        return _plain_ortho(s["x"])
    if c["op"] == "quant":
        return _plain_quant(s)
    if c["op"] == "train":
        return _plain_train(s)
    total, _, y = _plain_norm(s)
    return {"y": y.to(s["x"].dtype)} if s["residual"] is None else {"y": y.to(s["x"].dtype), "sum": total.to(s["residual"].dtype)}


# ------------------------------------------------------------------- work
def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] == "ortho":
        m, n = sorted((c["rows"], c["cols"]))
        # x x^T and its square are symmetric: half of their sums are the other half's
        step = m * m * n + m * m * m + 2 * m * m * n
        return {"bytes": c["batch"] * m * n * (e + 2), "flops": c["batch"] * len(STEPS) * step}
    wide = {"none": 0, "same": e, "f32": 4}[c["residual"]]
    values = c["n"] * c["h"]
    # x and the residual, the output and the sum
    bytes_ = values * (e + wide + (1 if c["op"] == "quant" else e) + wide) + (4 * c["n"] if c["op"] == "quant" else 0)
    if c["op"] == "train":
        # the upstream gradients and the sum again (x where there is none), the gradients, one for both where the types agree
        bytes_ += values * (e + (2 * wide if wide else e) + e + (wide if wide != e else 0))
    weights = c["h"] * e * (3 if c["op"] == "train" else 1) if c["weight"] else 0
    return {"bytes": bytes_ + weights, "flops": values * (14 if c["op"] == "train" else 5)}


# ------------------------------------------------------- 64-bit definitions
def _exact_ortho(g):
    g = g.double()
    tall = g.shape[0] > g.shape[1]
    x = (g.T if tall else g) / (torch.linalg.matrix_norm(g) + 1e-7)
    # every step multiplies by a polynomial of x x^T; these all commute, so the product of the
    # polynomials can be gathered first
    gram = torch.mm(x, x.T)
    factor = torch.eye(x.shape[0], dtype=torch.float64, device=x.device)
    for a, b, c in STEPS:
        p = torch.addmm(b * gram, gram, gram, alpha=c)
        p.diagonal().add_(a)
        factor = torch.mm(p, factor)
        gram = torch.mm(torch.mm(p, gram), p)
    x = torch.mm(factor, x)
    return x.T if tall else x


@torch.no_grad()
def exact(case, seed):
    c = case
    s = prepare(c, seed)
    if c["op"] == "ortho":
        return torch.stack([_exact_ortho(g) for g in s["x"]])
    total = s["x"].double()
    if s["residual"] is not None:
        total = total.add_(s["residual"])
    rms = (torch.linalg.vector_norm(total, dim=1, keepdim=True).square_().div_(c["h"]).add_(EPS)).sqrt_()
    unit = total / rms
    y = unit if s["weight"] is None else unit * s["weight"].double()
    if c["op"] == "norm":
        return {"y": y} if s["residual"] is None else {"y": y, "sum": total}
    if c["op"] == "quant":
        # the integers round what is computed, so that the values have no 64-bit form of their own
        out = {"values": None, "scale": torch.linalg.vector_norm(y, math.inf, dim=1) / 127}
        return out if s["residual"] is None else {**out, "sum": total}
    out = {"y": y}
    inner = s["grad_y"].double()
    if s["weight"] is not None:
        out["grad_weight"] = torch.einsum("nh,nh->h", inner, unit)
        inner = inner * s["weight"].double()
    along = torch.einsum("nh,nh->n", inner, unit).div_(c["h"]).unsqueeze_(1)
    grad = torch.addcmul(inner, unit, along, value=-1).div_(rms)
    if s["residual"] is not None:
        grad.add_(s["grad_sum"])
        out["sum"], out["grad_residual"] = total, grad
    out["grad_x"] = grad
    return out
