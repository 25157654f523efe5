"""What is measured of the operators next to the fused losses: gradient clipping over many
tensors, the choice and reordering of a beam search, and the 8-bit integer head.

Each operator has two forms. The plain one is written in elementary torch operations, in 32 bits
(64 where 32 would decide a comparison by rounding); the other is the package's own. `run` takes
the one that `own` names.
"""
import math

import torch

own = False

DEV = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


def _package():
    import linear_cross_entropy_vocab_gb300 as package
    return package


def _gen(seed, idx=0):
    return torch.Generator(DEV).manual_seed(int(seed) * 16 + idx)


# ------------------------------------------------------------------ cases
def listed():
    return [
        # the head of a small test model alone: three tensors, where only the calls' latency counts
        {"name": "clip_head_f32", "op": "clip", "layers": 0, "h": 128, "f": 1, "v": 1000, "dtype": "f32",
         "p": 2.0, "ratio": 0.3, "in_place": False, "pad": 1},
        # a training step of a 2.8-billion-parameter model with the Llama-3 head, norm above the limit
        {"name": "clip_model_bf16", "op": "clip", "layers": 8, "h": 4096, "f": 14336, "v": 128256, "dtype": "bf16",
         "p": 2.0, "ratio": 0.25, "in_place": False, "pad": 8},
        # the step that needs no clipping, in place, on tensors that start at odd addresses
        {"name": "clip_idle_f32", "op": "clip", "layers": 5, "h": 2048, "f": 5461, "v": 32001, "dtype": "f32",
         "p": 2.0, "ratio": 2.0, "in_place": True, "pad": 1},
        # one prompt, four beams: the smallest call of a decoding loop
        {"name": "select_one_bf16", "op": "select", "b": 1, "k": 4, "v": 32000, "m": 8, "dtype": "bf16", "mask": "none",
         "finished": 0, "std": 2.0},
        # constrained decoding: a mask for each prompt, some beams at their end, an odd vocabulary
        {"name": "select_masked_f16", "op": "select", "b": 7, "k": 5, "v": 9001, "m": 10, "dtype": "f16", "mask": "batch",
         "finished": 9, "std": 3.0},
        # offline generation: 64 prompts with eight beams over the Llama-3 vocabulary in 32 bits
        {"name": "select_many_f32", "op": "select", "b": 64, "k": 8, "v": 128256, "m": 16, "dtype": "f32", "mask": "none",
         "finished": 40, "std": 2.5},
        # a small cache and the token history behind it, for one prompt
        {"name": "reorder_one_bf16", "op": "reorder", "b": 1, "k": 4, "layers": 4, "heads": 8, "len": 129, "max_len": 256, "d": 64,
         "dtype": "bf16", "moved": 3, "sources": 2},
        # sixteen prompts with eight beams: caches of sixteen layers, filled to an odd length
        {"name": "reorder_many_bf16", "op": "reorder", "b": 16, "k": 8, "layers": 16, "heads": 8, "len": 777, "max_len": 1024, "d": 128,
         "dtype": "bf16", "moved": 6, "sources": 3},
        # laying out the Llama-3 head's weight in 8 bits, once for each checkpoint
        {"name": "quantize_head_bf16", "op": "quantize", "n": 128256, "h": 4096, "dtype": "bf16"},
        # the head of one decoding step with four beams
        {"name": "head_step_bf16", "op": "head", "n": 4, "h": 4096, "v": 128256, "dtype": "bf16", "bias": False, "softcap": 0.0},
        # the softcapped head of a batch of beams, logits with a bias, ragged in both directions
        {"name": "head_beams_f16", "op": "head", "n": 500, "h": 3584, "v": 152063, "dtype": "f16", "bias": True, "softcap": 30.0},
        # scoring a batch of prompts: every position's logits
        {"name": "head_prompt_bf16", "op": "head", "n": 8192, "h": 4096, "v": 128256, "dtype": "bf16", "bias": False, "softcap": 0.0},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["clip", "clip", "norm", "select", "select", "select", "reorder", "reorder", "quantize", "head", "head", "head"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("clip", "norm"):
        c = {"op": op, "layers": rng.randint(0, 8 if dtype != "f32" else 4), "h": _log_int(rng, 64, 4096), "f": 0,
             "v": _log_int(rng, 1000, 128256 if dtype != "f32" else 64000), "dtype": dtype, "p": rng.choice([2.0, 2.0, 2.0, 1.0, math.inf]),
             "ratio": rng.choice([0.25, 0.9, 2.0]), "in_place": False, "pad": rng.choice([1, 8, 8])}
        c["f"] = int(c["h"] * rng.uniform(1.0, 3.5))
        c["in_place"] = op == "norm" or c["ratio"] > 1.0 and rng.random() < 0.7
        return c
    if op == "select":
        b, k = _log_int(rng, 1, 64), rng.randint(1, 8)
        return {"op": op, "b": b, "k": k, "v": _log_int(rng, 500, 128256), "m": k * rng.choice([1, 2]), "dtype": dtype,
                "mask": rng.choice(["none", "none", "all", "batch", "beam"]), "finished": rng.choice([0, 0, b * k // 3]), "std": rng.uniform(0.5, 4.0)}
    if op == "reorder":
        k = rng.randint(2, 8)
        moved = rng.randint(1, k)
        length = _log_int(rng, 1, 1024)
        return {"op": op, "b": _log_int(rng, 1, 16), "k": k, "layers": rng.randint(1, 16), "heads": rng.choice([1, 4, 8]), "len": length,
                "max_len": length + rng.choice([0, 1, 60]), "d": rng.choice([64, 80, 128]), "dtype": dtype if dtype != "f32" else "bf16", "moved": moved,
                "sources": rng.randint(2 if moved > 1 and moved == k else 1, max(1, min(moved, k - 1) if moved < k else k))}
    h = _log_int(rng, 100, 4096)
    h = h if rng.random() < 0.25 else (h + 15) // 16 * 16
    if op == "quantize":
        return {"op": op, "n": _log_int(rng, 1, 128256), "h": h, "dtype": dtype if dtype != "f32" else "f16"}
    return {"op": op, "n": _log_int(rng, 1, 8192), "h": h, "v": _log_int(rng, 1000, 128256), "dtype": dtype if dtype != "f32" else "bf16",
            "bias": rng.random() < 0.4, "softcap": rng.choice([0.0, 0.0, 30.0])}


# ----------------------------------------------------------------- inputs
def _shapes(c):
    """The parameters of a decoder with grouped heads: projections, gated feed-forward, two norms a layer, and the head with a bias."""
    h, f = c["h"], c["f"]
    layer = [(h, h), (max(1, h // 4), h), (max(1, h // 4), h), (h, h), (f, h), (h,), (h,)]
    return layer * c["layers"] + [(c["v"], h), (c["v"],), (h,)]


def _grads(c, seed):
    """Gradients that are views of one flat buffer, as a bucketed training step has them, each starting at a multiple of `pad` elements."""
    starts, total = [], 0
    for s in _shapes(c):
        starts.append(total)
        total += -(-math.prod(s) // c["pad"]) * c["pad"]
    flat = torch.zeros(total, dtype=TYPES[c["dtype"]], device=DEV)
    g = _gen(seed)
    for i, (s, at) in enumerate(zip(_shapes(c), starts)):
        flat[at:at + math.prod(s)].normal_(0.0, 1e-3 * (1 + i % 3), generator=g)
    return flat, [flat[at:at + math.prod(s)].view(s) for s, at in zip(_shapes(c), starts)]


def _parents(c, seed):
    """[b, k] parents: in each row `moved` beams continue one of `sources` other beams and the rest continue themselves."""
    g = torch.Generator().manual_seed(int(seed) * 16 + 5)
    k, rows = c["k"], []
    for _ in range(c["b"]):
        src = torch.randperm(k, generator=g)[:c["sources"]].tolist()
        order = [j for j in torch.randperm(k, generator=g).tolist() if j not in src] + src
        parent = list(range(k))
        for i, j in enumerate(order[:c["moved"]]):
            parent[j] = src[i % len(src)] if src[i % len(src)] != j else src[(i + 1) % len(src)]
        rows.append(parent)
    return torch.tensor(rows, dtype=torch.int64, device=DEV)


def prepare(case, seed):
    c, t = case, TYPES[case["dtype"]]
    if c["op"] in ("clip", "norm"):
        flat, grads = _grads(c, seed)
        # max_norm is `ratio` of the norm that these inputs are expected to have
        n = [math.prod(s) for s in _shapes(c)]
        std = [1e-3 * (1 + i % 3) for i in range(len(n))]
        if c["p"] == 2.0:
            norm = math.sqrt(sum(m * s * s for m, s in zip(n, std)))
        elif c["p"] == 1.0:
            norm = sum(m * s for m, s in zip(n, std)) * math.sqrt(2 / math.pi)
        else:
            norm = max(s * math.sqrt(2 * math.log(m + 1)) for m, s in zip(n, std))
        s = {"flat": flat, "grads": grads, "max_norm": norm * c["ratio"] * (1.0 if c["p"] != math.inf else 0.9 if c["ratio"] < 1 else 1.5)}
        if c["op"] == "clip" and not c["in_place"]:
            out = torch.zeros_like(flat)
            s["out_flat"] = out
            s["out"] = [out[g.storage_offset():g.storage_offset() + g.numel()].view(g.shape) for g in grads]
    elif c["op"] == "select":
        g = _gen(seed)
        logits = torch.randn(c["b"], c["k"], c["v"], generator=g, device=DEV).mul_(c["std"])
        scores = torch.rand(c["b"], c["k"], generator=g, device=DEV).mul_(-4.0 * c["std"]).sub_(1.0)
        finished = torch.zeros(c["b"] * c["k"], dtype=torch.bool, device=DEV)
        finished[torch.randperm(c["b"] * c["k"], generator=g, device=DEV)[:c["finished"]]] = True
        allowed = None
        if c["mask"] != "none":
            shape = {"all": (1, 1, c["v"]), "batch": (c["b"], 1, c["v"]), "beam": (c["b"], c["k"], c["v"])}[c["mask"]]
            allowed = torch.rand(shape, generator=g, device=DEV) < 0.03
            allowed[0, 0] &= c["mask"] == "all"  # a prompt (or beam) that nothing can continue
            # what a masked place holds is left over from other work
            logits = torch.where((torch.rand(logits.shape, generator=g, device=DEV) < 0.01) & ~allowed, float("nan"), logits)
        s = {"logits": logits.to(t), "scores": scores, "finished": finished.view(c["b"], c["k"]), "allowed": allowed}
    elif c["op"] == "reorder":
        g = _gen(seed)
        shape = (c["layers"], c["b"] * c["k"], c["heads"], c["max_len"], c["d"])
        kv = [torch.empty(shape, dtype=t, device=DEV).normal_(generator=g) for _ in range(2)]
        tokens = torch.randint(0, 32000, (c["b"] * c["k"], c["len"]), generator=g, device=DEV)
        s = {"states": [x[:, :, :, :c["len"]] for x in kv] + [tokens.unsqueeze(0)], "parents": _parents(c, seed)}
    elif c["op"] == "quantize":
        s = {"x": torch.randn(c["n"], c["h"], generator=_gen(seed), device=DEV).mul_(c["h"] ** -0.5).to(t)}
    else:
        g = _gen(seed)
        x = torch.randn(c["n"], c["h"], generator=g, device=DEV).to(t)
        wq = torch.empty(c["v"], c["h"], device=DEV).normal_(0.0, 32.0, generator=g).round_().clamp_(-127, 127).to(torch.int8)
        ws = torch.rand(c["v"], generator=g, device=DEV).add_(0.5).mul_(c["h"] ** -0.5 / 32.0)
        bias = torch.randn(c["v"], generator=g, device=DEV).mul_(0.1).to(t) if c["bias"] else None
        s = {"x": x, "wq": wq, "ws": ws, "bias": bias, "softcap": c["softcap"] or None}
    s["case"] = c
    return s


# ------------------------------------------------------------ plain forms
def _plain_norm(grads, p):
    if p == math.inf:
        return torch.stack([g.float().abs().max() for g in grads]).max()
    each = torch.stack([g.float().abs().pow(p).sum(dtype=torch.float64) for g in grads])
    return each.sum().pow(1.0 / p).float()


def _plain_clip(s):
    grads, p = s["grads"], s["case"]["p"]
    norm = _plain_norm(grads, p)
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    [o.copy_(g.float() * coef) for g, o in zip(grads, s.get("out", grads))]
    return {"norm": norm, "grads": s.get("out_flat", s["flat"])}


def _plain_select(s):
    b, k, v = s["logits"].shape
    m = s["case"]["m"]
    z = s["logits"].double()
    if s["allowed"] is not None:
        z = torch.where(s["allowed"], z, -math.inf)
    # in 64 bits: what is chosen hangs on comparisons
    top = z.amax(2, keepdim=True)
    e = (z - torch.where(top > -math.inf, top, 0.0)).exp()
    z = z - (e.sum(2, keepdim=True).log() + top)
    z = torch.where(top > -math.inf, z, -math.inf) + s["scores"].double().unsqueeze(2)
    # a finished beam offers itself alone, under the padding token 0
    z[s["finished"]] = -math.inf
    z[:, :, 0] = torch.where(s["finished"], s["scores"].double(), z[:, :, 0])
    score, at = torch.sort(z.reshape(b, k * v), dim=1, descending=True, stable=True)
    score, at = score[:, :m], at[:, :m]
    some = score > -math.inf
    return {"scores": score.float(), "parents": torch.where(some, at // v, 0), "tokens": torch.where(some, at % v, 0)}


def _plain_reorder(s):
    b, k = s["parents"].shape
    rows = (s["parents"] + torch.arange(b, device=DEV).unsqueeze(1) * k).reshape(-1)
    return [x.copy_(x[:, rows]) for x in s["states"]]


def _plain_quantize(x):
    x = x.float()
    scale = x.abs().amax(1) / 127.0
    q = torch.where(scale.unsqueeze(1) > 0, x / scale.unsqueeze(1), 0.0).round().clamp(-127, 127)
    return q, scale


def _plain_head(s):
    q, scale = _plain_quantize(s["x"])
    z = (q @ s["wq"].float().t()) * s["ws"] * scale.unsqueeze(1)
    if s["bias"] is not None:
        z = z + s["bias"].float()
    if s["softcap"] is not None:
        z = s["softcap"] * torch.tanh(z / s["softcap"])
    return z.to(s["x"].dtype)


# -------------------------------------------------------------- the passes
def run(state):
    c = state["case"]
    if own:
        package = _package()
        if c["op"] == "norm":
            return package.grad_norm(state["grads"], c["p"])
        if c["op"] == "clip" and c["in_place"]:
            return {"norm": package.clip_grads_(state["grads"], state["max_norm"], c["p"]), "grads": state["flat"]}
        if c["op"] == "clip":
            return {"norm": package.clip_grads(state["grads"], state["max_norm"], c["p"], out=state["out"]), "grads": state["out_flat"]}
        if c["op"] == "select":
            r = package.beam_select(state["logits"], state["scores"], c["m"], finished=state["finished"], allowed=state["allowed"])
            return {"scores": r.scores, "parents": r.parents, "tokens": r.tokens}
        if c["op"] == "reorder":
            package.beam_reorder_(state["states"], state["parents"], dim=1)
            return state["states"]
        if c["op"] == "quantize":
            q, scale = package.quantize_rows(state["x"])
            return {"q": q, "scale": scale}
        return package.int8_linear(state["x"], state["wq"], state["ws"], state["bias"], softcap=state["softcap"])
    if c["op"] == "norm":
        return _plain_norm(state["grads"], c["p"])
    if c["op"] == "clip":
        return _plain_clip(state)
    if c["op"] == "select":
        return _plain_select(state)
    if c["op"] == "reorder":
        return _plain_reorder(state)
    if c["op"] == "quantize":
        q, scale = _plain_quantize(state["x"])
        return {"q": q.to(torch.int8), "scale": scale}
    return _plain_head(state)


# ------------------------------------------------------------------- work
def work(case):
    c, e = case, SIZE[case["dtype"]]
    if c["op"] in ("clip", "norm"):
        n = sum(math.prod(s) for s in _shapes(c))
        # a step that needs no clipping and is done in place has nothing to write
        writes = 0 if c["op"] == "norm" or c["in_place"] and c["ratio"] > 1 else 1
        return {"bytes": n * e * (1 + writes) + 4, "flops": (2 + writes) * n}
    if c["op"] == "select":
        live = c["b"] * c["k"] - c["finished"]
        masks = {"none": 0, "all": c["v"], "batch": c["b"] * c["v"], "beam": live * c["v"]}[c["mask"]]
        return {"bytes": live * c["v"] * e + masks + 5 * c["b"] * c["k"] + 20 * c["b"] * c["m"], "flops": 3 * live * c["v"]}
    if c["op"] == "reorder":
        row = c["layers"] * c["heads"] * c["len"] * c["d"] * e * 2 + c["len"] * 8
        return {"bytes": c["b"] * (c["moved"] + min(c["sources"], c["moved"])) * row + 8 * c["b"] * c["k"], "flops": 0}
    if c["op"] == "quantize":
        return {"bytes": c["n"] * (c["h"] * (e + 1) + 4), "flops": 3 * c["n"] * c["h"]}
    return {"bytes": c["n"] * c["h"] * e + c["v"] * (c["h"] + 4 + (e if c["bias"] else 0)) + c["n"] * c["v"] * e,
            "flops": 2 * c["n"] * c["h"] * c["v"]}


# ------------------------------------------------------- 64-bit definitions
def exact(case, seed):
    c = case
    if c["op"] == "head" and c["n"] * c["h"] * c["v"] > 1.5e12:
        return None  # the products take too long in 64 bits
    s = prepare(case, seed)
    if c["op"] in ("clip", "norm"):
        total, peak = torch.zeros((), dtype=torch.float64, device=DEV), torch.zeros((), dtype=torch.float64, device=DEV)
        for part in s["flat"].split(1 << 26):  # the places between tensors hold zeros
            a = part.double().abs()
            total += a.sum() if c["p"] == 1.0 else (a * a).sum()
            peak = torch.maximum(peak, a.max())
        norm = peak if c["p"] == math.inf else total if c["p"] == 1.0 else total.sqrt()
        if c["op"] == "norm":
            return norm
        factor = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
        return {"norm": norm, "grads": s["flat"].double() * factor}
    if c["op"] == "select":
        rows, parents, tokens = [], [], []
        for i in range(c["b"]):
            z = s["logits"][i].double()
            if s["allowed"] is not None:
                z = z.masked_fill(~s["allowed"].expand(c["b"], c["k"], c["v"])[i], -math.inf)
            lse = torch.logsumexp(z, 1, keepdim=True)
            z = (z - lse).nan_to_num(nan=-math.inf, neginf=-math.inf) + s["scores"][i].double()[:, None]
            for j in range(c["k"]):
                if s["finished"][i, j]:
                    z[j] = -math.inf
                    z[j, 0] = s["scores"][i, j].double()
            best, at = z.flatten().topk(c["m"])
            rows.append(best)
            parents.append(torch.where(best > -math.inf, at // c["v"], 0))
            tokens.append(torch.where(best > -math.inf, at % c["v"], 0))
        return {"scores": torch.stack(rows), "parents": torch.stack(parents), "tokens": torch.stack(tokens)}
    if c["op"] == "reorder":
        return None  # copies: nothing is computed
    if c["op"] == "quantize":
        return {"q": None, "scale": torch.linalg.vector_norm(s["x"].double(), math.inf, dim=1) / 127}
    x = s["x"].double()
    step = torch.linalg.vector_norm(x, math.inf, dim=1, keepdim=True) / 127
    z = torch.zeros(c["n"], c["v"], dtype=torch.float64, device=DEV)
    for at in range(0, c["v"], 16384):
        z[:, at:at + 16384] = torch.round(x / step) @ s["wq"][at:at + 16384].double().T
    z = z * step * s["ws"].double() + (0 if s["bias"] is None else s["bias"].double())
    return z if s["softcap"] is None else s["softcap"] * (z / s["softcap"]).tanh()
