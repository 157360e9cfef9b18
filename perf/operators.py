"""The training operators around the attention core, as they are measured: the
residual stream's layer norm, the gradients of the GAU projections, and the
softmax cross entropy over a vocabulary with its gradients.

``run`` computes each operator in its plain form (elementary torch operations
in 32 bits, rounded at the end), or, with ``own`` set, makes the calls of this
package that a training or serving program makes.
"""
import math

import torch

own = False

EPS = 1e-5
_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one decoded token's norm before its projections: latency alone
        {"name": "norm one token", "op": "norm", "M": 1, "d": 768, "type": "bf16", "res": True},
        # a decode batch in lockstep
        {"name": "norm 64 tokens", "op": "norm", "M": 64, "d": 768, "type": "bf16", "res": True},
        # a layer's norm in training, both directions: 2 sequences of 8192 tokens
        {"name": "norm train 16384", "op": "norm_train", "M": 16384, "d": 768, "type": "bf16",
         "res": True},
        # 32-bit activations, odd row length, no residual branch
        {"name": "norm train f32 odd", "op": "norm_train", "M": 5001, "d": 1001, "type": "f32",
         "res": False},
        # a layer's input projections in training: 2 sequences of 8192 tokens
        {"name": "project grad 16384", "op": "project", "M": 16384, "d": 768, "e": 1536, "s": 128},
        # a ragged last batch through a narrow layer
        {"name": "project grad 1001", "op": "project", "M": 1001, "d": 520, "e": 448, "s": 64},
        # the layer's output projection in training
        {"name": "output grad 16384", "op": "output", "M": 16384, "d": 768, "e": 1536},
        # and on a short batch
        {"name": "output grad 130", "op": "output", "M": 130, "d": 320, "e": 1000},
        # masked language modelling: 4 sequences of 4096, a target at 15 % of the tokens
        {"name": "loss masked 16384", "op": "loss_train", "M": 16384, "V": 32000, "d": 768,
         "keep": 0.15},
        # causal language modelling: 8 sequences of 1024, every token has a target
        {"name": "loss causal 8192", "op": "loss_train", "M": 8192, "V": 32000, "d": 768,
         "keep": 1.0},
        # evaluation: losses without gradients, odd vocabulary
        {"name": "loss eval 2048", "op": "loss", "M": 2048, "V": 50001, "d": 512, "keep": 1.0},
        # fine-tuning on a short answer: most of a short sequence is prompt
        {"name": "loss short 37", "op": "loss_train", "M": 37, "V": 8191, "d": 256, "keep": 0.4},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def draw(rng):
    op = rng.choice(["norm", "norm_train", "project", "output", "loss", "loss_train"])
    limit = 6 * 8192 * 32000 * 768 / 50
    while True:
        if op.startswith("norm"):
            case = {"op": op, "M": _log(rng, 1, 20000), "d": _log(rng, 32, 4096),
                    "type": rng.choice(["bf16", "bf16", "f32"]), "res": rng.random() < 0.6}
            if rng.random() < 0.6:
                case["d"] = max(32, case["d"] // 8 * 8)
        elif op == "project":
            case = {"op": op, "M": _log(rng, 1, 16384), "d": 8 * _log(rng, 8, 128),
                    "e": 64 * _log(rng, 1, 32), "s": 64 * rng.randint(1, 4)}
        elif op == "output":
            case = {"op": op, "M": _log(rng, 1, 16384), "d": 64 * _log(rng, 1, 16),
                    "e": 8 * _log(rng, 8, 256)}
        else:
            case = {"op": op, "M": _log(rng, 1, 16384), "V": _log(rng, 100, 50000),
                    "d": 8 * _log(rng, 8, 128), "keep": rng.choice([0.15, 0.5, 0.9, 1.0])}
        if _cost(case) <= limit and case["M"] * case.get("V", 1) <= 600_000_000:
            return case


def _kept(case):
    return max(1, int(round(case["M"] * case["keep"])))


def work(case):
    op, M, d = case["op"], case["M"], case["d"]
    if op.startswith("norm"):
        el = M * d * (2 if case["type"] == "bf16" else 4)
        # x, y; with a residual branch also that branch and the sum
        moved = el * (4 if case["res"] else 2) + 8 * d
        flops = 8 * M * d
        if op == "norm_train":
            # dy and dx, the residual stream's own gradient, dweight and dbias
            moved += el * (3 if case["res"] else 2) + 8 * d
            flops += 12 * M * d
        else:
            moved += 8 * M  # the rows' mean and 1 / deviation
        return {"bytes": moved, "flops": flops}
    if op == "project":
        N = 2 * case["e"] + case["s"]
        return {"bytes": 2 * (2 * M * d + 2 * N * d + M * N), "flops": 6 * M * N * d}
    if op == "output":
        e = case["e"]
        return {"bytes": 2 * (M * d + 2 * M * e + 2 * d * e), "flops": 4 * M * e * d}
    V, n = case["V"], _kept(case)
    if op == "loss":
        return {"bytes": 2 * (n * d + V * d) + 16 * M, "flops": 2 * n * V * d}
    return {"bytes": 2 * (n * d + M * d + 2 * V * d) + 20 * M, "flops": 6 * n * V * d}


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, M, d = case["op"], case["M"], case["d"]

    def normal(*shape, scale=1.0, shift=0.0, dtype=torch.bfloat16):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(scale).add_(shift).to(dtype)

    state = {"op": op}
    if op.startswith("norm"):
        t = _TYPES[case["type"]]
        # activations with a mean of their own, as a residual stream has
        state["x"] = normal(M, d, scale=1.5, shift=0.2, dtype=t)
        state["res"] = normal(M, d, scale=0.7, dtype=t) if case["res"] else None
        state["weight"] = normal(d, scale=0.2, shift=1.0, dtype=torch.float32)
        state["bias"] = normal(d, scale=0.2, dtype=torch.float32)
        if op == "norm_train":
            state["dy"] = normal(M, d, dtype=t)
            state["dh"] = normal(M, d, dtype=t) if case["res"] else None
    elif op == "project":
        e, s = case["e"], case["s"]
        state["x"] = normal(M, d)
        state["w"] = normal(2 * e + s, d, scale=1.0 / math.sqrt(d))
        state["du"], state["dv"] = normal(M, e), normal(M, e)
        state["dz"] = normal(M, s)
    elif op == "output":
        e = case["e"]
        state["y"] = normal(M, e)
        state["w"] = normal(d, e, scale=1.0 / math.sqrt(e))
        state["dout"] = normal(M, d)
    else:
        V, n = case["V"], _kept(case)
        state["x"] = normal(M, d)
        state["w"] = normal(V, d, scale=2.0 / math.sqrt(d))  # logits of deviation 2
        target = torch.randint(0, V, (M,), generator=g, device="cuda")
        at = torch.randperm(M, generator=g, device="cuda")[:n]
        state["target"] = torch.full_like(target, -100)
        state["target"][at] = target[at]
        # the mean over the tokens that have a target
        state["dloss"] = torch.full((M,), 1.0 / n, device="cuda")
    return state


# ------------------------------------------------------------ one pass of each

def run(state):
    return _RUN[state["op"]](state)


def _norm(s):
    if own:
        import flash_mixed_chunk_gb300 as fm
        y, h, mean, rstd = fm.layer_norm(s["x"], s["weight"], s["bias"], EPS, residual=s["res"])
        return {"y": y, "h": h, "mean": mean, "rstd": rstd}
    h, mean, rstd, xhat = _plain_norm(s)
    y = xhat * s["weight"] + s["bias"]
    return {"y": y.to(h.dtype), "h": h, "mean": mean[:, 0], "rstd": rstd[:, 0]}


def _plain_norm(s):
    x, r = s["x"], s["res"]
    h = x if r is None else (x.float() + r.float()).to(x.dtype)
    f = h.float()
    mean = f.mean(1, keepdim=True)
    c = f - mean
    rstd = 1.0 / torch.sqrt((c * c).mean(1, keepdim=True) + EPS)
    return h, mean, rstd, c * rstd


def _norm_train(s):
    if own:
        import flash_mixed_chunk_gb300 as fm
        y, h, mean, rstd = fm.layer_norm(s["x"], s["weight"], s["bias"], EPS, residual=s["res"])
        dx, dw, db = fm.layer_norm_backward(s["dy"], h, s["weight"], mean, rstd, dh=s["dh"])
        return {"y": y, "h": h, "dx": dx, "dweight": dw, "dbias": db}
    h, mean, rstd, xhat = _plain_norm(s)
    y = (xhat * s["weight"] + s["bias"]).to(h.dtype)
    dy = s["dy"].float()
    t = dy * s["weight"]
    dx = rstd * (t - t.mean(1, keepdim=True) - xhat * (t * xhat).mean(1, keepdim=True))
    if s["dh"] is not None:
        dx = dx + s["dh"].float()
    return {"y": y, "h": h, "dx": dx.to(h.dtype), "dweight": (dy * xhat).sum(0),
            "dbias": dy.sum(0)}


def _project(s):
    if own:
        import flash_mixed_chunk_gb300 as fm
        dx, dw = fm.gau_project_backward(s["x"], s["w"], s["du"], s["dv"], s["dz"])
        return {"dx": dx, "dw": dw}
    x, w = s["x"].float(), s["w"].float()
    pre = x @ w.T
    sig = 1.0 / (1.0 + torch.exp(-pre))
    d = torch.cat([s["du"], s["dv"], s["dz"]], 1).float() * sig * (1.0 + pre * (1.0 - sig))
    return {"dx": (d @ w).to(torch.bfloat16), "dw": (d.T @ x).to(torch.bfloat16)}


def _output(s):
    if own:
        import flash_mixed_chunk_gb300 as fm
        dy, dw = fm.gau_output_backward(s["y"], s["w"], s["dout"])
        return {"dy": dy, "dw": dw}
    d = s["dout"].float()
    return {"dy": (d @ s["w"].float()).to(torch.bfloat16),
            "dw": (d.T @ s["y"].float()).to(torch.bfloat16)}


def _plain_loss(s):
    z = s["x"].float() @ s["w"].float().T
    has = s["target"] >= 0
    at = torch.where(has, s["target"], torch.zeros_like(s["target"]))
    top = z.amax(1, keepdim=True)
    lse = torch.log(torch.exp(z - top).sum(1)) + top[:, 0]
    loss = lse - z.gather(1, at[:, None])[:, 0]
    zero = torch.zeros_like(lse)
    return z, has, at, torch.where(has, loss, zero), torch.where(has, lse, zero)


def _loss(s):
    if own:
        import flash_mixed_chunk_gb300 as fm
        loss, lse = fm.vocab_loss(s["x"], s["w"], s["target"])
        return {"loss": loss, "lse": lse}
    _, _, _, loss, lse = _plain_loss(s)
    return {"loss": loss, "lse": lse}


def _loss_train(s):
    if own:
        import flash_mixed_chunk_gb300 as fm
        loss, lse = fm.vocab_loss(s["x"], s["w"], s["target"])
        dx, dw = fm.vocab_loss_backward(s["x"], s["w"], s["target"], lse, s["dloss"])
        return {"loss": loss, "dx": dx, "dw": dw}
    z, has, at, loss, lse = _plain_loss(s)
    scale = torch.where(has, s["dloss"], torch.zeros_like(s["dloss"]))
    p = z.sub_(lse[:, None]).exp_().mul_(scale[:, None])
    p.scatter_add_(1, at[:, None], -scale[:, None])
    return {"loss": loss, "dx": (p @ s["w"].float()).to(torch.bfloat16),
            "dw": (p.T @ s["x"].float()).to(torch.bfloat16)}


_RUN = {"norm": _norm, "norm_train": _norm_train, "project": _project, "output": _output,
        "loss": _loss, "loss_train": _loss_train}


# ------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    leaf = lambda t: t.double().requires_grad_(True)  # noqa: E731
    if op.startswith("norm"):
        # the norm is that of the sum as it is stored
        h = s["x"] if s["res"] is None else (s["x"].double() + s["res"].double()).to(s["x"].dtype)
        a, w, b = leaf(h), leaf(s["weight"]), leaf(s["bias"])
        y = torch.nn.functional.layer_norm(a, (case["d"],), w, b, EPS)
        if op == "norm":
            var, mean = torch.var_mean(h.double(), dim=1, correction=0)
            return {"y": y.detach(), "h": h.double(), "mean": mean, "rstd": (var + EPS).rsqrt()}
        da, dw, db = torch.autograd.grad(y, (a, w, b), s["dy"].double())
        if s["dh"] is not None:
            da = da + s["dh"].double()
        return {"y": y.detach(), "h": h.double(), "dx": da, "dweight": dw, "dbias": db}
    if op == "project":
        x, w = leaf(s["x"]), leaf(s["w"])
        out = torch.nn.functional.silu(torch.nn.functional.linear(x, w))
        up = torch.cat([s["du"], s["dv"], s["dz"]], 1).double()
        dx, dw = torch.autograd.grad(out, (x, w), up)
        return {"dx": dx, "dw": dw}
    if op == "output":
        y, w = leaf(s["y"]), leaf(s["w"])
        out = torch.nn.functional.linear(y, w)
        dy, dw = torch.autograd.grad(out, (y, w), s["dout"].double())
        return {"dy": dy, "dw": dw}
    has = s["target"] >= 0
    x, w = leaf(s["x"]), leaf(s["w"])
    rows = torch.nn.functional.linear(x[has], w)
    each = torch.nn.functional.cross_entropy(rows, s["target"][has], reduction="none")
    loss = torch.zeros(case["M"], device="cuda", dtype=torch.float64)
    loss[has] = each.detach()
    if op == "loss":
        lse = torch.zeros_like(loss)
        lse[has] = torch.logsumexp(rows.detach(), 1)
        return {"loss": loss, "lse": lse}
    dx, dw = torch.autograd.grad(each, (x, w), s["dloss"][has].double())
    return {"loss": loss, "dx": dx, "dw": dw}
