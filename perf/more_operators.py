"""The operators of generation with states, as they are measured: linear attention
with a decay for each head over whole prompts and for single tokens, beam search's
selection over beams and vocabulary, and the reordering of states by its parents.

``run`` computes each operator in its plain form (elementary torch operations in 32
bits, in 64 where a selection or an exponent needs it, rounded at the end), or, with
``own`` set, makes the calls of this package that a serving program makes.
"""
import math

import torch

own = False

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # a short question's prompt, a small model: latency alone
        {"name": "prompt 37", "op": "prompt", "B": 1, "T": 37, "H": 4, "Hq": 4, "Hk": 4, "Hv": 4,
         "dk": 64, "dv": 64, "type": "bf16", "packed": True, "ragged": False, "carried": False},
        # a batch of prompts of different lengths, each behind an earlier turn's state; queries
        # and keys shared by all heads, as a gated attention unit's Z is
        {"name": "prompt ragged 8 x 1024", "op": "prompt", "B": 8, "T": 1024, "H": 12, "Hq": 1,
         "Hk": 1, "Hv": 12, "dk": 128, "dv": 128, "type": "bf16", "packed": False,
         "ragged": True, "carried": True},
        # two long documents through a layer of width 1536, q, k and v out of one projection
        {"name": "prompt 2 x 8192", "op": "prompt", "B": 2, "T": 8192, "H": 12, "Hq": 12,
         "Hk": 12, "Hv": 12, "dk": 128, "dv": 128, "type": "bf16", "packed": True,
         "ragged": False, "carried": False},
        # one very long document through a layer of width 2048
        {"name": "prompt 1 x 32768", "op": "prompt", "B": 1, "T": 32768, "H": 16, "Hq": 16,
         "Hk": 16, "Hv": 16, "dk": 128, "dv": 128, "type": "bf16", "packed": False,
         "ragged": False, "carried": False},
        # 32-bit activations, odd head sizes, grouped queries and keys
        {"name": "prompt f32 odd", "op": "prompt", "B": 3, "T": 777, "H": 6, "Hq": 6, "Hk": 2,
         "Hv": 3, "dk": 37, "dv": 75, "type": "f32", "packed": False, "ragged": True,
         "carried": True},
        # one sequence's next token
        {"name": "step 1", "op": "step", "B": 1, "H": 12, "Hq": 12, "Hk": 12, "Hv": 12,
         "dk": 128, "dv": 128, "type": "bf16"},
        # 64 sequences in lockstep, each a layer of width 1536
        {"name": "step 64", "op": "step", "B": 64, "H": 12, "Hq": 12, "Hk": 12, "Hv": 12,
         "dk": 128, "dv": 128, "type": "bf16"},
        # odd sizes in 32 bits, queries and keys shared
        {"name": "step f32 odd", "op": "step", "B": 9, "H": 6, "Hq": 2, "Hk": 1, "Hv": 6,
         "dk": 37, "dv": 75, "type": "f32"},
        # one request with 4 beams, logits as the output projection leaves them
        {"name": "select 1 x 4", "op": "select", "B": 1, "K": 4, "n": 4, "V": 32000,
         "type": "bf16", "done": 0.0},
        # a large batch of 8 beams, twice as many candidates as beams, 32-bit logits of an odd
        # vocabulary, some beams finished
        {"name": "select 64 x 8", "op": "select", "B": 64, "K": 8, "n": 16, "V": 50001,
         "type": "f32", "done": 0.2},
        # the states of one request's beams follow their parents
        {"name": "reorder 1 x 4", "op": "reorder", "B": 1, "K": 4, "layers": 2, "H": 4, "dk": 64,
         "dv": 64, "history": 100},
        # and those of a batch with several layers
        {"name": "reorder 8 x 8", "op": "reorder", "B": 8, "K": 8, "layers": 6, "H": 12,
         "dk": 128, "dv": 128, "history": 1000},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _cost(case):
    w = work(case)
    return max(w["bytes"], w["flops"] / 50)


def _heads(rng):
    H = _log(rng, 1, 24)
    of = [x for x in range(1, H + 1) if H % x == 0]
    q = rng.choice(of + [H, H])
    return H, q, rng.choice([q, q, rng.choice(of)]), rng.choice(of + [H, H, H])


def draw(rng):
    op = rng.choice(["prompt", "prompt", "step", "select", "reorder"])
    limit = max(_cost(c) for c in listed() if c["op"] == op)
    while True:
        if op in ("prompt", "step"):
            H, q, k, v = _heads(rng)
            case = {"op": op, "B": _log(rng, 1, 16 if op == "prompt" else 256), "H": H, "Hq": q,
                    "Hk": k, "Hv": v, "type": rng.choice(["bf16", "bf16", "bf16", "f32"])}
            if rng.random() < 0.7:
                case["dk"], case["dv"] = 8 * rng.randint(2, 16), 8 * rng.randint(2, 16)
            else:
                case["dk"], case["dv"] = _log(rng, 8, 200), _log(rng, 8, 300)
            if op == "prompt":
                case |= {"T": _log(rng, 1, 16384), "packed": rng.random() < 0.4,
                         "ragged": rng.random() < 0.4, "carried": rng.random() < 0.5}
        elif op == "select":
            case = {"op": op, "B": _log(rng, 1, 128), "K": rng.randint(1, 16),
                    "V": _log(rng, 50, 150000), "type": rng.choice(["bf16", "f32"]),
                    "done": rng.choice([0.0, 0.1, 0.5])}
            case["n"] = case["K"] * rng.randint(1, 2)
        else:
            case = {"op": op, "B": _log(rng, 1, 32), "K": rng.randint(2, 16),
                    "layers": rng.randint(1, 8), "H": _log(rng, 1, 16), "dk": _log(rng, 16, 128),
                    "dv": _log(rng, 16, 128), "history": _log(rng, 1, 4000)}
        # the plain form of a prompt keeps a state for every 128 tokens of a head
        states = case.get("T", 1) * case["B"] * case.get("H", 1) / 128
        if _cost(case) <= limit and states * case.get("dk", 1) * case.get("dv", 1) <= 1 << 28:
            return case


def _width(case):
    return 2 if case.get("type") == "bf16" else 4


def _tokens(case):
    """The batch's lengths: all T, or spread from none to T."""
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return [T] * B
    return [T if b == 0 else (T * ((37 * b) % 64)) // 63 for b in range(B)]


def work(case):
    op = case["op"]
    if op in ("prompt", "step"):
        B, H, dk, dv = case["B"], case["H"], case["dk"], case["dv"]
        el, state = _width(case), 4 * B * H * dk * dv
        token = (case["Hq"] + case["Hk"]) * dk + case["Hv"] * dv
        if op == "step":
            return {"bytes": el * B * (token + H * dv) + 2 * state, "flops": 5 * B * H * dk * dv}
        n, T = sum(_tokens(case)), case["T"]
        # outputs behind a sequence's end are zeros, and written
        return {"bytes": el * (n * token + B * T * H * dv) + state * (2 if case["carried"] else 1),
                "flops": 4 * n * H * dk * dv}
    if op == "select":
        n = case["B"] * case["K"] * case["V"]
        return {"bytes": _width(case) * n + 20 * case["B"] * case["n"], "flops": 4 * n}
    K = case["K"]
    row = case["layers"] * 4 * case["H"] * case["dk"] * case["dv"] + 8 * case["history"]
    # the rows that another beam takes, once, and the rows that change (as parents fall)
    taken, changed = K * (1 - (1 - 1 / K) ** (K - 1)), K - 1
    return {"bytes": case["B"] * row * (taken + changed) + 8 * case["B"] * K, "flops": 0}


# ----------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0, dtype=torch.float32):
        t = torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32)
        return t.mul_(scale).to(dtype)

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda", dtype=torch.float32)

    op, B = case["op"], case["B"]
    state = {"op": op}
    if op in ("prompt", "step"):
        t, H, dk, dv = _TYPES[case["type"]], case["H"], case["dk"], case["dv"]
        sizes = [(case["Hq"], dk), (case["Hk"], dk), (case["Hv"], dv)]
        lead = (B, case["T"]) if op == "prompt" else (B,)
        if case.get("packed"):  # one projection's output, cut by columns
            rows = normal(*lead, sum(h * d for h, d in sizes), dtype=t)
            parts = rows.split([h * d for h, d in sizes], dim=-1)
            q, k, v = (p.unflatten(-1, s) for p, s in zip(parts, sizes))
        else:
            q, k, v = (normal(*lead, *s, dtype=t) for s in sizes)
        state |= {"q": q, "k": k, "v": v, "scale": dk ** -0.5}
        # half-lives from 4 to 4000 tokens, one for each head
        state["log_decay"] = -math.log(2.0) / torch.exp(
            math.log(4.0) + uniform(H) * math.log(1000.0))
        state["lengths"] = None
        if case.get("ragged"):
            state["lengths"] = torch.tensor(_tokens(case), dtype=torch.int32, device="cuda")
        state["state"] = None
        if op == "step" or case["carried"]:
            state["state"] = normal(B, H, dk, dv, scale=3.0)
    elif op == "select":
        K, V = case["K"], case["V"]
        state["logits"] = normal(B, K, V, scale=2.5, dtype=_TYPES[case["type"]])
        # beams of a few tokens' length, the best first
        state["scores"] = -5.0 - torch.cumsum(uniform(B, K), 1)
        state["finished"] = uniform(B, K) < case["done"] if case["done"] else None
        state["n"] = case["n"]
    else:
        K, rows = case["K"], B * case["K"]
        shape = (rows, case["H"], case["dk"], case["dv"])
        state["tensors"] = [normal(*shape) for _ in range(case["layers"])]
        state["tensors"].append(torch.randint(0, 32000, (rows, case["history"]), generator=g,
                                              device="cuda"))
        state["parent"] = torch.randint(0, K, (B, K), generator=g, device="cuda")
    return state


# ------------------------------------------------------------ one pass of each

def run(state):
    return _RUN[state["op"]](state)


def _by_head(t, H):
    """[..., h, d] in 32 bits with a head for each of the H decays."""
    return t.float().repeat_interleave(H // t.shape[-2], dim=-2)


CHUNK = 128


def _prompt(s):
    q, k, v, ld, scale = s["q"], s["k"], s["v"], s["log_decay"], s["scale"]
    if own:
        import flash_mixed_chunk_gb300 as fm
        o, out = fm.decay_attention(q, k, v, ld, state=s["state"], scale=scale,
                                    lengths=s["lengths"])
        return {"o": o, "state": out}
    B, T = q.shape[:2]
    H = ld.shape[0]
    G = -(-T // CHUNK)
    # exponents of far positions in 64 bits
    rate, at = ld.double(), torch.arange(G * CHUNK, device=q.device)
    length = torch.full((B,), T, device=q.device) if s["lengths"] is None else s["lengths"]
    inside = at[None, :T] < length[:, None]

    def chunks(t):  # [B, H, G, CHUNK, d], nothing behind a sequence's end
        t = torch.where(inside[:, :, None, None], _by_head(t, H), 0.0)
        t = torch.cat([t, t.new_zeros(B, G * CHUNK - T, *t.shape[2:])], 1)
        return t.unflatten(1, (G, CHUNK)).permute(0, 3, 1, 2, 4)

    qc, kc, vc = chunks(q), chunks(k), chunks(v)
    i = torch.arange(CHUNK, device=q.device)
    gap = (i[:, None] - i[None, :]).double()
    near = torch.where(gap >= 0, torch.exp(rate[:, None, None] * gap.clamp(min=0)), 0.0).float()
    intra = (qc @ kc.transpose(-1, -2) * near[None, :, None]) @ vc
    left = torch.exp(rate[:, None] * (CHUNK - 1 - i)).float()
    grown = (kc * left[None, :, None, :, None]).transpose(-1, -2) @ vc  # of each chunk
    c = torch.arange(G, device=q.device)
    gap = (c[:, None] - 1 - c[None, :]).double()
    far = torch.where(gap >= 0, torch.exp(rate[:, None, None] * CHUNK * gap.clamp(min=0)),
                      0.0).float()
    before = (far @ grown.flatten(3)).unflatten(3, grown.shape[3:])
    if s["state"] is not None:
        start = torch.exp(rate[:, None] * CHUNK * c).float()
        before = before + start[None, :, :, None, None] * s["state"][:, :, None]
    ahead = torch.exp(rate[:, None] * (i + 1)).float()
    o = (intra + ahead[None, :, None, :, None] * (qc @ before)) * scale
    o = o.permute(0, 2, 3, 1, 4).flatten(1, 2)[:, :T]
    # the state after each sequence's own last token
    rest = length[:, None].double() - 1 - at[None]
    w = torch.where(rest[:, None] >= 0,
                    torch.exp(rate[None, :, None] * rest[:, None].clamp(min=0)), 0.0).float()
    out = (kc.flatten(2, 3) * w[..., None]).transpose(-1, -2) @ vc.flatten(2, 3)
    if s["state"] is not None:
        out = out + torch.exp(rate[None] * length[:, None]).float()[..., None, None] * s["state"]
    return {"o": o.to(q.dtype), "state": out}


def _step(s):
    q, k, v, ld, state = s["q"], s["k"], s["v"], s["log_decay"], s["state"]
    if own:
        import flash_mixed_chunk_gb300 as fm
        return {"o": fm.decay_step(q, k, v, ld, state, scale=s["scale"]), "state": state}
    H = ld.shape[0]
    q, k, v = _by_head(q, H), _by_head(k, H), _by_head(v, H)
    state.mul_(torch.exp(ld)[None, :, None, None]).add_(k[..., None] * v[..., None, :])
    o = (q[..., None] * state).sum(-2) * s["scale"]
    return {"o": o.to(s["q"].dtype), "state": state}


def _select(s):
    logits, scores, n = s["logits"], s["scores"], s["n"]
    if own:
        import flash_mixed_chunk_gb300 as fm
        score, parent, token = fm.beam_select(logits, scores, n, finished=s["finished"])
        return {"score": score, "parent": parent, "token": token}
    B, K, V = logits.shape
    # near the border between two beams' candidates 32 bits would take the wrong one
    z = logits.double()
    top = z.amax(2, keepdim=True)
    c = z.sub_(top)
    c -= torch.log(torch.exp(c).sum(2, keepdim=True))
    c += scores.double()[..., None]
    if s["finished"] is not None:  # a finished beam offers itself, with token 0
        alone = torch.full_like(c[:1, :1], -math.inf)
        c = torch.where(s["finished"][..., None], alone, c)
        c[..., 0] = torch.where(s["finished"], scores.double(), c[..., 0])
    c = c.flatten(1)
    m = min(n, K * V)
    least = c.topk(m, dim=1).values[:, -1:]
    above, tie = c > least, c == least
    room = m - above.sum(1, keepdim=True)
    taken = above | (tie & (torch.cumsum(tie, 1) <= room))
    at = torch.arange(K * V, device=c.device, dtype=torch.float64)
    index = torch.where(taken, -at, -math.inf).topk(m, dim=1).values.neg().long()
    found = c.gather(1, index)
    order = torch.sort(found, dim=1, descending=True, stable=True).indices
    return _answer(found.gather(1, order), index.gather(1, order), n, K, V)


def _answer(found, index, n, K, V):
    """Scores, parents and tokens; places without a candidate: the beam in turn, token 0."""
    B, m = found.shape
    found = torch.cat([found, found.new_full((B, n - m), -math.inf)], 1)
    index = torch.cat([index, index.new_zeros(B, n - m)], 1)
    none = torch.isinf(found)
    turn = torch.arange(n, device=found.device) % K
    return {"score": found.float(), "parent": torch.where(none, turn, index // V),
            "token": torch.where(none, 0, index % V)}


def _reorder(s):
    if own:
        import flash_mixed_chunk_gb300 as fm
        fm.beam_reorder(s["tensors"], s["parent"])
        return s["tensors"]
    B, K = s["parent"].shape
    rows = (s["parent"] + K * torch.arange(B, device=s["parent"].device)[:, None]).flatten()
    return [t.copy_(t[rows]) for t in s["tensors"]]


_RUN = {"prompt": _prompt, "step": _step, "select": _select, "reorder": _reorder}


# ------------------------------------------------ the definitions in 64 bits

def _exact_prompt(s, case):
    """Row by row blocks of the whole T x T form, a head at a time."""
    q, k, v = s["q"], s["k"], s["v"]
    B, T = q.shape[:2]
    H, dk, dv = case["H"], case["dk"], case["dv"]
    o = torch.zeros(B, T, H, dv, device="cuda", dtype=torch.float64)
    out = torch.zeros(B, H, dk, dv, device="cuda", dtype=torch.float64)
    if s["state"] is not None:
        out += s["state"].double()
    for b, n in enumerate(_tokens(case)):
        for h in range(H):
            if n == 0:
                continue
            lam = torch.exp(s["log_decay"][h].double() *
                            torch.arange(n + 1, device="cuda", dtype=torch.float64))
            x = q[b, :n, h // (H // case["Hq"])].double()
            y = k[b, :n, h // (H // case["Hk"])].double()
            z = v[b, :n, h // (H // case["Hv"])].double()
            s0 = out[b, h].clone()
            for i in range(0, n, 2048):
                j = min(n, i + 2048)
                gap = torch.arange(i, j, device="cuda")[:, None] - torch.arange(j, device="cuda")
                d = torch.where(gap >= 0, lam[gap.clamp(min=0)], 0.0)
                o[b, i:j, h] = (x[i:j] @ y[:j].T * d) @ z[:j] + lam[i + 1:j + 1, None] * (x[i:j] @ s0)
            out[b, h] = lam[n] * s0 + torch.einsum("ti,t,tj->ij", y, lam[:n].flip(0), z)
    return {"o": o * s["scale"], "state": out}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "prompt":
        return _exact_prompt(s, case)
    if op == "step":
        one = dict(case, T=1, ragged=False)
        return {key: t[:, 0] if key == "o" else t for key, t in _exact_prompt(
            {**s, "q": s["q"][:, None], "k": s["k"][:, None], "v": s["v"][:, None]}, one).items()}
    if op == "select":
        B, K, V = s["logits"].shape
        c = torch.log_softmax(s["logits"].double(), 2) + s["scores"].double()[..., None]
        if s["finished"] is not None:
            for b, k in s["finished"].nonzero().tolist():
                c[b, k] = -math.inf
                c[b, k, 0] = s["scores"][b, k].double()
        best, index = torch.sort(c.flatten(1), dim=1, descending=True, stable=True)
        m = min(case["n"], K * V)
        r = _answer(best[:, :m], index[:, :m], case["n"], K, V)
        none = torch.isinf(r["score"])
        pad = torch.full((B, case["n"] - m), -math.inf, device="cuda", dtype=torch.float64)
        r["score"] = torch.where(none, -math.inf, torch.cat([best[:, :m], pad], 1))
        return r
    K = case["K"]
    parent = s["parent"].tolist()
    return [torch.stack([t[b * K + p] for b, row in enumerate(parent) for p in row]).to(
        torch.float64 if t.is_floating_point() else t.dtype) for t in s["tensors"]]
