"""The operators of one expert block around the token exchange, as measured workloads: the balance
loss of its router (with its gradient), the experts' products in 8-bit integers, and the norms
before and after the block (with their gradients).

`listed()` names the cases, `draw()` gives more of the same ranges, `prepare()` makes a case's inputs
on the GPU, `run()` is one pass and `exact()` the same outputs in 64 bits.  With `own` false `run()`
computes them with elementary torch operations, with `own` true through the package's calls.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}
_EPS = 1e-6


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # One layer's balance and z losses in training, forward and backward, over the whole batch.
        {"name": "balance train", "op": "balance", "dtype": BF16, "T": 4096, "E": 128, "K": 8, "S": 1, "score": "softmax",
         "padding": False},
        # The same of a sigmoid router, a loss for each of 24 packed sequences, padding masked out.
        {"name": "balance packed", "op": "balance", "dtype": F32, "T": 16384, "E": 256, "K": 8, "S": 24, "score": "sigmoid",
         "padding": True},
        # One user's next token through the experts' first product, gated: latency.
        {"name": "i8 up one token", "op": "up", "dtype": BF16, "T": 1, "E": 128, "K": 8, "H": 2048, "I": 768, "act": "silu"},
        # A full decode batch: nearly every expert has some rows, so every weight is read.
        {"name": "i8 up decode", "op": "up", "dtype": BF16, "T": 64, "E": 128, "K": 8, "H": 2048, "I": 768, "act": "silu"},
        # A prefill's first product: 256 rows an expert on average, none a whole number of tiles.
        {"name": "i8 up prefill", "op": "up", "dtype": BF16, "T": 4096, "E": 128, "K": 8, "H": 2048, "I": 768, "act": "silu"},
        # Its second product, back to the row width.
        {"name": "i8 down prefill", "op": "down", "dtype": BF16, "T": 4096, "E": 128, "K": 8, "H": 2048, "I": 768},
        # A wide layer's shared expert on every token, from the norm before the block on.
        {"name": "i8 shared wide", "op": "shared", "dtype": BF16, "T": 4096, "H": 7168, "I": 2048, "act": "silu"},
        # A small float32 layer with ragged widths, as in a parity run.
        {"name": "i8 f32 ragged", "op": "up", "dtype": F32, "T": 333, "E": 5, "K": 2, "H": 624, "I": 332,
         "act": "gelu_tanh"},
        # The end of a decode step's block: combine, norm, residual and the next block's norm.
        {"name": "norm decode", "op": "after", "dtype": BF16, "T": 32, "H": 2048, "K": 8, "E": 128, "G": 0, "post": True,
         "next": True, "grad": False},
        # The same of a long prefill with a gate for each channel.
        {"name": "norm prefill", "op": "after", "dtype": BF16, "T": 8192, "H": 2816, "K": 8, "E": 128, "G": 1, "post": True,
         "next": True, "grad": False},
        # Training: both norms, a gate for each of 8 sequences, forward and every gradient.
        {"name": "norm train", "op": "after", "dtype": BF16, "T": 4096, "H": 2048, "K": 0, "E": 0, "G": 8, "post": True,
         "next": True, "grad": True},
        # Ragged float32 rows with a gate for each token, forward and every gradient.
        {"name": "norm f32 ragged", "op": "after", "dtype": F32, "T": 333, "H": 1004, "K": 0, "E": 0, "G": 333,
         "post": True, "next": True, "grad": True},
    ]


def _between(rng, lo, hi, step=1):
    """A whole number of [lo, hi], evenly spread over its logarithm, down to a multiple of `step`."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return max(lo, min(hi, v) // step * step)


def draw(rng):
    op = rng.choice(["balance", "i8", "i8", "after"])
    dtype = rng.choice([BF16, BF16, F32])
    chunk = 8 if dtype == BF16 else 4  # elements of a 16-byte chunk: rows are whole chunks
    if op == "balance":
        T, E = _between(rng, 1, 16384), _between(rng, 8, 384)
        return {"op": op, "dtype": dtype, "T": T, "E": E, "K": rng.randint(1, min(12, E)),
                "S": rng.choice([1, _between(rng, 1, min(64, T))]), "score": rng.choice(["softmax", "sigmoid"]),
                "padding": rng.random() < 0.5}
    if op == "i8":
        c = {"op": rng.choice(["up", "up", "down", "shared"]), "dtype": dtype, "T": _between(rng, 1, 4096),
             "H": _between(rng, 256, 4096, 16), "I": _between(rng, 96, 1024, 16)}
        if c["op"] != "down":
            c["act"] = rng.choice(["silu", "gelu_tanh"])
        if c["op"] == "shared":  # a norm's last bit may turn a rounding to 8 bits: the exact rows are bfloat16
            return c | {"dtype": BF16}
        E = _between(rng, 4, 128)
        K = rng.randint(1, min(8, E))
        if c["T"] * K > 4096:
            c["H"] = min(c["H"], 2048)
        return c | {"E": E, "K": K}
    T = _between(rng, 1, 4096)
    c = {"op": op, "dtype": dtype, "T": T, "H": _between(rng, 256, 4096, chunk), "K": 0, "E": 0,
         "G": rng.choice([0, 1, T, rng.choice([g for g in range(1, 65) if T % g == 0])]), "post": rng.random() < 0.7,
         "next": rng.random() < 0.7, "grad": rng.random() < 0.5}
    if not c["grad"] and rng.random() < 0.6:
        c |= {"K": rng.randint(1, 8), "E": _between(rng, 8, 128)}
    return c


# ---- inputs ------------------------------------------------------------------------------------

def _routing(T, E, K, g):
    v, idx = torch.topk(torch.softmax(torch.empty(T, E, device="cuda").normal_(generator=g), 1), K, 1)
    return idx.to(torch.int32).contiguous(), (v / v.sum(1, keepdim=True)).contiguous()


def _bank(shape, g):
    """Weights as a program has them: 8-bit values and a scale for each channel."""
    q = torch.empty(shape, dtype=torch.float16, device="cuda").normal_(0.0, 32.0, generator=g)
    q = q.round_().clamp_(-127, 127).to(torch.int8)
    s = torch.rand(shape[:-1], device="cuda", generator=g).add_(0.5).mul_(shape[-1] ** -0.5 / 32.0)
    return q, s


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[c["dtype"]]
    dev = "cuda"

    def rows(*shape, scale=1.0):
        return torch.empty(shape, dtype=dt, device=dev).normal_(0.0, scale, generator=g)

    s, T = {"case": c}, c["T"]
    if c["op"] == "balance":
        E, S = c["E"], c["S"]
        s["logits"] = rows(T, E)
        s["logits"] += torch.linspace(0, 1, E, device=dev).to(dt)  # some experts are sought more
        s["idx"] = torch.topk(s["logits"], c["K"], 1)[1].to(torch.int32).contiguous()
        cut = torch.sort(torch.randperm(T - 1, device=dev, generator=g)[:S - 1] + 1)[0] if S > 1 else None
        ends = [torch.zeros(1, device=dev)] + ([cut] if S > 1 else []) + [torch.full((1,), T, device=dev)]
        s["offset"] = torch.cat([e.to(torch.int32) for e in ends]).contiguous()
        s["seq"] = torch.searchsorted(s["offset"][1:].contiguous(), torch.arange(T, device=dev, dtype=torch.int32), right=True)
        s["mask"] = (torch.rand(T, device=dev, generator=g) > 0.1) if c["padding"] else None
        s["grad_loss"] = torch.rand(2, device=dev, generator=g) * 0.01
    elif c["op"] in ("up", "down"):
        E, K, H, I = c["E"], c["K"], c["H"], c["I"]
        s["idx"], _ = _routing(T, E, K, g)
        # the plain form's plan: rows of the largest expert
        s["most"] = int(torch.bincount(s["idx"].view(-1).long(), minlength=E).max())
        s["x"] = rows(T, H) if c["op"] == "up" else rows(T * K, I)
        s["w"], s["w_scale"] = _bank((E, 2 * I, H) if c["op"] == "up" else (E, H, I), g)
    elif c["op"] == "shared":
        s["x"], s["weight"] = rows(T, c["H"]), rows(c["H"], scale=0.1) + 1
        s["w"], s["w_scale"] = _bank((2 * c["I"], c["H"]), g)
    else:
        H, K = c["H"], c["K"]
        s["x"] = rows(T, H)
        if K:
            s["idx"], s["weights"] = _routing(T, c["E"], K, g)
        s["y"] = rows(T * K if K else T, H)
        s["gate"] = rows(c["G"], H, scale=0.5) if c["G"] else None
        s["weight"] = rows(H, scale=0.1) + 1 if c["post"] else None
        s["next"] = rows(H, scale=0.1) + 1 if c["next"] else None
        if c["grad"]:
            s["grad_out"] = rows(T, H)
            s["grad_n"] = rows(T, H) if c["next"] else None
    return s


# ---- one pass ----------------------------------------------------------------------------------

_RESIDUAL = 0.5  # the residual's scale


def run(state):
    c = state["case"]
    if own:
        return {"balance": _own_balance, "up": _own_up, "down": _own_down, "shared": _own_shared, "after": _own_after}[c["op"]](state, c)
    return {"balance": _plain_balance, "up": _plain_up, "down": _plain_down, "shared": _plain_shared, "after": _plain_after}[c["op"]](state, c)


def _own_balance(s, c):
    import combine_moe_layout_04_amd as M
    kw = dict(seq_offset=s["offset"], token_mask=s["mask"], score=c["score"])
    loss, counts, probs, tokens = M.moe_balance(s["logits"], s["idx"], **kw)
    grad = M.moe_balance_bwd(s["logits"], counts, tokens, s["grad_loss"], c["K"], **kw)
    return {"loss": loss, "counts": counts, "probs": probs, "tokens": tokens, "grad_logits": grad}


def _own_up(s, c):
    import combine_moe_layout_04_amd as M
    # the handle object is kept by the program; the layout on it is this pass's own
    h = s["handle"] = M.moe_layout(s["idx"], c["E"], 1, handle=s.get("handle"))
    q, scale = M.moe_quant_rows(s["x"])
    return M.moe_matmul_i8(q, scale, s["w"], s["w_scale"], handle=h, tokens=True, activation=c["act"], dtype=_TYPES[c["dtype"]])


def _own_down(s, c):
    import combine_moe_layout_04_amd as M
    h = s["handle"] = M.moe_layout(s["idx"], c["E"], 1, handle=s.get("handle"))
    q, scale = M.moe_quant_rows(s["x"])
    return M.moe_matmul_i8(q, scale, s["w"], s["w_scale"], handle=h, dtype=_TYPES[c["dtype"]])


def _own_shared(s, c):
    import combine_moe_layout_04_amd as M
    q, scale = M.moe_prenorm(s["x"], s["weight"], eps=_EPS, quantize=True)
    return M.moe_matmul_i8(q, scale, s["w"], s["w_scale"], activation=c["act"], dtype=_TYPES[c["dtype"]])


def _own_after(s, c):
    import combine_moe_layout_04_amd as M
    kw = dict(gate=s["gate"], residual_scale=_RESIDUAL)
    h = None
    if c["K"]:
        h = s["handle"] = M.moe_layout(s["idx"], c["E"], 1, handle=s.get("handle"))
    out, n, rstd = M.moe_postnorm(s["x"], s["y"], s["weight"], next_weight=s["next"], eps=_EPS, handle=h,
                                  topk_weights=s.get("weights"), **kw)
    got = {"out": out, "n": n}
    if c["grad"]:
        gx, gy, gw, gg, gn = M.moe_postnorm_bwd(s["grad_out"], s["grad_n"], s["x"], s["y"], rstd, s["weight"],
                                                next_weight=s["next"], **kw)
        got |= {"grad_x": gx, "grad_y": gy, "grad_weight": gw, "grad_gate": gg, "grad_next": gn}
    return {k: v for k, v in got.items() if v is not None}


# ---- the plain forms: elementary operations in 32 bits, rounded once at the end -----------------

def _plain_balance(s, c):
    z, E, K, S = s["logits"].float(), c["E"], c["K"], c["S"]
    there = torch.ones(c["T"], 1, device=z.device) if s["mask"] is None else s["mask"].float().view(-1, 1)
    top = z.max(1, keepdim=True)[0]
    e = torch.exp(z - top)
    total = e.sum(1, keepdim=True)
    soft, lse = e / total, top + torch.log(total)
    if c["score"] == "softmax":
        p, slope = soft, soft
    else:
        sig = 1.0 / (1.0 + torch.exp(-z))
        p = sig / sig.sum(1, keepdim=True)
        slope = p * (1.0 - sig)
    member = (s["seq"].view(-1, 1) == torch.arange(S, device=z.device)).float() * there      # [T, S]
    chosen = torch.zeros_like(z).scatter_add_(1, s["idx"].long(), torch.ones_like(s["idx"], dtype=torch.float32))
    counts = torch.matmul(member.t(), chosen)                                                # whole numbers below 2^24
    probs = torch.matmul(member.t(), p)
    n = member.sum(0)                                                                        # [S]
    share = torch.where(n > 0, E / (K * (n > 0).sum() * n.clamp(min=1) ** 2), 0.0).view(-1, 1)
    all_n = n.sum().clamp(min=1)
    loss = torch.stack([(share * counts * probs).sum(), (there * lse * lse).sum() / all_n])
    a = s["grad_loss"][0] * torch.matmul(member, share * counts)                             # [T, E]
    grad = slope * (a - (p * a).sum(1, keepdim=True)) + there * (s["grad_loss"][1] * 2.0 / all_n) * lse * soft
    return {"loss": loss, "counts": counts.to(torch.int32), "probs": probs, "tokens": n.to(torch.int32),
            "grad_logits": grad.to(s["logits"].dtype)}


def _plain_quant(x):
    """Rows as whole numbers in [-127, 127] and their scales; in 64 bits, for values next to a border."""
    scale = (x.abs().max(1, keepdim=True)[0].float() / 127.0).clamp(min=2.0 ** -126)
    return torch.round(x.double() / scale.double()).float(), scale


def _plain_act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_product(s, c, q, scale, of_token):
    """The grouped product: pairs sorted by expert, each expert's in a block of the largest one's size."""
    flat, most = s["idx"].view(-1).long(), s["most"]
    e, order = torch.sort(flat, stable=True)
    if len(flat) <= c["E"]:  # fewer pairs than experts: their experts' weights, one copy a pair
        source = order // c["K"] if of_token else torch.arange(len(e), device=flat.device)
        y = torch.matmul(s["w"][e].float(), q[source].unsqueeze(2)).squeeze(2)
        return y * scale[source] * s["w_scale"][e]
    counts = torch.zeros(c["E"], dtype=torch.int64, device=flat.device).scatter_add_(0, e, torch.ones_like(e))
    place = torch.arange(len(e), device=flat.device) - (torch.cumsum(counts, 0) - counts)[e] + e * most
    source = order // c["K"] if of_token else torch.arange(len(e), device=flat.device)
    blocks = torch.zeros(c["E"] * most, q.shape[1], device=flat.device)
    blocks[place] = q[source]
    y = torch.matmul(blocks.view(c["E"], most, -1), s["w"].float().transpose(1, 2))
    y = y.view(c["E"] * most, -1)[place]
    return y * scale[source] * s["w_scale"][e]


def _plain_up(s, c):
    q, scale = _plain_quant(s["x"])
    y = _plain_product(s, c, q, scale, True)
    return (_plain_act(y[:, :c["I"]], c["act"]) * y[:, c["I"]:]).to(s["x"].dtype)


def _plain_down(s, c):
    q, scale = _plain_quant(s["x"])
    return _plain_product(s, c, q, scale, False).to(s["x"].dtype)


def _plain_shared(s, c):
    x = s["x"].float()
    n = x * (1.0 / torch.sqrt((x * x).mean(1, keepdim=True) + _EPS)) * s["weight"].float()
    q, scale = _plain_quant(n)
    y = torch.matmul(q, s["w"].float().t()) * scale * s["w_scale"]
    return (_plain_act(y[:, :c["I"]], c["act"]) * y[:, c["I"]:]).to(s["x"].dtype)


def _plain_after(s, c):
    x, y, dt, T, H = s["x"].float(), s["y"].float(), s["x"].dtype, c["T"], c["H"]
    if c["K"]:
        # receive rows: the pairs in the order of their experts, stable
        place = torch.empty(T * c["K"], dtype=torch.int64, device=x.device)
        place[torch.sort(s["idx"].view(-1), stable=True)[1]] = torch.arange(T * c["K"], device=x.device)
        y = (y[place].view(T, c["K"], H) * s["weights"].unsqueeze(2)).sum(1)
    G = c["G"]
    gate = s["gate"].float().repeat_interleave(T // G, 0) if G else 1.0
    yn, hat = y, y
    if c["post"]:
        r1 = 1.0 / torch.sqrt((y * y).mean(1, keepdim=True) + _EPS)
        hat = y * r1
        yn = hat * s["weight"].float()
    out = _RESIDUAL * x + gate * yn
    got = {"out": out.to(dt)}
    if c["next"]:
        r2 = 1.0 / torch.sqrt((out * out).mean(1, keepdim=True) + _EPS)
        on = out * r2
        got["n"] = (on * s["next"].float()).to(dt)
    if c["grad"]:
        d = s["grad_out"].float()
        if c["next"]:
            gn = s["grad_n"].float()
            got["grad_next"] = (gn * on).sum(0).to(dt)
            gn = gn * s["next"].float()
            d = d + r2 * (gn - on * (gn * on).mean(1, keepdim=True))
        got["grad_x"] = (_RESIDUAL * d).to(dt)
        v = d * gate
        if G:
            got["grad_gate"] = (d * yn).view(G, T // G, H).sum(1).to(dt)
        if c["post"]:
            got["grad_weight"] = (v * hat).sum(0).to(dt)
            v = v * s["weight"].float()
            v = r1 * (v - hat * (v * hat).mean(1, keepdim=True))
        got["grad_y"] = v.to(dt)
    return got


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    c = case
    es, T = 2 if c["dtype"] == BF16 else 4, c["T"]
    if c["op"] == "balance":
        E, K, S = c["E"], c["K"], c["S"]
        return {"bytes": 2 * T * E * es + T * K * 4 + 8 * S * E + (T if c["padding"] else 0), "flops": 20.0 * T * E}
    if c["op"] in ("up", "down"):
        E, K, H, I = c["E"], c["K"], c["H"], c["I"]
        used = E * (1.0 - (1.0 - K / E) ** T)             # experts that some token chose, on average
        if c["op"] == "up":
            b = T * H * es + T * K * (4 + I * es) + used * 2 * I * (H + 4)
            return {"bytes": b, "flops": 4.0 * T * K * H * I}
        return {"bytes": T * K * (4 + (I + H) * es) + used * H * (I + 4), "flops": 2.0 * T * K * H * I}
    if c["op"] == "shared":
        H, I = c["H"], c["I"]
        return {"bytes": T * (H + I) * es + H * es + 2 * I * (H + 4), "flops": 4.0 * T * H * I}
    H, K, G = c["H"], c["K"], c["G"]
    row = T * H * es
    b = row * (2 + (K or 1) + c["next"]) + 8 * T * K + G * H * es + H * es * (c["post"] + c["next"])
    f = T * H * (2.0 * K + 12)
    if c["grad"]:
        # grad_out, grad_n, x and y read, grad_x and grad_y written; the forward pass read x and y, but a backward
        # pass comes later
        b += row * (4 + 2 * c["next"]) + 2 * G * H * es + H * es * (c["post"] + c["next"])
        f += T * H * 30.0
    return {"bytes": b, "flops": f}


# ---- the definition in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"balance": _exact_balance, "up": _exact_experts, "down": _exact_experts, "shared": _exact_shared, "after": _exact_after}[case["op"]](s, case)


def _exact_balance(s, c):
    z = s["logits"].double().requires_grad_(True)
    S, E, K = c["S"], c["E"], c["K"]
    bounds = s["offset"].tolist()
    keep = torch.ones(c["T"], dtype=torch.bool, device=z.device) if s["mask"] is None else s["mask"]
    counts, probs, tokens, parts = [], [], [], []
    for q in range(S):
        at = torch.arange(bounds[q], bounds[q + 1], device=z.device)
        at = at[keep[at]]
        p = torch.softmax(z[at], 1) if c["score"] == "softmax" else torch.nn.functional.normalize(torch.special.expit(z[at]), p=1.0, dim=1)
        counts.append(torch.bincount(s["idx"][at].reshape(-1).long(), minlength=E))
        probs.append(p.sum(0))
        tokens.append(len(at))
        if len(at):
            parts.append(E * torch.dot(counts[-1].double() / (K * len(at)), p.mean(0)))
    lse = torch.logsumexp(z[keep], 1)
    n = max(1, sum(tokens))
    loss = torch.stack([sum(parts) / len(parts) if parts else 0 * z.sum(), (lse ** 2).sum() / n])
    grad, = torch.autograd.grad(loss, z, s["grad_loss"].double())
    return {"loss": loss.detach(), "counts": torch.stack(counts).to(torch.int32), "probs": torch.stack(probs).detach(),
            "tokens": torch.tensor(tokens, dtype=torch.int32, device=z.device), "grad_logits": grad}


def _exact_quant(x):
    scale = torch.clamp((x.abs().amax(1) / 127).float(), min=2.0 ** -126).double()
    return torch.round(x / scale[:, None]), scale


def _exact_gated(y, c):
    gate, up = torch.chunk(y, 2, 1)
    f = torch.nn.functional
    return (f.silu(gate) if c["act"] == "silu" else f.gelu(gate, approximate="tanh")) * up


def _exact_experts(s, c):
    # a float32 row's largest value over 127 is rounded to float32 as the definition's scale is
    q, scale = _exact_quant(s["x"].double())
    out, first = [], 0
    for e in range(c["E"]):
        t, k = torch.nonzero(s["idx"] == e, as_tuple=True)
        rows = t if c["op"] == "up" else torch.arange(first, first + len(t), device=t.device)
        first += len(t)
        if not len(t):
            continue
        y = (q[rows] @ s["w"][e].double().t().contiguous()) * scale[rows, None] * s["w_scale"][e].double()
        out.append(_exact_gated(y, c) if c["op"] == "up" else y)
    return torch.cat(out)


def _exact_shared(s, c):
    x = s["x"].double()
    n = x * torch.rsqrt(x.square().mean(1, keepdim=True) + _EPS) * s["weight"].double()
    q, scale = _exact_quant(n)
    y = (q @ s["w"].double().t().contiguous()) * scale[:, None] * s["w_scale"].double()
    return _exact_gated(y, c)


def _exact_after(s, c):
    leaf = {k: s[k].double().requires_grad_(c["grad"]) for k in ("x", "y", "gate", "weight", "next") if s.get(k) is not None}
    T, H = c["T"], c["H"]
    y = leaf["y"]
    if c["K"]:
        pair = torch.argsort(s["idx"].reshape(-1).long() * (T * c["K"]) + torch.arange(T * c["K"], device=y.device))
        y = torch.zeros(T, H, dtype=torch.float64, device=y.device).index_add_(
            0, pair // c["K"], y * s["weights"].double().reshape(-1)[pair][:, None])
    if c["post"]:
        y = torch.nn.functional.rms_norm(y, (H,), leaf["weight"], _EPS)
    if c["G"]:
        y = (y.view(c["G"], T // c["G"], H) * leaf["gate"][:, None]).reshape(T, H)
    out = torch.add(y, leaf["x"], alpha=_RESIDUAL)
    got = {"out": out}
    if c["next"]:
        got["n"] = torch.nn.functional.rms_norm(out, (H,), leaf["next"], _EPS)
    if c["grad"]:
        up = [s["grad_out"].double()] + ([s["grad_n"].double()] if c["next"] else [])
        grads = dict(zip(leaf, torch.autograd.grad(list(got.values()), list(leaf.values()), up)))
        got |= {"grad_" + k: v for k, v in grads.items()}
    return {k: v.detach() for k, v in got.items()}
