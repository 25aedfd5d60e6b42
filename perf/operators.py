"""The operators around the token exchange, as measured workloads: the router that decides a layer's
routing (with its gradient), a whole expert layer for a few tokens, and low-rank adapters of many
requests beside a shared projection (with their gradients).

`listed()` names the cases, `draw()` gives more of the same ranges, `prepare()` makes a case's inputs
on the GPU, `run()` is one pass and `exact()` the same outputs in 64 bits.  With `own` false `run()`
computes them with elementary torch operations, with `own` true through the package's calls.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TYPES = {BF16: torch.bfloat16, F32: torch.float32}


# ---- cases -------------------------------------------------------------------------------------

def listed():
    return [
        # A decode step's routing: 32 sequences, one token each, 8 of 128 experts.
        {"name": "route decode", "op": "route", "dtype": BF16, "T": 32, "E": 128, "K": 8, "score": "softmax",
         "bias": False, "renormalize": True, "groups": 1, "topk_groups": 1, "scale": 1.0, "grad": False},
        # One layer's routing in training, forward and backward; the scores are not renormalised, so
        # the gradient is dense.
        {"name": "route train", "op": "route", "dtype": BF16, "T": 4096, "E": 128, "K": 8, "score": "softmax",
         "bias": False, "renormalize": False, "groups": 1, "topk_groups": 1, "scale": 1.0, "grad": True},
        # A long prefill through a group-limited sigmoid router with a balancing bias: 4 of 8 groups.
        {"name": "route grouped prefill", "op": "route", "dtype": F32, "T": 16384, "E": 256, "K": 8,
         "score": "sigmoid", "bias": True, "renormalize": True, "groups": 8, "topk_groups": 4, "scale": 2.5,
         "grad": False},
        # The same router in training.
        {"name": "route grouped train", "op": "route", "dtype": F32, "T": 4096, "E": 256, "K": 8,
         "score": "sigmoid", "bias": True, "renormalize": True, "groups": 8, "topk_groups": 4, "scale": 2.5,
         "grad": True},
        # One user's next token through one layer: latency.
        {"name": "few one token", "op": "few", "dtype": BF16, "T": 1, "E": 128, "K": 8, "H": 2048, "I": 768,
         "act": "silu", "of": 128},
        # A full decode batch: nearly every expert has some rows, so every weight is read.
        {"name": "few batch", "op": "few", "dtype": BF16, "T": 64, "E": 128, "K": 8, "H": 2048, "I": 768,
         "act": "silu", "of": 128},
        # One rank's 32 of 256 experts of a wide layer: most pairs go to other ranks (no local expert).
        {"name": "few wide share", "op": "few", "dtype": BF16, "T": 13, "E": 32, "K": 8, "H": 7168, "I": 2048,
         "act": "silu", "of": 256},
        # A small float32 layer with ragged widths, as in a parity run.
        {"name": "few f32 ragged", "op": "few", "dtype": F32, "T": 7, "E": 8, "K": 2, "H": 1004, "I": 332,
         "act": "gelu_tanh", "of": 8},
        # A decode step of 48 requests over 32 adapters; some requests have none.
        {"name": "lowrank decode", "op": "lowrank", "dtype": BF16, "T": 48, "A": 32, "H": 2048, "N": 2048, "r": 16,
         "weights": False, "grad": False},
        # Prefill of several requests at once beside one projection.
        {"name": "lowrank prefill", "op": "lowrank", "dtype": BF16, "T": 8192, "A": 16, "H": 4096, "N": 4096,
         "r": 32, "weights": False, "grad": False},
        # Training a few adapters side by side: forward and every gradient.
        {"name": "lowrank train", "op": "lowrank", "dtype": BF16, "T": 4096, "A": 4, "H": 2048, "N": 4096, "r": 64,
         "weights": False, "grad": True},
        # Ragged float32 adapters with a learned weight per token, forward and every gradient.
        {"name": "lowrank f32 ragged", "op": "lowrank", "dtype": F32, "T": 333, "A": 5, "H": 612, "N": 1028,
         "r": 12, "weights": True, "grad": True},
    ]


def _between(rng, lo, hi, step=1):
    """A whole number of [lo, hi], evenly spread over its logarithm, down to a multiple of `step`."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
    return max(lo, min(hi, v) // step * step)


def draw(rng):
    op = rng.choice(["route", "few", "lowrank"])
    dtype = rng.choice([BF16, BF16, F32])
    chunk = 8 if dtype == BF16 else 4  # elements of a 16-byte chunk: rows are whole chunks
    if op == "route":
        c = {"op": op, "dtype": dtype, "T": _between(rng, 1, 16384), "grad": rng.random() < 0.5,
             "renormalize": rng.random() < 0.6, "scale": rng.choice([1.0, 1.0, 2.5])}
        if rng.random() < 0.5:
            E = _between(rng, 8, 384)
            c |= {"E": E, "score": rng.choice(["softmax", "sigmoid"]), "bias": False, "groups": 1, "topk_groups": 1}
            most = E
        else:
            groups = rng.choice([1, 4, 8])
            per = _between(rng, 4, 32 if groups > 1 else 256)
            keep = rng.randint(1, groups)
            c |= {"E": groups * per, "score": "sigmoid", "bias": True, "groups": groups, "topk_groups": keep}
            most = keep * per
        return c | {"K": rng.randint(1, min(12, most))}
    if op == "few":
        E = _between(rng, 4, 128)
        K = rng.randint(1, min(8, E))
        return {"op": op, "dtype": dtype, "T": _between(rng, 1, 64), "E": E, "K": K,
                "H": _between(rng, 256, 2816 if dtype == BF16 else 1408, chunk), "I": _between(rng, 96, 768, chunk),
                "act": rng.choice(["silu", "gelu_tanh"]), "of": E * rng.choice([1, 1, 4])}
    grad = rng.random() < 0.5
    return {"op": op, "dtype": dtype, "T": _between(rng, 1, 4096), "A": _between(rng, 1, 64),
            "H": _between(rng, 256, 4096, chunk), "N": _between(rng, 256, 4096, chunk), "r": _between(rng, chunk, 64, chunk),
            "weights": rng.random() < 0.3, "grad": grad}


# ---- inputs ------------------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _TYPES[c["dtype"]]
    dev = "cuda"

    def rows(*shape, scale=1.0):
        t = torch.empty(shape, dtype=dt, device=dev)
        return t.normal_(0.0, scale, generator=g)

    s = {"case": c}
    if c["op"] == "route":
        s["logits"] = rows(c["T"], c["E"])
        if c["bias"]:
            s["bias"] = torch.empty(c["E"], device=dev).normal_(0.0, 0.05, generator=g)
        if c["grad"]:
            s["grad_w"] = torch.empty(c["T"], c["K"], device=dev).normal_(generator=g)
    elif c["op"] == "few":
        T, E, K, H, I = c["T"], c["E"], c["K"], c["H"], c["I"]
        z = torch.empty(T, c["of"], device=dev).normal_(generator=g)
        v, idx = torch.topk(torch.softmax(z, 1), K, 1)
        first = (c["of"] - E) // 2  # this rank's experts; the others' ids are no local expert
        local = idx - first
        s["topk_idx"] = torch.where((local >= 0) & (local < E), local, -1).to(torch.int32).contiguous()
        s["topk_weights"] = (v / v.sum(1, keepdim=True)).contiguous()
        s["x"] = rows(T, H)
        s["w13"] = rows(E, 2 * I, H, scale=H ** -0.5)
        s["w2"] = rows(E, H, I, scale=I ** -0.5)
    else:
        T, A, H, N, r = c["T"], c["A"], c["H"], c["N"], c["r"]
        # one adapter in eight requests is none: id A
        ids = torch.randint(0, A, (T,), device=dev, generator=g)
        none = torch.rand(T, device=dev, generator=g) < 0.125
        s["ids"] = torch.where(none, A, ids).to(torch.int32).view(T, 1).contiguous()
        s["x"], s["base"] = rows(T, H), rows(T, N)
        s["a"], s["b"] = rows(A, r, H, scale=H ** -0.5), rows(A, r, N, scale=r ** -0.5)
        if c["weights"]:
            s["weights"] = torch.rand(T, 1, device=dev, generator=g) + 0.5
        if c["grad"]:
            s["grad_out"] = rows(T, N)
    return s


# ---- one pass ----------------------------------------------------------------------------------

def run(state):
    c = state["case"]
    if own:
        return {"route": _own_route, "few": _own_few, "lowrank": _own_lowrank}[c["op"]](state, c)
    return {"route": _plain_route, "few": _plain_few, "lowrank": _plain_lowrank}[c["op"]](state, c)


def _own_route(s, c):
    import combine_moe_layout_04_amd as M
    kw = dict(score=c["score"], renormalize=c["renormalize"], scale=c["scale"])
    idx, w = M.moe_route(s["logits"], c["K"], bias=s.get("bias"), num_groups=c["groups"], topk_groups=c["topk_groups"], **kw)
    if not c["grad"]:
        return {"idx": idx, "w": w}
    return {"idx": idx, "w": w, "grad_logits": M.moe_route_bwd(s["logits"], idx, s["grad_w"], **kw)}


def _own_few(s, c):
    import combine_moe_layout_04_amd as M
    return M.moe_few(s["x"], s["topk_idx"], s["topk_weights"], s["w13"], s["w2"], activation=c["act"])


def _own_lowrank(s, c):
    import combine_moe_layout_04_amd as M
    # the handle object is kept by the program; the layout on it is this pass's own
    h = s["handle"] = M.moe_layout(s["ids"], c["A"] + 1, 1, handle=s.get("handle"))
    w = s.get("weights")
    out, u = M.moe_lowrank(h, s["x"], s["a"], s["b"], w, base=s["base"])
    if not c["grad"]:
        return out
    grad_x, grad_a, grad_b, grad_w = M.moe_lowrank_bwd(h, s["grad_out"], s["x"], s["a"], s["b"], u, w, grad_w=c["weights"])
    got = {"out": out, "grad_x": grad_x, "grad_a": grad_a, "grad_b": grad_b}
    return got | {"grad_w": grad_w} if c["weights"] else got


# ---- the plain forms: elementary operations in 32 bits, rounded once at the end -----------------

def _plain_route(s, c):
    z = s["logits"]
    T, E, K, G = z.shape[0], z.shape[1], c["K"], c["groups"]
    if c["bias"] or G > 1:
        # scores are compared with each other: 64 bits, for values next to a border
        key = torch.sigmoid(z.double()) + s["bias"].double()
        if G > 1:
            best2 = torch.sort(key.view(T, G, E // G), dim=2, descending=True)[0][:, :, :2].sum(2)
            keep = torch.sort(best2, dim=1, descending=True, stable=True)[1][:, :c["topk_groups"]]
            mask = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, keep, True)
            key = torch.where(mask.repeat_interleave(E // G, 1), key, -math.inf)
    else:
        key = z  # both scores grow with the logit
    idx = torch.sort(key, dim=1, descending=True, stable=True)[1][:, :K]
    z = z.float()
    if c["score"] == "softmax":
        e = torch.exp(z - z.max(1, keepdim=True)[0])
        p = e / e.sum(1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-z))
    sel = torch.gather(p, 1, idx)
    total = sel.sum(1, keepdim=True) if c["renormalize"] else 1.0
    w = sel * (c["scale"] / total)
    out = {"idx": idx.to(torch.int32), "w": w}
    if c["grad"]:
        gs = s["grad_w"] * c["scale"]
        if c["renormalize"]:
            gs = (gs - (gs * sel).sum(1, keepdim=True) / total) / total
        gp = torch.zeros_like(p).scatter_(1, idx, gs)
        if c["score"] == "softmax":
            gz = p * (gp - (gs * sel).sum(1, keepdim=True))
        else:
            gz = gp * p * (1.0 - p)
        out["grad_logits"] = gz.to(s["logits"].dtype)
    return out


def _plain_act(g, act):
    if act == "silu":
        return g / (1.0 + torch.exp(-g))
    return 0.5 * g * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (g + 0.044715 * g * g * g)))


def _plain_few(s, c):
    x, idx, w = s["x"].float(), s["topk_idx"].long(), s["topk_weights"]
    (T, K), E, I = idx.shape, c["E"], c["I"]
    there = idx >= 0
    if T * K <= E:  # fewer pairs than experts: their experts' weights, one copy a pair
        at = idx.clamp(min=0).view(-1)
        w13, w2 = s["w13"][at].float(), s["w2"][at].float()
        gu = torch.matmul(w13, x.repeat_interleave(K, 0).unsqueeze(2)).squeeze(2)
        a = _plain_act(gu[:, :I], c["act"]) * gu[:, I:]
        y = torch.matmul(w2, a.unsqueeze(2)).squeeze(2).view(T, K, -1)
        wt = torch.where(there, w, 0.0)
        return (y * wt.unsqueeze(2)).sum(1).to(s["x"].dtype)
    # every expert on every token, then each token's own
    gu = torch.matmul(x, s["w13"].float().transpose(1, 2))           # [E, T, 2I]
    a = _plain_act(gu[..., :I], c["act"]) * gu[..., I:]
    wt = torch.zeros(T, E, device=x.device).scatter_add_(1, idx.clamp(min=0), torch.where(there, w, 0.0))
    y = torch.matmul(a * wt.t().unsqueeze(2), s["w2"].float().transpose(1, 2))
    return y.sum(0).to(s["x"].dtype)


def _plain_lowrank(s, c):
    x, base = s["x"].float(), s["base"].float()
    A, r, H, N, T = c["A"], c["r"], c["H"], c["N"], c["T"]
    a, b = s["a"].float().view(A * r, H), s["b"].float().view(A * r, N)
    mine = (s["ids"] == torch.arange(A, device=x.device)).repeat_interleave(r, 1)  # [T, A r]
    w = s["weights"] if c["weights"] else 1.0
    u = torch.where(mine, torch.matmul(x, a.t()), 0.0)
    out = (base + w * torch.matmul(u, b)).to(s["x"].dtype)
    if not c["grad"]:
        return out
    g = s["grad_out"].float()
    raw = torch.where(mine, torch.matmul(g, b.t()), 0.0)
    gu = w * raw
    got = {"out": out, "grad_x": torch.matmul(gu, a).to(s["x"].dtype),
           "grad_a": torch.matmul(gu.t(), x).view(A, r, H).to(s["x"].dtype),
           "grad_b": torch.matmul((w * u).t(), g).view(A, r, N).to(s["x"].dtype)}
    return got | {"grad_w": (raw * u).sum(1, keepdim=True)} if c["weights"] else got


# ---- what a pass cannot do without ---------------------------------------------------------------

def work(case):
    c = case
    es = 2 if c["dtype"] == BF16 else 4
    if c["op"] == "route":
        T, E, K = c["T"], c["E"], c["K"]
        b = T * E * es + T * K * 8 + (4 * E if c["bias"] else 0)
        f = T * E * 8
        if c["grad"]:
            b += T * K * 4 + T * E * es
            f += T * E * 8
        return {"bytes": b, "flops": f}
    if c["op"] == "few":
        T, E, K, H, I = c["T"], c["E"], c["K"], c["H"], c["I"]
        used = E * (1.0 - (1.0 - K / c["of"]) ** T)      # experts that some token chose, on average
        pairs = T * K * E / c["of"]
        return {"bytes": used * 3 * H * I * es + 2 * T * H * es + T * K * 8, "flops": 6.0 * pairs * H * I}
    T, A, H, N, r = c["T"], c["A"], c["H"], c["N"], c["r"]
    used = A * (1.0 - (1.0 - 0.875 / A) ** T)
    with_one = 0.875 * T
    b = T * H * es + 2 * T * N * es + used * r * (H + N) * es + 4 * T * (2 if c["weights"] else 1)
    f = 2.0 * with_one * r * (H + N)
    if c["grad"]:
        b += T * N * es + T * H * es + A * r * (H + N) * es + (4 * T if c["weights"] else 0)
        f *= 3
    return {"bytes": b, "flops": f}


# ---- the definition in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "few": _exact_few, "lowrank": _exact_lowrank}[case["op"]](s, case)


def _exact_route(s, c):
    z = s["logits"].double()
    T, E = z.shape
    K, G = c["K"], c["groups"]
    p = torch.softmax(z, 1) if c["score"] == "softmax" else torch.special.expit(z)
    key = p + s["bias"].double() if c["bias"] else z
    if G > 1:
        top = torch.topk(key.reshape(T * G, E // G), 2, 1)[0].sum(1).reshape(T, G)
        order = torch.argsort(-top, dim=1, stable=True)
        place = torch.empty_like(order).scatter_(1, order, torch.arange(G, device=z.device).expand(T, G).contiguous())
        out_of = torch.repeat_interleave(place >= c["topk_groups"], E // G, dim=1)
        key = key.masked_fill(out_of, -math.inf)
    idx = torch.argsort(-key, dim=1, stable=True)[:, :K].contiguous()
    leaf = z.clone().requires_grad_(c["grad"])
    q = torch.softmax(leaf, 1) if c["score"] == "softmax" else torch.special.expit(leaf)
    w = q.gather(1, idx)
    if c["renormalize"]:
        w = w / w.sum(1, keepdim=True)
    w = w * c["scale"]
    out = {"idx": idx.to(torch.int32), "w": w.detach()}
    if c["grad"]:
        out["grad_logits"] = torch.autograd.grad(w, leaf, s["grad_w"].double())[0]
    return out


def _exact_few(s, c):
    x, I = s["x"].double(), c["I"]
    out = torch.zeros(x.shape, dtype=torch.float64, device=x.device)
    for e in range(c["E"]):
        t, k = torch.nonzero(s["topk_idx"] == e, as_tuple=True)
        if not len(t):
            continue
        h = x[t] @ s["w13"][e].double().t().contiguous()
        gate, up = h[:, :I], h[:, I:]
        if c["act"] == "silu":
            a = torch.nn.functional.silu(gate)
        else:
            a = torch.nn.functional.gelu(gate, approximate="tanh")
        y = (a * up) @ s["w2"][e].double().t().contiguous()
        out.index_add_(0, t, y * s["topk_weights"][t, k].double().unsqueeze(1))
    return out


def _exact_lowrank(s, c):
    A = c["A"]
    x, base, a, b = (s[n].double() for n in ("x", "base", "a", "b"))
    w = s["weights"].double() if c["weights"] else torch.ones(c["T"], 1, dtype=torch.float64, device=x.device)
    ids = s["ids"].view(-1)
    out, gx, gw = base.clone(), torch.zeros_like(x), torch.zeros_like(w)
    ga, gb = torch.zeros_like(a), torch.zeros_like(b)
    for e in range(A):
        t = torch.nonzero(ids == e).view(-1)
        if not len(t):
            continue
        u = x[t] @ a[e].t().contiguous()
        out[t] += w[t] * (u @ b[e])
        if c["grad"]:
            g = s["grad_out"][t].double()
            back = g @ b[e].t().contiguous()
            gx[t] = (w[t] * back) @ a[e]
            ga[e] = (w[t] * back).t().contiguous() @ x[t]
            gb[e] = (w[t] * u).t().contiguous() @ g
            gw[t] = (back * u).sum(1, keepdim=True)
    if not c["grad"]:
        return out
    got = {"out": out, "grad_x": gx, "grad_a": ga, "grad_b": gb}
    return got | {"grad_w": gw} if c["weights"] else got
