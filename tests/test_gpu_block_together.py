"""One expert block as a program runs it, from the norm before it to the norm of the next: a
training step through autograd, a prefill and a decode step in 8 bits, in a HIP graph and on
another stream."""
import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
BF16, F32 = torch.bfloat16, torch.float32


def make(T, H, E, I, dtype, seed, G=1):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=n(T, H), gate_w=n(E, H) * H ** -0.5, w13=n(E, 2 * I, H) * H ** -0.5, w2=n(E, H, I) * I ** -0.5,
             w_in=1 + 0.1 * n(H), w_out=1 + 0.1 * n(H), w_next=1 + 0.1 * n(H), gate=n(G, H), g_out=n(T, H), g_n=n(T, H))
    return {k: v.to(dtype).to(DEV) for k, v in d.items()}


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_training_step_is_the_calls_in_order(dtype):
    """Norm, router with its balance loss, exchange, (one elementwise expert) and the end of the block
    through autograd give bit for bit what the calls give one by one."""
    T, H, E, K, G = 240, 64, 16, 4, 6
    d = make(T, H, E, 8, dtype, 1, G)
    seq = torch.tensor([0, 100, 100, 240], dtype=torch.int32, device=DEV)
    mask = torch.rand(T, device=DEV) > 0.1
    gw = d["gate_w"].float().t().contiguous()
    coef = torch.tensor([0.01, 0.001], device=DEV)
    names = ("x", "w_in", "w_out", "w_next", "gate")
    leaf = {k: d[k].clone().requires_grad_() for k in names}
    n = M.autograd.prenorm(leaf["x"], leaf["w_in"])
    z = n.detach().float() @ gw
    z.requires_grad_()
    idx, w = M.autograd.route(z, K)
    loss, counts, probs, tokens = M.autograd.balance(z, idx, seq, mask)
    h = M.moe_layout(idx, E, 1)
    recv, _ = M.autograd.dispatch(n, None, h)
    y = M.autograd.combine(recv * 2, w, h)
    out, nn = M.autograd.postnorm(leaf["x"], y, leaf["w_out"], leaf["gate"], 0.5, leaf["w_next"])
    torch.autograd.backward([out, nn, loss], [d["g_out"], d["g_n"], coef])

    n2, r_in = M.moe_prenorm(d["x"], d["w_in"])
    z2 = n2.float() @ gw
    idx2, w2 = M.moe_route(z2, K)
    loss2, counts2, probs2, tokens2 = M.moe_balance(z2, idx2, seq, mask)
    h2 = M.moe_layout(idx2, E, 1)
    y2 = M.moe_dispatch(h2, n2)[0] * 2
    c2 = M.moe_combine(h2, y2, w2)
    kw = dict(weight=d["w_out"], gate=d["gate"], residual_scale=0.5, next_weight=d["w_next"])
    out2, nn2, rstd = M.moe_postnorm(d["x"], c2, **kw)
    assert all(torch.equal(a, b) for a, b in ((n, n2), (loss, loss2), (counts, counts2), (probs, probs2), (tokens, tokens2),
                                              (out, out2), (nn, nn2)))
    gx, gc, gwo, gg, gwn = M.moe_postnorm_bwd(d["g_out"], d["g_n"], d["x"], c2, rstd, **kw)
    gy, gwt = M.moe_combine_bwd(h2, gc, w2, y2, grad_w=True)
    gn, _ = M.moe_dispatch_bwd(h2, gy * 2)
    gx_in, gwi = M.moe_prenorm_bwd(gn, d["x"], r_in, d["w_in"])
    gz = M.moe_route_bwd(z2, idx2, gwt)
    gz = M.moe_balance_bwd(z2, counts2, tokens2, coef, K, seq, mask) + gz
    assert torch.equal(leaf["w_out"].grad, gwo) and torch.equal(leaf["gate"].grad, gg) and torch.equal(leaf["w_next"].grad, gwn)
    assert torch.equal(leaf["w_in"].grad, gwi) and torch.equal(leaf["x"].grad, gx + gx_in)
    assert torch.equal(z.grad, gz)
    # the residual's gradient added on the way: one rounding less, so not bit for bit in bfloat16
    one, _ = M.moe_prenorm_bwd(gn, d["x"], r_in, d["w_in"], grad_base=gx, grad_weight=False)
    eps = torch.finfo(dtype).eps
    size = gx.float().abs() + gx_in.float().abs()
    assert bool(((one.float() - (gx.float() + gx_in.float())).abs() <= eps * size + 1e-30).all())


def layer(d, q13, q2, idx, w, h, x, n=None, out=None, nn=None, bufs=None):
    """A block in 8 bits from x on."""
    b = bufs or {}
    q, s = M.moe_prenorm(x, d["w_in"], quantize=True, out=b.get("q"), scale=b.get("s"))
    M.moe_layout(idx, q13[0].shape[0], 1, handle=h, workspace=b.get("ws"))
    act = M.moe_matmul_i8(q, s, *q13, handle=h, tokens=True, activation="silu", out=b.get("act"))
    qa, sa = M.moe_quant_rows(act, q=b.get("qa"), scale=b.get("sa"))
    y = M.moe_matmul_i8(qa, sa, *q2, handle=h, out=b.get("y"))
    return M.moe_postnorm(x, y, d["w_out"], d["gate"], 0.5, d["w_next"], handle=h, topk_weights=w, out=out, n=nn, rstd=b.get("rstd"))


@pytest.mark.parametrize("T", [1, 16, 300])
def test_a_block_in_8_bits_is_near_the_block_itself(T):
    """Against float64 on the same rows.  A row's or channel's value moves by at most half a step,
    amax / 254, in each of the four roundings, of which a product's error is the sum; with normal
    values amax is below 6 standard deviations, so a product of width n is off by about
    6 / 254 sqrt(2 n / 3) of its terms' size, 2% of its own; twice, and through gate and up: below 6%."""
    H, E, K, I = 256, 8, 2, 128
    d = make(T, H, E, I, BF16, T)
    q13, q2 = M.moe_quant_rows(d["w13"]), M.moe_quant_rows(d["w2"])
    z = torch.randn(T, E, device=DEV)
    idx, w = M.moe_route(z, K)
    out, nn, _ = layer(d, q13, q2, idx, w, M.Handle(), d["x"])
    f = {k: v.cpu().double() for k, v in d.items()}
    rms = lambda v: v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)  # noqa: E731
    n = rms(f["x"]) * f["w_in"]
    y = torch.zeros(T, H, dtype=torch.float64)
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k])
            gu = f["w13"][e] @ n[t]
            a = gu[:I] / (1 + torch.exp(-gu[:I])) * gu[I:]
            y[t] += float(w[t, k]) * (f["w2"][e] @ a)
    y = rms(y) * f["w_out"] * f["gate"]
    ref = 0.5 * f["x"] + y
    assert float((out.cpu().double() - ref).norm() / y.norm()) < 0.06
    assert float((nn.cpu().double() - rms(ref) * f["w_next"]).norm() / nn.double().norm()) < 0.06


@pytest.mark.parametrize("T,E,K", [(16, 32, 4), (1, 16, 2), (400, 8, 2)])
def test_a_block_in_a_graph(T, E, K):
    """Everything in one graph; each replay with new inputs against the eager calls, other work between."""
    H, I = 128, 64
    d = make(T, H, E, I, BF16, 2)
    q13, q2 = M.moe_quant_rows(d["w13"]), M.moe_quant_rows(d["w2"])
    logits = torch.randn(T, E, device=DEV)
    idx, w = M.moe_route(logits, K)
    h = M.Handle()
    new = lambda *s, dtype=BF16: torch.empty(s, dtype=dtype, device=DEV)  # noqa: E731
    b = dict(q=new(T, H, dtype=torch.int8), s=new(T, dtype=F32), act=new(T * K, I), qa=new(T * K, I, dtype=torch.int8),
             sa=new(T * K, dtype=F32), y=new(T * K, H), rstd=new(T, 2, dtype=F32),
             ws=new(M.moe_workspace_size(T, K, E, 1), dtype=torch.uint8))
    out, nn = new(T, H), new(T, H)
    loss, counts, probs, tokens = new(2, dtype=F32), new(1, E, dtype=torch.int32), new(1, E, dtype=F32), new(1, dtype=torch.int32)
    bws = new(M.moe_balance_workspace_size(T, E), dtype=torch.uint8)

    def step():
        M.moe_route(logits, K, topk_idx=idx, topk_weights=w)
        M.moe_balance(logits, idx, loss=loss, counts=counts, probs=probs, tokens=tokens, workspace=bws)
        layer(d, q13, q2, idx, w, h, d["x"], out=out, nn=nn, bufs=b)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        torch.manual_seed(seed)
        d["x"].normal_(), logits.normal_()
        ri, rw = M.moe_route(logits, K)
        rb = M.moe_balance(logits, ri)
        ro, rn, _ = layer(d, q13, q2, ri, rw, M.Handle(), d["x"])
        torch.cuda.synchronize()
        for t in list(b.values()) + [out, nn, loss, counts, probs, tokens, bws]:
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ro) and torch.equal(nn, rn)
        assert all(torch.equal(p, q) for p, q in zip((loss, counts, probs, tokens), rb))


def test_training_pass_in_a_graph():
    """Forward and backward of the norms and the balance loss captured together, replayed on new values."""
    T, H, E, K, G = 1100, 96, 24, 3, 11
    d = make(T, H, E, 8, BF16, 3, G)
    static = [d["x"], torch.randn_like(d["x"]), d["w_in"], d["w_out"], d["gate"], d["w_next"], torch.randn(T, E, device=DEV)]
    idx = torch.randint(0, E, (T, K), device=DEV, dtype=torch.int32)
    coef = torch.tensor([0.01, 0.001], device=DEV)

    def step():
        x, y, wi, wo, gate, wn, z = (t.detach().requires_grad_() for t in static)
        n = M.autograd.prenorm(x, wi)
        out, nn = M.autograd.postnorm(n, y, wo, gate, 0.5, wn)
        loss, _, _, _ = M.autograd.balance(z, idx)
        return (out, nn, loss) + torch.autograd.grad((out, nn, loss), (x, y, wi, wo, gate, wn, z), (d["g_out"], d["g_n"], coef))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in range(3):
        torch.manual_seed(seed)
        for t in static:
            t.normal_()
        ref = step()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, ref))


def test_calls_on_another_stream_than_the_default():
    T, H, E, K, I = 90, 128, 16, 4, 64
    d = make(T, H, E, I, BF16, 4)
    q13, q2 = M.moe_quant_rows(d["w13"]), M.moe_quant_rows(d["w2"])
    logits = torch.randn(T, E, device=DEV)
    torch.cuda.synchronize()

    def chain():
        idx, w = M.moe_route(logits, K)
        loss, counts, probs, tokens = M.moe_balance(logits, idx)
        gz = M.moe_balance_bwd(logits, counts, tokens, loss, K)
        out, nn, rstd = layer(d, q13, q2, idx, w, M.Handle(), d["x"])
        return (loss, gz, out, nn) + M.moe_postnorm_bwd(d["g_out"], d["g_n"], d["x"], out, rstd, d["w_out"], d["gate"],
                                                        next_weight=d["w_next"])

    ref = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = chain()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, ref))


def test_a_second_derivative_raises():
    d = make(10, 64, 4, 8, F32, 5)
    x = d["x"].clone().requires_grad_()
    for out in (M.autograd.prenorm(x, d["w_in"]), M.autograd.postnorm(x, d["g_n"], d["w_out"]),
                M.autograd.balance(x, torch.zeros(10, 1, dtype=torch.int32, device=DEV))[0]):
        g, = torch.autograd.grad((out * out).sum(), x, create_graph=True)
        with pytest.raises(RuntimeError):
            g.sum().backward()


def test_gradients_where_only_some_are_needed():
    """Leaves that need none, outputs that nobody used."""
    d = make(30, 64, 4, 8, BF16, 6, 3)
    y, wo = d["g_n"].clone().requires_grad_(), d["w_out"].clone().requires_grad_()
    out, nn = M.autograd.postnorm(d["x"], y, wo, d["gate"], 0.5, d["w_next"])
    out.backward(d["g_out"])
    _, _, rstd = M.moe_postnorm(d["x"], d["g_n"], d["w_out"], d["gate"], 0.5, d["w_next"])
    ref = M.moe_postnorm_bwd(d["g_out"], None, d["x"], d["g_n"], rstd, d["w_out"], d["gate"], 0.5, d["w_next"])
    assert torch.equal(y.grad, ref[1]) and torch.equal(wo.grad, ref[2])
    gate = d["gate"].clone().requires_grad_()
    only = M.autograd.postnorm(d["x"], d["g_n"], None, gate)
    assert torch.is_tensor(only)
    only.backward(d["g_out"])
    assert gate.grad.shape == gate.shape
    x = d["x"].clone().requires_grad_()
    n = M.autograd.prenorm(x, d["w_in"])
    n.backward(d["g_n"].t().contiguous().t())  # a gradient of other strides
    assert x.grad.shape == x.shape
