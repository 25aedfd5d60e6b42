"""The router, the exchange, the few-token layer and the adapters as a program
runs them together: a training step through autograd, and a decode step in a
HIP graph."""
import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")


def make(T, H, E, K, I, A, r, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=n(T, H), gate=n(E, H) * H ** -0.5, w13=n(E, 2 * I, H) * H ** -0.5, w2=n(E, H, I) * I ** -0.5,
             a=n(A, r, H) * H ** -0.5, b=n(A, r, H) * r ** -0.5, g=n(T, H))
    d = {k: v.to(dtype).to(DEV) for k, v in d.items()}
    d["ids"] = torch.randint(0, A + 1, (T, 1), generator=g).to(torch.int32).to(DEV)
    return d


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_training_step_is_the_calls_in_order(dtype):
    """Router, dispatch, (one elementwise expert), combine and adapters beside it
    through autograd give bit for bit what the calls give one by one."""
    T, H, E, K, A, r = 200, 64, 16, 4, 5, 8
    d = make(T, H, E, K, 8, A, r, dtype, 1)
    logits = (d["x"].float() @ d["gate"].float().t().contiguous())
    leaf = {k: d[k].clone().requires_grad_() for k in ("x", "a", "b")}
    z = logits.clone().requires_grad_()
    idx, w = M.autograd.route(z, K, scale=1.5)
    h = M.moe_layout(idx, E, 1)
    recv, _ = M.autograd.dispatch(leaf["x"], None, h)
    y = recv * 2
    out = M.autograd.combine(y, w, h)
    ha = M.moe_layout(d["ids"], A + 1, 1)
    full = M.autograd.lowrank(leaf["x"], leaf["a"], leaf["b"], None, ha, out)
    full.backward(d["g"])

    idx2, w2 = M.moe_route(logits, K, scale=1.5)
    assert torch.equal(idx, idx2) and torch.equal(w, w2)
    h2 = M.moe_layout(idx2, E, 1)
    recv2, _ = M.moe_dispatch(h2, d["x"])
    y2 = recv2 * 2
    out2 = M.moe_combine(h2, y2, w2)
    ha2 = M.moe_layout(d["ids"], A + 1, 1)
    full2, u = M.moe_lowrank(ha2, d["x"], d["a"], d["b"], base=out2)
    assert torch.equal(full, full2)
    gx_a, ga, gb, _ = M.moe_lowrank_bwd(ha2, d["g"], d["x"], d["a"], d["b"], u)
    gy, gw = M.moe_combine_bwd(h2, d["g"], w2, y2, grad_w=True)
    gx_e, _ = M.moe_dispatch_bwd(h2, gy * 2)
    gz = M.moe_route_bwd(logits, idx2, gw, scale=1.5)
    assert torch.equal(leaf["a"].grad, ga) and torch.equal(leaf["b"].grad, gb)
    assert torch.equal(z.grad, gz)
    assert torch.equal(leaf["x"].grad, gx_a + gx_e) or torch.equal(leaf["x"].grad, gx_e + gx_a)


def test_decode_step_in_a_graph():
    """Router, few-token layer, adapter layout and adapters in one graph; each
    replay with new inputs against the eager calls, other work between."""
    T, H, E, K, I, A, r = 16, 256, 32, 4, 96, 6, 16
    d = make(T, H, E, K, I, A, r, torch.bfloat16, 2)
    logits = torch.randn(T, E, device=DEV)
    idx = torch.empty((T, K), dtype=torch.int32, device=DEV)
    w = torch.empty((T, K), device=DEV)
    few, out = torch.empty_like(d["x"]), torch.empty_like(d["x"])
    u = torch.empty((T, r), device=DEV)
    ws = torch.empty(M.moe_few_workspace_size(torch.bfloat16, T, K, I), dtype=torch.uint8, device=DEV)
    h = M.Handle()
    lws = torch.empty(M.moe_workspace_size(T, 1, A + 1, 1), dtype=torch.uint8, device=DEV)

    def step():
        M.moe_route(logits, K, topk_idx=idx, topk_weights=w)
        M.moe_few(d["x"], idx, w, d["w13"], d["w2"], out=few, workspace=ws)
        M.moe_layout(d["ids"], A + 1, 1, handle=h, workspace=lws)
        M.moe_lowrank(h, d["x"], d["a"], d["b"], base=few, out=out, u=u)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(4):
        new = make(T, H, E, K, I, A, r, torch.bfloat16, 10 + seed)
        d["x"].copy_(new["x"]), d["ids"].copy_(new["ids"]), logits.normal_()
        ri, rw = M.moe_route(logits, K)
        rf = M.moe_few(d["x"], ri, rw, d["w13"], d["w2"])
        ro, _ = M.moe_lowrank(M.moe_layout(d["ids"], A + 1, 1), d["x"], d["a"], d["b"], base=rf)
        torch.cuda.synchronize()
        for t in (idx, w, few, out, u, ws):
            t.fill_(0)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, ri) and torch.equal(w, rw) and torch.equal(few, rf) and torch.equal(out, ro)


def test_calls_on_another_stream_than_the_default():
    d = make(24, 128, 16, 4, 40, 3, 8, torch.bfloat16, 3)
    logits = torch.randn(24, 16, device=DEV)
    torch.cuda.synchronize()

    def chain():
        idx, w = M.moe_route(logits, 4)
        y = M.moe_few(d["x"], idx, w, d["w13"], d["w2"], activation="gelu_tanh")
        out, u = M.moe_lowrank(M.moe_layout(d["ids"], 4, 1), d["x"], d["a"], d["b"], base=y)
        return out

    ref = chain()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = chain()
    side.synchronize()
    assert torch.equal(got, ref)


def test_a_second_derivative_raises():
    d = make(24, 128, 16, 4, 40, 3, 8, torch.float32, 3)
    logits = torch.randn(24, 16, device=DEV, requires_grad=True)
    _, w = M.autograd.route(logits, 4, renormalize=False)
    g, = torch.autograd.grad((w * w).sum(), logits, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
    x = d["x"].clone().requires_grad_()
    out = M.autograd.lowrank(x, d["a"], d["b"], None, M.moe_layout(d["ids"], 4, 1))
    g, = torch.autograd.grad((out * out).sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


@pytest.mark.parametrize("T,A", [(48, 3), (4200, 1)])
def test_training_pass_in_a_graph(T, A):
    """Forward and backward of router and adapters captured together, replayed on new values."""
    E, K = 16, 4
    d = make(T, 128, E, K, 40, A, 16, torch.bfloat16, 5)
    h = M.moe_layout(d["ids"], A + 1, 1)
    base = torch.zeros_like(d["x"])
    gw = torch.randn(T, K, device=DEV)
    logits = torch.randn(T, E, device=DEV)
    static = [d["x"], d["a"], d["b"], base, logits]

    def step():
        x, a, b, c, z = (t.detach().requires_grad_() for t in static)
        _, w = M.autograd.route(z, K, renormalize=False)
        out = M.autograd.lowrank(x, a, b, None, h, c)
        return (out, w) + torch.autograd.grad((out, w), (x, a, b, c, z), (d["g"], gw))

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
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
