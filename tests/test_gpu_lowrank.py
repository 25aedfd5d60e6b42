"""Low-rank adapters and their gradients against the formulas in float64.

Bounds, with u = 2^-24 and n terms of a float32 sum in any order off by n u
times the sum of magnitudes.  A rank-space value s (u, raw, gu) from rows of W
terms: ds = W u sum|bank||row|, one more product by w.  Where it is an operand
of a bfloat16 instruction its two halves leave (eps/2)^2 = 2^-16 of it, and
the sum has twice the terms.  The result is rounded once: eps/2 for bfloat16,
u for float32 (with the addition of the base).
"""
import math

import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def make(T, A, r, H, N, dtype, seed, weights=True, none=0.2, E=None):
    g = torch.Generator().manual_seed(seed)
    E = E or A + 1
    ids = torch.randint(0, A, (T, 1), generator=g)
    ids = torch.where(torch.rand(T, 1, generator=g) < none, torch.randint(A, E, (T, 1), generator=g) if E > A else ids, ids)
    d = dict(x=torch.randn(T, H, generator=g).to(dtype), a=(torch.randn(A, r, H, generator=g) * H ** -0.5).to(dtype),
             b=(torch.randn(A, r, N, generator=g) * r ** -0.5).to(dtype), base=torch.randn(T, N, generator=g).to(dtype),
             g=torch.randn(T, N, generator=g).to(dtype), gbase=torch.randn(T, H, generator=g).to(dtype),
             w=torch.randn(T, 1, generator=g) if weights else None)
    d = {k: None if v is None else v.to(DEV) for k, v in d.items()}
    return ids.to(torch.int32).to(DEV), E, d


def reference(ids, d, with_base=True, with_gbase=True):
    """{name: (value, bound)} in float64 on the CPU."""
    dtype = d["x"].dtype
    half = torch.finfo(dtype).eps / 2
    split = 2.0 ** -16 if dtype == BF16 else 0.0
    c = {k: None if v is None else v.cpu().double() for k, v in d.items()}
    T, H = c["x"].shape
    A, r, N = c["b"].shape
    w = c["w"] if c["w"] is not None else torch.ones(T, 1, dtype=torch.float64)
    ids = ids.cpu().view(-1)
    z = lambda *s: torch.zeros(*s, dtype=torch.float64)  # noqa: E731
    out = c["base"].clone() if with_base else z(T, N)
    gx = c["gbase"].clone() if with_gbase else z(T, H)
    ga, gb, gw = z(A, r, H), z(A, r, N), z(T, 1)
    to, tx, ta, tb, tw = z(T, N), z(T, H), z(A, r, H), z(A, r, N), z(T, 1)
    for e in range(A):
        t = torch.nonzero(ids == e).view(-1)
        n = len(t)
        if not n:
            continue
        a, b, x, g, wt = c["a"][e], c["b"][e], c["x"][t], c["g"][t], w[t]
        u, du = x @ a.t(), H * U * (x.abs() @ a.abs().t())
        raw, draw = g @ b.t(), N * U * (g.abs() @ b.abs().t())
        wu, gu = wt * u, wt * raw
        dwu = wt.abs() * du + 2 * U * wu.abs() + split * wu.abs()
        dgu = wt.abs() * draw + 2 * U * gu.abs() + split * gu.abs()
        out[t] += wu @ b
        to[t] = dwu @ b.abs() + (2 * r + 2) * U * (wu.abs() @ b.abs())
        gx[t] += gu @ a
        tx[t] = dgu @ a.abs() + (2 * r + 2) * U * (gu.abs() @ a.abs())
        ga[e] = gu.t() @ x
        ta[e] = dgu.t() @ x.abs() + (2 * n + 8) * U * (gu.abs().t() @ x.abs())
        gb[e] = wu.t() @ g
        tb[e] = dwu.t() @ g.abs() + (2 * n + 8) * U * (wu.abs().t() @ g.abs())
        gw[t] = (raw * u).sum(1, keepdim=True)
        tw[t] = ((draw * (u.abs() + du) + raw.abs() * du) + (r + 4) * U * (raw * u).abs()).sum(1, keepdim=True)
    done = lambda v, tol: (v, tol + half * (v.abs() + tol) + U * v.abs() + 1e-37)  # noqa: E731
    return dict(out=done(out, to), grad_x=done(gx, tx), grad_a=done(ga, ta), grad_b=done(gb, tb), grad_w=(gw, tw + 1e-37))


def near(got, ref, what):
    v, tol = ref
    err = (got.cpu().double() - v).abs()
    assert got.shape == v.shape and bool((err <= tol).all()), (what, float((err - tol).max()))


def check(ids, E, d, pad=1):
    h = M.moe_layout(ids, E, 1, handle=M.Handle(pad_multiple=pad))
    ref = reference(ids, d)
    u0 = torch.full((h.R, d["a"].shape[1]), math.nan, device=DEV)
    out, u = M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"], u=u0)
    near(out, ref["out"], "out")
    assert not torch.isnan(u[:int(h.field("expert_offset")[-1])]).any()  # every row is written
    got = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_base=d["gbase"], grad_w=True)
    for n, t in zip(("grad_x", "grad_a", "grad_b", "grad_w"), got):
        near(t, ref[n], n)
    # without grad_w, whose sum over the rank the others need not wait for
    for n, t in zip(("grad_x", "grad_a", "grad_b"), M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_base=d["gbase"])):
        near(t, ref[n], n)
    assert h.check() == 0
    return h, u, out, got


SHAPES = [(1, 1, 8, 64, 64), (1, 40, 16, 2048, 96), (3, 2, 8, 8, 8), (17, 3, 24, 136, 264), (64, 32, 16, 256, 512),
          (100, 7, 40, 1000, 72), (333, 5, 64, 520, 1032), (1000, 1, 128, 128, 192), (257, 200, 8, 64, 40),
          (2000, 11, 32, 264, 136), (50, 1000, 16, 32, 24), (130, 4, 72, 96, 4096), (77, 6, 96, 168, 64),
          (60, 3, 128, 64, 72), (500, 9, 32, 520, 264), (18, 900, 16, 128, 1032), (200, 2, 120, 40, 328)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,A,r,H,N", SHAPES)
def test_every_output_against_the_formulas(dtype, T, A, r, H, N):
    ids, E, d = make(T, A, r, H, N, dtype, T + A + r)
    check(ids, E, d)


@pytest.mark.parametrize("T,A,r,H,N", [(19, 3, 4, 12, 20), (65, 2, 12, 612, 36), (40, 5, 20, 4, 4), (9, 4, 124, 44, 1028)])
def test_float32_chunks_of_four(T, A, r, H, N):
    ids, E, d = make(T, A, r, H, N, F32, T)
    check(ids, E, d)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,A,r,H,N", [(8200, 5, 16, 40, 4104), (8209, 700, 40, 264, 72), (9000, 3, 24, 1032, 2056)])
def test_large_batches(dtype, T, A, r, H, N):
    """Several tiles a workgroup or wave: tiles that adapters share among them."""
    ids, E, d = make(T, A, r, H, N, dtype, T)
    check(ids, E, d)


@pytest.mark.parametrize("pad", [2, 16, 100])
def test_padded_layouts(pad):
    ids, E, d = make(150, 6, 16, 72, 136, BF16, pad, E=9)
    check(ids, E, d, pad)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_all_none_one_adapter_and_sorted(dtype):
    ids, E, d = make(90, 4, 16, 64, 80, dtype, 1)
    for fill in (4, 2):
        ids[:] = fill
        _, _, out, (gx, ga, gb, gw) = check(ids, E, d)
        if fill == 4:  # nobody has an adapter
            assert torch.equal(out, d["base"]) and torch.equal(gx, d["gbase"])
            assert (ga == 0).all() and (gb == 0).all() and (gw == 0).all()
    ids[:] = torch.arange(90, device=DEV).view(-1, 1) // 23
    check(ids, E, d)


def far_check(name, got, ref, mag, terms, dtype=BF16):
    """got against ref (float64, on the GPU): terms * U of the sum of magnitudes,
    the halves' 2^-16 of it, and the result's rounding."""
    tol = mag * (2 * terms * U + 2.0 ** -16) + (torch.finfo(dtype).eps / 2 + U) * ref.abs() + 1e-30
    tol = tol * (1 + torch.finfo(dtype).eps)
    assert bool(((got.double() - ref).abs() <= tol).all()), name


@pytest.mark.parametrize("wide", ["x", "out"])
def test_rows_past_two_gib(wide):
    """More wide rows than 32-bit offsets reach, on either side; every element is
    checked, in blocks of tokens, with float64 on the GPU."""
    T, A, r = 70000, 3, 8
    H, N = (16392, 64) if wide == "x" else (64, 16392)
    assert T * max(H, N) * 2 > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(1)
    new = lambda *s: torch.empty(s, dtype=BF16, device=DEV).normal_(generator=g)  # noqa: E731
    x, base, go = new(T, H), new(T, N), new(T, N)
    a, b = new(A, r, H) * H ** -0.5, new(A, r, N) * r ** -0.5
    ids = torch.randint(0, A + 1, (T, 1), generator=g, device=DEV).to(torch.int32)
    h = M.moe_layout(ids, A + 1, 1)
    out, u = M.moe_lowrank(h, x, a, b, base=base)
    gx, ga, gb, gw = M.moe_lowrank_bwd(h, go, x, a, b, u, grad_w=True)
    ad, bd = a.double(), b.double()
    ra, rb = torch.zeros_like(ad), torch.zeros_like(bd)
    ma, mb = torch.zeros_like(ad), torch.zeros_like(bd)
    for t0 in range(0, T, 5000):
        t1 = min(t0 + 5000, T)
        i, xs, gs = ids[t0:t1].view(-1), x[t0:t1].double(), go[t0:t1].double()
        for e in range(A):
            k = torch.nonzero(i == e).view(-1)
            xe, ge = xs[k], gs[k]
            at, bt = ad[e].t().contiguous(), bd[e].t().contiguous()
            ue, re = xe @ at, ge @ bt
            um, rm = xe.abs() @ at.abs(), ge.abs() @ bt.abs()
            far_check("out", out[t0:t1][k], base[t0:t1][k].double() + ue @ bd[e], um @ bd[e].abs(), H + r)
            far_check("grad_x", gx[t0:t1][k], re @ ad[e], rm @ ad[e].abs(), N + r)
            far_check("grad_w", gw[t0:t1].view(-1)[k], (ue * re).sum(1), (um * rm).sum(1), H + N + r, F32)
            ra[e] += re.t().contiguous() @ xe
            ma[e] += rm.t().contiguous() @ xe.abs()
            rb[e] += ue.t().contiguous() @ ge
            mb[e] += um.t().contiguous() @ ge.abs()
        none = i == A
        assert torch.equal(out[t0:t1][none], base[t0:t1][none]) and (gx[t0:t1][none] == 0).all()
    far_check("grad_a", ga, ra, ma, N + T)
    far_check("grad_b", gb, rb, mb, H + T)


def test_without_weights_and_base_and_in_place():
    ids, E, d = make(70, 5, 16, 136, 72, BF16, 2, weights=False)
    h = M.moe_layout(ids, E, 1)
    ref = reference(ids, d, with_base=False, with_gbase=False)
    out, u = M.moe_lowrank(h, d["x"], d["a"], d["b"])
    near(out, ref["out"], "out")
    gx, ga, gb, gw = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u)
    near(gx, ref["grad_x"], "grad_x")
    assert gw is None
    only = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, grad_x=False, grad_a=False, grad_w=True)
    assert only[0] is None and only[1] is None and torch.equal(only[2], gb)
    near(only[3], ref["grad_w"], "grad_w")
    # in place: out on base, grad_x on grad_base
    base, gbase = d["base"].clone(), d["gbase"].clone()
    full, u2 = M.moe_lowrank(h, d["x"], d["a"], d["b"], base=d["base"])
    M.moe_lowrank(h, d["x"], d["a"], d["b"], base=base, out=base)
    assert torch.equal(base, full) and torch.equal(u2, u)
    want = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, grad_base=d["gbase"])[0]
    M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, grad_base=gbase, grad_x=gbase)
    assert torch.equal(gbase, want)


def test_nothing_leaks_between_tokens_and_adapters():
    ids, E, d = make(100, 8, 16, 64, 72, BF16, 4, none=0.0)
    ids[ids == 3] = 2        # adapter 3 has no token
    ids[40] = 8              # token 40 has no adapter
    h = M.moe_layout(ids, E, 1)
    ref, u = M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"])
    rgx, rga, rgb, _ = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"])
    d["a"][3], d["b"][3] = math.nan, math.inf
    d["x"][40] = math.nan
    d["x"][41] = math.inf
    d["g"][40], d["g"][41] = math.nan, math.nan
    got, u = M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"])
    gx, ga, gb, _ = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"])
    keep = [t for t in range(100) if t != 41]
    assert torch.equal(got[keep], ref[keep]) and torch.equal(gx[keep], rgx[keep])
    other = [e for e in range(8) if e != int(ids[41])]
    assert torch.equal(ga[other], rga[other]) and torch.equal(gb[other], rgb[other])


def test_gradients_against_differences():
    """Central differences of the float64 formula along random directions.  It is
    linear in each argument, so a difference is exact but for float64 rounding
    (1e-12 of its terms here); the kernel's side is bound as in the module text."""
    ids, E, d = make(30, 3, 8, 32, 40, F32, 6)
    h, u, out, got = check(ids, E, d)
    g = torch.Generator().manual_seed(0)
    c = {k: v.cpu().double() for k, v in d.items()}
    flat = ids.cpu().view(-1).long()

    def value(c):
        y = torch.zeros(30, 40, dtype=torch.float64)
        for t in range(30):
            if flat[t] < 3:
                y[t] = c["w"][t] * ((c["a"][flat[t]] @ c["x"][t]) @ c["b"][flat[t]])
        return (y * c["g"]).sum()

    ref = reference(ids, d, with_gbase=False)
    plain = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_w=True)
    for name, n, t in (("x", "grad_x", plain[0]), ("a", "grad_a", plain[1]), ("b", "grad_b", plain[2]), ("w", "grad_w", plain[3])):
        v = torch.randn(c[name].shape, generator=g, dtype=torch.float64)
        up, down = dict(c), dict(c)
        up[name], down[name] = c[name] + v, c[name] - v
        slope = (value(up) - value(down)) / 2
        mine = (t.cpu().double() * v).sum()
        assert abs(float(slope - mine)) <= float((ref[n][1] * v.abs()).sum()) + 1e-9, name


def test_autograd_matches_the_calls_and_refuses_a_stale_layout():
    ids, E, d = make(60, 4, 16, 64, 72, BF16, 8)
    h = M.moe_layout(ids, E, 1)
    leaves = {k: d[k].clone().requires_grad_() for k in ("x", "a", "b", "w", "base")}
    out = M.autograd.lowrank(leaves["x"], leaves["a"], leaves["b"], leaves["w"], h, leaves["base"])
    out.backward(d["g"])
    ref, u = M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"])
    assert torch.equal(out, ref)
    got = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_w=True)
    for k, t in zip(("x", "a", "b", "w"), got):
        assert torch.equal(leaves[k].grad, t), k
    assert torch.equal(leaves["base"].grad, d["g"])
    # only the adapters learn
    a2 = d["a"].clone().requires_grad_()
    M.autograd.lowrank(d["x"], a2, d["b"], None, h, d["base"]).sum().backward()
    assert a2.grad is not None
    out = M.autograd.lowrank(leaves["x"], leaves["a"], leaves["b"], None, h)
    M.moe_layout(ids, E, 1, handle=h)
    with pytest.raises(M.autograd.StaleLayoutError):
        out.sum().backward()


def test_empty_batch():
    ids, E, d = make(5, 3, 8, 16, 24, BF16, 1)
    h = M.moe_layout(ids[:0], E, 1)
    out, u = M.moe_lowrank(h, d["x"][:0], d["a"], d["b"], base=d["base"][:0])
    assert out.shape == (0, 24) and u.shape == (0, 8)
    ga = torch.full_like(d["a"], 5)
    gx, ga, gb, _ = M.moe_lowrank_bwd(h, d["g"][:0], d["x"][:0], d["a"], d["b"], u, grad_a=ga)
    assert gx.shape == (0, 16) and (ga == 0).all() and (gb == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,A,r,H,N,pad", [(4100, 1, 16, 136, 264, 1), (9001, 2, 40, 72, 520, 1), (5000, 3, 24, 64, 128, 16),
                                           (17000, 1, 64, 24, 40, 1)])
def test_gradients_summed_in_parts(dtype, T, A, r, H, N, pad):
    """Long segments of few adapters: one adapter has nearly all tokens, the last
    none; with the workspace for parts, one short of it, and the smallest."""
    ids, E, d = make(T, A, r, H, N, dtype, 6, E=A + 2)
    if A > 1:
        few = (ids == 1) & (torch.arange(T, device=DEV).view(-1, 1) % 50 != 0)
        ids[few] = 0
        ids[ids == A - 1] = A
    h = M.moe_layout(ids, E, 1, handle=M.Handle(pad_multiple=pad))
    ref = reference(ids, d)
    _, u = M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"])
    n = M.moe_lowrank_bwd_workspace_size(h, dtype, H, N, A, r) // 4
    assert n > h.R * r  # there are parts
    ws = torch.full((n + 4,), math.nan, device=DEV)
    for size in (n, n - 4, h.R * r):
        for want in ((None, None), (None, False), (False, None)):
            ws.fill_(math.nan)
            got = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_x=False, grad_a=want[0],
                                    grad_b=want[1], workspace=ws[:size])
            for name, t, w in zip(("grad_a", "grad_b"), got[1:3], want):
                if w is None:
                    near(t, ref[name], name)
            assert torch.isnan(ws[size:]).all()
    one = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"])
    two = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"])
    assert all(torch.equal(p, q) for p, q in zip(one[:3], two[:3]))


@pytest.mark.parametrize("T", [40, 3000])
@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ids_outside_the_layout_touch_no_other_token(dtype, T):
    ids, E, d = make(T, 6, 16, 256, 264, dtype, 8)
    h = M.Handle()
    M.moe_layout(ids, E, 1, handle=h)  # leaves every row's token behind
    bad = ids.clone()
    off = torch.arange(T, device=DEV) % 3 == 0
    bad[off] = E
    bad[0] = -1
    M.moe_layout(bad, E, 1, handle=h)
    ref = reference(torch.where(off.view(-1, 1), E, ids), d)
    out, gx = torch.full_like(d["base"], 7), torch.full_like(d["x"], 7)
    gw = torch.full((T, 1), 7.0, device=DEV)
    _, u = M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"], out=out)
    _, ga, gb, _ = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_base=d["gbase"], grad_x=gx, grad_w=gw)
    keep = ~off.cpu()
    for n, t in (("out", out), ("grad_x", gx), ("grad_w", gw)):
        near(t[~off], tuple(v[keep] for v in ref[n]), n)
        assert (t[off] == 7).all()
    near(ga, ref["grad_a"], "grad_a")
    near(gb, ref["grad_b"], "grad_b")


def test_results_repeat_and_neighbours_stay():
    ids, E, d = make(700, 6, 32, 264, 520, BF16, 3)
    h, u, out, got = check(ids, E, d)
    buf = torch.full((704, 520), 3.0, dtype=BF16, device=DEV)
    for _ in range(4):
        M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"], out=buf[2:702])
        assert torch.equal(buf[2:702], out) and (buf[:2] == 3).all() and (buf[702:] == 3).all()
        again = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_base=d["gbase"], grad_w=True)
        assert all(torch.equal(p, q) for p, q in zip(got, again))


def test_graph_replays_with_new_ids():
    ids, E, d = make(48, 8, 16, 256, 264, BF16, 5)
    h = M.Handle()
    ws = torch.empty(M.moe_workspace_size(48, 1, E, 1), dtype=torch.uint8, device=DEV)
    out, u = torch.empty_like(d["base"]), torch.empty((48, 16), device=DEV)
    gx, ga, gb = torch.empty_like(d["x"]), torch.empty_like(d["a"]), torch.empty_like(d["b"])
    gu = torch.empty((48, 16), device=DEV)

    def step():
        M.moe_layout(ids, E, 1, handle=h, workspace=ws)
        M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"], out=out, u=u)
        M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_x=gx, grad_a=ga, grad_b=gb, workspace=gu)

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
        ids2, _, d2 = make(48, 8, 16, 256, 264, BF16, 60 + seed)
        ids.copy_(ids2)
        for k in ("x", "g", "base", "w"):
            d[k].copy_(d2[k])
        h2 = M.moe_layout(ids, E, 1)
        ro, ru = M.moe_lowrank(h2, d["x"], d["a"], d["b"], d["w"], base=d["base"])
        rg = M.moe_lowrank_bwd(h2, d["g"], d["x"], d["a"], d["b"], ru, d["w"])
        torch.cuda.synchronize()
        for t in (out, u, gx, ga, gb, gu):
            t.fill_(9)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ro) and torch.equal(gx, rg[0]) and torch.equal(ga, rg[1]) and torch.equal(gb, rg[2])


def test_refusals():
    ids, E, d = make(10, 3, 8, 16, 24, F32, 1)
    x, a, b = d["x"], d["a"], d["b"]
    h = M.moe_layout(ids, E, 1)
    with pytest.raises(M.MoeError) as e:  # two adapters a token
        M.moe_lowrank(M.moe_layout(ids.view(5, 2).contiguous(), E, 1), x[:5], a, b)
    assert e.value.code == -2
    with pytest.raises(M.MoeError) as e:  # more adapters than the layout has ids
        M.moe_lowrank(M.moe_layout(ids.clamp(max=1), 2, 1), x, a, b)
    assert e.value.code == -2
    wide = torch.zeros(3, 132, 16, device=DEV)
    with pytest.raises(M.MoeError) as e:
        M.moe_lowrank(h, x, wide, torch.zeros(3, 132, 24, device=DEV))
    assert e.value.code == -3
    with pytest.raises(M.MoeError) as e:
        M.moe_lowrank(h, x, torch.zeros(3, 6, 16, device=DEV), torch.zeros(3, 6, 24, device=DEV))
    assert e.value.code == -2
    with pytest.raises(RuntimeError, match="no layout"):
        M.moe_lowrank(M.Handle(), x, a, b)
    for bad in (lambda: M.moe_lowrank(h, x[:9], a, b), lambda: M.moe_lowrank(h, x, a[:2], b),
                lambda: M.moe_lowrank(h, x, a.to(BF16), b), lambda: M.moe_lowrank(h, x, a, b, torch.ones(10, device=DEV)),
                lambda: M.moe_lowrank(h, x, a, b, base=d["base"].t().contiguous().t()),
                lambda: M.moe_lowrank_bwd(h, d["g"], x, a, b, torch.zeros(9, 8, device=DEV))):
        with pytest.raises(ValueError):
            bad()
    _, u = M.moe_lowrank(h, x, a, b)
    with pytest.raises(M.MoeError) as e:
        M.moe_lowrank_bwd(h, d["g"], x, a, b, u, workspace=torch.empty(8, device=DEV))
    assert e.value.code == -5
    with pytest.raises(M.MoeError) as e:
        M.moe_lowrank_bwd(h, d["g"], x, a, b, u, grad_x=False, grad_a=False, grad_b=False)
    assert e.value.code == -1


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,A,r,H,N", [(3, 2, 32, 64, 72), (40, 3, 32, 2048, 2048), (200, 2, 64, 1040, 2056),
                                       (1100, 1, 128, 264, 264), (8300, 2, 32, 136, 136)])
def test_every_bit_of_the_rank_space_counts(dtype, T, A, r, H, N):
    """Ranks (and rows) in pairs with the values 1 + 2^-9 + 2^-s and 1 + 2^-9, s = 10
    ... 23, subtracted by the second product, which leaves exactly 2^-s.  Every step
    is exact: the values in rank space have three terms with 24 bits between them,
    sums of the rest one or two that are not zero; the results, powers of two, need
    no rounding.  One launch, two, and several tiles a wave."""
    steps = list(range(10, 24))
    n = len(steps)
    wide = torch.tensor([2.0 ** (4 - s) for s in steps])

    def pairs(W):  # [r, W]: rows 2k and 2k + 1 give 1 + 2^-9 + 2^-s_k and 1 + 2^-9 on the row `probe`
        m = torch.zeros(r, W)
        m[:2 * n, 0], m[:2 * n, 2] = 1.0, 2.0 ** -5
        m[0:2 * n:2, 1] = wide
        return m

    def probe(W):
        v = torch.zeros(T, W)
        v[:, 0], v[:, 1], v[:, 2] = 1.0, 2.0 ** -4, 2.0 ** -4
        return v

    def minus(W):  # [r, W]: column k is rank 2k minus rank 2k + 1
        m = torch.zeros(r, W)
        m[torch.arange(0, 2 * n, 2), torch.arange(n)] = 1.0
        m[torch.arange(1, 2 * n, 2), torch.arange(n)] = -1.0
        return m

    dev = lambda t: t.to(dtype).to(DEV)  # noqa: E731
    bank = lambda m: dev(m.expand(A, *m.shape)).contiguous()  # noqa: E731
    ids = (torch.arange(T) % A).to(torch.int32).view(T, 1).to(DEV)
    h = M.moe_layout(ids, A, 1)
    left = torch.tensor([2.0 ** -s for s in steps])
    # forward: out = u b
    out, u = M.moe_lowrank(h, dev(probe(H)), bank(pairs(H)), bank(minus(N)))
    assert torch.equal(out.cpu().float()[:, :n], left.expand(T, n)) and (out[:, n:] == 0).all()
    # backward: grad_x = gu a
    gx, _, _, _ = M.moe_lowrank_bwd(h, dev(probe(N)), dev(probe(H)), bank(minus(H)), bank(pairs(N)), u, grad_a=False,
                                    grad_b=False)
    assert torch.equal(gx.cpu().float()[:, :n], left.expand(T, n)) and (gx[:, n:] == 0).all()
    # two tokens of adapter 0 whose rows cancel: a weight of 1 + 2^-9 + 2^-s
    # against one of 1 + 2^-9 for grad_a and grad_b, at rank k
    for k, s in ((0, 10), (5, 18), (11, 20), (14, 23)):
        x, g = torch.zeros(T, H), torch.zeros(T, N)
        w = torch.full((T, 1), 1.0 + 2.0 ** -9)
        last = (T - 1) // A * A  # the last token of adapter 0
        x[0, 0], x[last, 0], g[0, 0], g[last, 0] = 1.0, -1.0, 1.0, 1.0
        w[0] += 2.0 ** -s
        ones = torch.zeros(r, 1)
        ones[k] = 1.0
        a, b = torch.zeros(r, H), torch.zeros(r, N)
        a[:, :1], b[:, :1] = ones, ones
        _, u = M.moe_lowrank(h, dev(x), bank(a), bank(b), w.to(DEV))
        _, ga, gb, _ = M.moe_lowrank_bwd(h, dev(g), dev(x), bank(a), bank(b), u, w.to(DEV), grad_x=False)
        for got in (ga, gb):
            want = torch.zeros(got.shape)
            want[0, k, 0] = 2.0 ** -s
            assert torch.equal(got.cpu().float(), want), (k, s)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,A,r,H,N", [(1, 1, 8, 64, 64), (40, 3, 16, 264, 520), (200, 3, 40, 1000, 72), (1030, 2, 128, 2056, 2064),
                                       (4100, 1, 16, 136, 264), (8300, 2, 64, 136, 136)])
def test_infinities_where_they_count(dtype, T, A, r, H, N):
    """Single infinities in chosen banks, in rows and in the output's gradient come
    out as the formulas in float64 have them; everything finite stays within its
    bound."""
    for where in ("a", "b", "x", "g", "all"):
        ids, E, d = make(T, A, r, H, N, dtype, T + r, none=0.0, E=A + 1)
        last = int(ids[T - 1])
        if where in ("b", "all"):
            d["b"][last, 3, 5], d["b"][int(ids[0]), r - 1, N - 1] = math.inf, -math.inf
        if where in ("a", "all"):
            d["a"][int(ids[0]), 1, 2], d["a"][last, 2, H - 1] = -math.inf, math.inf
        if where in ("x", "all"):
            d["x"][T // 2, 7] = math.inf
        if where in ("g", "all"):
            d["g"][T // 3, N - 2] = -math.inf
        ref = reference(ids, d)
        h = M.moe_layout(ids, E, 1)
        out, u = M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"])
        got = M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_base=d["gbase"], grad_w=True)
        for name, t in zip(("out", "grad_x", "grad_a", "grad_b", "grad_w"), (out, *got)):
            v, tol = ref[name]
            t = t.cpu().double()
            fin, inf = torch.isfinite(v), torch.isinf(v)
            assert torch.equal(torch.isnan(t), torch.isnan(v)), (where, name)
            assert torch.equal(t[inf], v[inf]), (where, name)
            assert bool(((t - v).abs() <= tol)[fin].all()), (where, name)


@pytest.mark.parametrize("dtype,r", [(BF16, 32), (BF16, 40), (BF16, 128), (F32, 20), (F32, 36), (F32, 128)])
@pytest.mark.parametrize("wide", ["x", "out"])
def test_every_form_past_two_gib(dtype, r, wide):
    """The kernels for more wide rows than 32-bit offsets reach: both rank widths and
    types, on either side, tiles that adapters share, tokens without one, weights and
    grad_w.  Every element, in blocks of tokens, against float64 on the GPU."""
    T, A = (66000 if dtype == BF16 else 33000), 3
    H, N = (16392, 64) if wide == "x" else (64, 16392)
    assert T * max(H, N) * torch.finfo(dtype).bits // 8 > 1 << 31
    g = torch.Generator(device=DEV).manual_seed(r)
    new = lambda *s: torch.empty(s, dtype=dtype, device=DEV).normal_(generator=g)  # noqa: E731
    x, base, go = new(T, H), new(T, N), new(T, N)
    a, b = new(A, r, H) * H ** -0.5, new(A, r, N) * r ** -0.5
    w = torch.empty((T, 1), device=DEV).normal_(generator=g)
    ids = torch.randint(0, A + 1, (T, 1), generator=g, device=DEV).to(torch.int32)
    h = M.moe_layout(ids, A + 1, 1)
    out, u = M.moe_lowrank(h, x, a, b, w, base=base)
    gx, ga, gb, gw = M.moe_lowrank_bwd(h, go, x, a, b, u, w, grad_w=True)
    ad, bd = a.double(), b.double()
    ra, rb = torch.zeros_like(ad), torch.zeros_like(bd)
    ma, mb = torch.zeros_like(ad), torch.zeros_like(bd)
    for t0 in range(0, T, 5000):
        t1 = min(t0 + 5000, T)
        i, xs, gs = ids[t0:t1].view(-1), x[t0:t1].double(), go[t0:t1].double()
        for e in range(A):
            k = torch.nonzero(i == e).view(-1)
            xe, ge, we = xs[k], gs[k], w[t0:t1][k].double()
            at, bt = ad[e].t().contiguous(), bd[e].t().contiguous()
            ue, re = xe @ at, ge @ bt
            um, rm = xe.abs() @ at.abs(), ge.abs() @ bt.abs()
            far_check("out", out[t0:t1][k], base[t0:t1][k].double() + we * (ue @ bd[e]), we.abs() * (um @ bd[e].abs()),
                      H + r + 2, dtype)
            far_check("grad_x", gx[t0:t1][k], we * (re @ ad[e]), we.abs() * (rm @ ad[e].abs()), N + r + 2, dtype)
            far_check("grad_w", gw[t0:t1].view(-1)[k], (ue * re).sum(1), (um * rm).sum(1), H + N + r, F32)
            ra[e] += (we * re).t().contiguous() @ xe
            ma[e] += (we.abs() * rm).t().contiguous() @ xe.abs()
            rb[e] += (we * ue).t().contiguous() @ ge
            mb[e] += (we.abs() * um).t().contiguous() @ ge.abs()
        none = i == A
        assert torch.equal(out[t0:t1][none], base[t0:t1][none]) and (gx[t0:t1][none] == 0).all()
    far_check("grad_a", ga, ra, ma, N + T + 2, dtype)
    far_check("grad_b", gb, rb, mb, H + T + 2, dtype)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_ranks_of_more_rows_than_32_bits_count(dtype):
    """u and the backward's workspace past 2^31 elements (8 GiB): every element of the
    outputs against float64 on the GPU, in blocks of tokens."""
    T, A, r, H, N = (1 << 24) + 999, 3, 128, 8, 16
    g = torch.Generator(device=DEV).manual_seed(2)
    new = lambda *s: torch.empty(s, dtype=dtype, device=DEV).normal_(generator=g)  # noqa: E731
    x, base, go = new(T, H), new(T, N), new(T, N)
    a, b = new(A, r, H) * H ** -0.5, new(A, r, N) * r ** -0.5
    ids = torch.randint(0, A + 1, (T, 1), generator=g, device=DEV).to(torch.int32)
    h = M.moe_layout(ids, A + 1, 1)
    out, u = M.moe_lowrank(h, x, a, b, base=base)
    assert u.numel() > 1 << 31
    gx, ga, gb, gw = M.moe_lowrank_bwd(h, go, x, a, b, u, grad_w=True)
    ad, bd = a.double(), b.double()
    ra, rb = torch.zeros_like(ad), torch.zeros_like(bd)
    ma, mb = torch.zeros_like(ad), torch.zeros_like(bd)
    for t0 in range(0, T, 1 << 20):
        t1 = min(t0 + (1 << 20), T)
        i, xs, gs = ids[t0:t1].view(-1), x[t0:t1].double(), go[t0:t1].double()
        for e in range(A):
            k = torch.nonzero(i == e).view(-1)
            xe, ge = xs[k], gs[k]
            at, bt = ad[e].t().contiguous(), bd[e].t().contiguous()
            ue, re = xe @ at, ge @ bt
            um, rm = xe.abs() @ at.abs(), ge.abs() @ bt.abs()
            far_check("out", out[t0:t1][k], base[t0:t1][k].double() + ue @ bd[e], um @ bd[e].abs(), H + r, dtype)
            far_check("grad_x", gx[t0:t1][k], re @ ad[e], rm @ ad[e].abs(), N + r, dtype)
            far_check("grad_w", gw[t0:t1].view(-1)[k], (ue * re).sum(1), (um * rm).sum(1), H + N + r, F32)
            ra[e] += re.t().contiguous() @ xe
            ma[e] += rm.t().contiguous() @ xe.abs()
            rb[e] += ue.t().contiguous() @ ge
            mb[e] += um.t().contiguous() @ ge.abs()
        none = i == A
        assert torch.equal(out[t0:t1][none], base[t0:t1][none]) and (gx[t0:t1][none] == 0).all()
    far_check("grad_a", ga, ra, ma, N + T, dtype)
    far_check("grad_b", gb, rb, mb, H + T, dtype)


def test_layouts_of_other_forms_give_the_same():
    """Ids of 64 bits, several partitions, a layout without allocations: the adapters' rows are the same."""
    ids, _, d = make(300, 6, 16, 136, 264, BF16, 5, E=8)

    def run(h):
        out, u = M.moe_lowrank(h, d["x"], d["a"], d["b"], d["w"], base=d["base"])
        return (out, u) + M.moe_lowrank_bwd(h, d["g"], d["x"], d["a"], d["b"], u, d["w"], grad_w=True)

    ref = run(M.moe_layout(ids, 8, 1))
    for h in (M.moe_layout(ids.long(), 8, 1), M.moe_layout(ids, 8, 4), M.moe_layout_noalloc(ids, 8, 2)):
        assert all(torch.equal(p, q) for p, q in zip(run(h), ref))
