"""The norms before and after a block and their gradients against the formulas in float64.

Bounds, with u = 2^-24.  A sum over a row adds at most 32 values a lane, 6 steps in the wave and 16
waves: 54 u of the sum of magnitudes, called S = 60 with the products; a root mean square is off by
S/2 u, its reciprocal by 40 u with the division and the root.  Errors are carried through each step
below as arrays (e_*), and an output adds eps/2 of itself for the rounding to its type.  A sum over
n tokens adds n u of the sum of magnitudes, whatever its order.
"""
import math

import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
S = 60


def make(T, H, dtype, seed, G=0, post=True, nxt=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    d = dict(x=n(T, H), y=n(T, H) * 3, weight=1 + 0.3 * n(H) if post else None, gate=n(G, H) if G else None,
             next_weight=1 + 0.3 * n(H) if nxt else None, grad_out=n(T, H), grad_n=n(T, H) if nxt else None)
    return {k: None if v is None else v.to(dtype).to(DEV) for k, v in d.items()}


def up(t):
    return None if t is None else t.cpu().double()


def norm(v, e_v, eps):
    """v^ = v r, r, their bounds: r is off by 40 u and what the row's own error does to it."""
    r = 1 / torch.sqrt((v * v).mean(1, keepdim=True) + eps)
    rho = 40 * U + e_v.norm(dim=1, keepdim=True) * r / math.sqrt(v.shape[1])
    return v * r, r, r * e_v + (rho + U) * (v * r).abs(), rho


def reference(d, a, eps, offset, y=None, e_y=None, half=None):
    """{name: (value, bound)} of everything, in float64."""
    dtype = d["x"].dtype
    half = torch.finfo(dtype).eps / 2
    x, w1, w2 = up(d["x"]), up(d.get("weight")), up(d.get("next_weight"))
    y = up(d["y"]) if y is None else y
    e_y = torch.zeros_like(y) if e_y is None else e_y
    T, H = x.shape
    gate = up(d.get("gate"))
    G = 0 if gate is None else gate.shape[0]
    gt = torch.ones(T, 1, dtype=torch.float64) if G == 0 else gate.repeat_interleave(T // G, 0)
    res = {}

    def put(name, v, e):
        res[name] = (v, e + half * (v.abs() + e) + 1e-37)

    if w1 is not None:
        w1 = w1 + offset
        yh, r1, e_yh, rho1 = norm(y, e_y, eps)
        yn, e_yn = yh * w1, w1.abs() * e_yh + 3 * U * (yh * w1).abs()
        res["rstd_y"] = (r1[:, 0], (r1 * rho1)[:, 0])
    else:
        yh, e_yh, yn, e_yn = y, e_y, y, e_y
    f, e_f = gt * yn, gt.abs() * e_yn + U * (gt * yn).abs()
    z = a * x + f
    e_z = e_f + 2 * U * ((a * x).abs() + f.abs())
    put("out", z, e_z)
    if w2 is not None:
        w2 = w2 + offset
        zh, r2, e_zh, rho2 = norm(z, e_z, eps)
        put("n", zh * w2, w2.abs() * e_zh + 3 * U * (zh * w2).abs())
        res["rstd_z"] = (r2[:, 0], (r2 * rho2)[:, 0])
    if "grad_out" not in d:
        return res
    dd = up(d["grad_out"]) if d["grad_out"] is not None else torch.zeros_like(x)
    e_d = torch.zeros_like(x)
    tokens = (T + 64) * U
    if d.get("grad_n") is not None:
        gn = up(d["grad_n"])
        put("grad_next_weight", (gn * zh).sum(0), (gn.abs() * e_zh).sum(0) + tokens * (gn * zh).abs().sum(0))
        g2 = gn * w2
        m = (g2 * zh).mean(1, keepdim=True)
        e_m = (g2.abs() * e_zh + (S + 4) * U * (g2 * zh).abs()).mean(1, keepdim=True)
        t = g2 - zh * m
        size = g2.abs() + (zh * m).abs()
        dd = dd + r2 * t
        e_d = r2 * (4 * U * size + zh.abs() * e_m + e_zh * (m.abs() + e_m)) + rho2 * r2 * t.abs() + 4 * U * (dd.abs() + r2 * size)
    put("grad_x", a * dd, abs(a) * e_d + U * (a * dd).abs())
    if G:
        p = dd * yn
        e_p = e_d * yn.abs() + (dd.abs() + e_d) * e_yn + 2 * U * p.abs()
        put("grad_gate", p.view(G, T // G, H).sum(1), (e_p + tokens * p.abs()).view(G, T // G, H).sum(1))
    v, e_v = gt * dd, gt.abs() * e_d + U * (gt * dd).abs()
    if w1 is not None:
        p = v * yh
        put("grad_weight", p.sum(0), (e_v * yh.abs() + (v.abs() + e_v) * e_yh + (tokens + U) * p.abs()).sum(0))
        e_v = w1.abs() * e_v + 2 * U * (w1 * v).abs()
        v = w1 * v
        m = (v * yh).mean(1, keepdim=True)
        e_m = (e_v * yh.abs() + (v.abs() + e_v) * e_yh + (S + 4) * U * (v * yh).abs()).mean(1, keepdim=True)
        t = v - yh * m
        e_v = r1 * (e_v + yh.abs() * e_m + e_yh * (m.abs() + e_m) + 4 * U * (v.abs() + (yh * m).abs())) + (rho1 + 2 * U) * r1 * t.abs()
        v = r1 * t
    put("grad_y", v, e_v)
    return res


def compare(got, ref):
    for name, t in got.items():
        if t is None:
            assert name not in ref, name
            continue
        v, e = ref[name]
        err = (t.cpu().double() - v).abs()
        assert t.shape == v.shape and bool((err <= e).all()), (name, float((err - e).max()), float((err / e).max()))


def names(got):
    return dict(zip(("grad_x", "grad_y", "grad_weight", "grad_gate", "grad_next_weight"), got))


def run_all(d, a=1.0, eps=1e-6, offset=0.0):
    kw = dict(weight=d["weight"], gate=d["gate"], residual_scale=a, next_weight=d["next_weight"], offset=offset)
    out, n, rstd = M.moe_postnorm(d["x"], d["y"], eps=eps, **kw)
    ref = reference(d, a, eps, offset)
    compare({"out": out, "n": n} | ({"rstd_y": rstd[:, 0]} if d["weight"] is not None else {})
            | ({"rstd_z": rstd[:, 1]} if n is not None else {}), ref)
    got = names(M.moe_postnorm_bwd(d["grad_out"], d["grad_n"], d["x"], d["y"], rstd, **kw))
    compare(got, ref)
    return out, n, rstd, got


SHAPES = [(1, 8), (3, 16), (1, 2048), (5, 1000), (17, 40), (64, 4104), (513, 264), (700, 64), (9, 8192 + 8), (2, 16384), (1100, 128)]


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H", SHAPES + [(33, 7168)])
def test_after_a_block(dtype, T, H):
    """Every combination of a post-norm, gates (none, one, one a token, groups) and a next norm, in turn."""
    kinds = [(G, post, nxt) for G in sorted({0, 1, T, next((g for g in (7, 5, 3, 2, 10, 20) if T % g == 0), 1)})
             for post in (True, False) for nxt in (True, False)]
    for i, (G, post, nxt) in enumerate(kinds):
        d = make(T, H, dtype, T + H + i, G, post, nxt)
        run_all(d, a=(1.0, 0.5, -0.25)[i % 3], offset=float(i % 2))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,G", [(1024, 2), (1030, 206), (1530, 510), (1536, 512), (2048, 683 - 171), (3000, 300), (2600, 2), (2600, 1300)])
def test_gates_and_runs_of_rows(dtype, T, G):
    """Gates of more and of fewer tokens than a run has."""
    run_all(make(T, 64, dtype, T + G, G), a=0.5)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H", SHAPES + [(4, 32768 // 2)])
def test_before_a_block(dtype, T, H):
    for offset in (0.0, 1.0):
        d = make(T, H, dtype, T * 3 + H)
        n, rstd = M.moe_prenorm(d["x"], d["next_weight"], 1e-5, offset)
        e = {"x": d["x"], "y": torch.zeros_like(d["x"]), "next_weight": d["next_weight"], "grad_out": None, "grad_n": d["grad_n"]}
        ref = reference(e, 1.0, 1e-5, offset)
        compare({"n": n, "rstd_z": rstd}, ref)
        gx, gw = M.moe_prenorm_bwd(d["grad_n"], d["x"], rstd, d["next_weight"], offset)
        compare({"grad_x": gx, "grad_next_weight": gw}, ref)
        ref = reference(e | {"grad_out": d["grad_out"]}, 1.0, 1e-5, offset)
        base = d["grad_out"].clone()
        gx, none = M.moe_prenorm_bwd(d["grad_n"], d["x"], rstd, d["next_weight"], offset, grad_base=base, grad_x=base, grad_weight=False)
        assert none is None and gx is base
        compare({"grad_x": gx}, ref)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H", [(1, 16), (5, 2048), (33, 624), (64, 7168), (3, 16384), (2, 4112)])
def test_rows_in_8_bits(dtype, T, H):
    """q times scale is within half a step of the norm, and the scale is its largest value's; the
    same numbers through moe_quant_rows where the row type rounds nothing."""
    d = make(T, H, dtype, T + H)
    q, scale = M.moe_prenorm(d["x"], d["next_weight"], quantize=True)
    e = {"x": d["x"], "y": torch.zeros_like(d["x"]), "next_weight": d["next_weight"]}
    v, tol = reference({**e, "x": d["x"]}, 1.0, 1e-6, 0.0)["n"]
    tol = tol - torch.finfo(dtype).eps / 2 * v.abs() * (dtype == BF16)  # not rounded to the row type
    s = scale.cpu().double()[:, None]
    assert bool(((s * 127 - v.abs().amax(1, keepdim=True)).abs() <= tol.amax(1, keepdim=True) + 128 * U * s).all())
    assert bool(((q.cpu().double() * s - v).abs() <= 0.5 * s * (1 + 1e-6) + tol + 128 * U * s).all())
    if dtype == F32:
        n, _ = M.moe_prenorm(d["x"], d["next_weight"])
        q2, s2 = M.moe_quant_rows(n)
        assert torch.equal(q, q2) and torch.equal(scale, s2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,E,H,pad,weighted", [(1, 8, 128, 256, 1, True), (32, 8, 16, 2048, 1, True), (77, 3, 5, 1000, 1, False),
                                                  (130, 2, 9, 104, 16, True), (9, 32, 40, 520, 1, True), (20, 5, 5, 8200, 4, True)])
def test_combine_on_the_way(dtype, T, K, E, H, pad, weighted):
    """Receive rows through the layout; the sum is off by (K + 1) u of its magnitudes."""
    g = torch.Generator().manual_seed(T)
    idx = torch.randint(0, E, (T, K), generator=g).to(torch.int32).to(DEV)
    tw = torch.randn(T, K, generator=g).to(DEV) if weighted else None
    h = M.moe_layout(idx, E, 1, handle=M.Handle(pad_multiple=pad))
    rows = torch.full((h.R, H), math.nan, dtype=dtype, device=DEV)
    pos = h.field("recv_pos").long()
    rows[pos.view(-1)] = torch.randn(T * K, H, generator=g).to(dtype).to(DEV)
    for gate, post in ((0, True), (1, True), (T, False)):
        d = make(T, H, dtype, T + H, gate, post)
        y = rows[pos].cpu().double()
        wt = torch.ones(T, K, 1, dtype=torch.float64) if tw is None else tw.cpu().double()[:, :, None]
        ref = reference({k: d[k] for k in ("x", "weight", "gate", "next_weight")}, 0.5, 1e-6, 0.0, (wt * y).sum(1),
                        (K + 1) * U * (wt * y).abs().sum(1))
        out, n, rstd = M.moe_postnorm(d["x"], rows, d["weight"], d["gate"], 0.5, d["next_weight"], handle=h, topk_weights=tw)
        compare({"out": out, "n": n, "rstd_z": rstd[:, 1]}, ref)
        if dtype == F32:  # the same sums as moe_combine, whose rows are not rounded here
            two = M.moe_postnorm(d["x"], M.moe_combine(h, rows, tw), d["weight"], d["gate"], 0.5, d["next_weight"])
            assert torch.equal(two[0], out) and torch.equal(two[1], n) and torch.equal(two[2], rstd)
    assert h.check() == 0


def test_magnitudes_whose_squares_leave_the_range():
    """Rows of 1e30 and of 1e-30, of zeros, and of one value."""
    for dtype in (F32, BF16):
        x = torch.randn(6, 512, generator=torch.Generator().manual_seed(0))
        x[0] *= 1e30
        x[1] *= 1e-30
        x[2] = 0
        x[3] = 0
        x[3, 7] = 2e38
        x[4] *= 1e19
        x = x.to(dtype).to(DEV)
        w = torch.ones(512, dtype=dtype, device=DEV)
        for eps in (1e-6, 1e-38, 1e-30):
            n, rstd = M.moe_prenorm(x, w, eps)
            v = x.cpu().double()
            r = 1 / torch.sqrt((v * v).mean(1) + eps)
            assert bool(((rstd.cpu().double() - r).abs() <= 60 * U * r).all()), (dtype, eps)
            assert bool(((n.cpu().double() - v * r[:, None]).abs()
                         <= (64 * U + torch.finfo(dtype).eps / 2) * (v * r[:, None]).abs() + 1e-37).all())


def test_rows_keep_to_themselves():
    """NaN and infinities in one row reach that row's results and the weights' gradients alone."""
    d = make(40, 128, F32, 3, 40)
    ref = run_all(d)
    d["y"][7, 3], d["x"][9, 4] = math.nan, math.inf
    kw = dict(weight=d["weight"], gate=d["gate"], next_weight=d["next_weight"])
    out, n, rstd = M.moe_postnorm(d["x"], d["y"], **kw)
    keep = [t for t in range(40) if t not in (7, 9)]
    assert torch.equal(out[keep], ref[0][keep]) and torch.equal(n[keep], ref[1][keep]) and torch.isnan(n[7]).all()
    got = names(M.moe_postnorm_bwd(d["grad_out"], d["grad_n"], d["x"], d["y"], rstd, **kw))
    for k in ("grad_x", "grad_y", "grad_gate"):
        assert torch.equal(got[k][keep], ref[3][k][keep])


def test_gradients_that_are_asked_for():
    """Each output alone and none of the others gives the same; missing upstream gradients are zero."""
    d = make(150, 96, BF16, 5, 5)
    _, _, rstd, ref = run_all(d, 0.5)
    kw = dict(weight=d["weight"], gate=d["gate"], residual_scale=0.5, next_weight=d["next_weight"])
    order = list(ref)
    for name in order:
        ask = {k: k == name for k in order}
        got = names(M.moe_postnorm_bwd(d["grad_out"], d["grad_n"], d["x"], d["y"], rstd, **kw, **ask))
        assert torch.equal(got[name], ref[name]) and all(got[k] is None for k in order if k != name)
    zero = torch.zeros_like(d["x"])
    for one in (dict(grad_out=None), dict(grad_n=None)):
        a = d | one
        b = d | {k: zero for k in one}
        p = M.moe_postnorm_bwd(a["grad_out"], a["grad_n"], d["x"], d["y"], rstd, **kw)
        q = M.moe_postnorm_bwd(b["grad_out"], b["grad_n"], d["x"], d["y"], rstd, **kw)
        assert all(torch.equal(s, t) for s, t in zip(p, q))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,H,G", [(200, 8200, 2), (200, 8200, 100), (130, 9216, 130), (3, 12288, 1), (65, 16384, 0)])
def test_wide_rows_backward(dtype, T, H, G):
    """Past MOE_NORM_WIDE: gates of more and of fewer tokens than a run, in place, each output alone."""
    d = make(T, H, dtype, T + H, G)
    _, _, rstd, ref = run_all(d, 0.5)
    kw = dict(weight=d["weight"], gate=d.get("gate"), residual_scale=0.5, next_weight=d["next_weight"])
    g = d["grad_out"].clone()
    size = M.moe_norm_bwd_workspace_size(dtype, T, H, G)
    ws = torch.full((size + 512,), 171, dtype=torch.uint8, device=DEV)
    got = names(M.moe_postnorm_bwd(g, d["grad_n"], d["x"], d["y"], rstd, grad_x=g, workspace=ws, **kw))
    assert all(got[k] is None or torch.equal(got[k], ref[k]) for k in got) and (ws[size:] == 171).all()
    for name in ref:
        if ref[name] is None:
            continue
        ask = {k: k == name for k in ref}
        got = names(M.moe_postnorm_bwd(d["grad_out"], d["grad_n"], d["x"], d["y"], rstd, **kw, **ask))
        assert torch.equal(got[name], ref[name])
    run_all(make(T, H, dtype, 1, 0, False, False), 0.5)
    run_all(make(T, H, dtype, 2, G, False, True), 0.5)


def test_outputs_in_place_and_what_lies_around():
    d = make(20, 128, BF16, 2, 4)
    ref = run_all(d)
    kw = dict(weight=d["weight"], gate=d["gate"], next_weight=d["next_weight"])
    x, y = d["x"].clone(), d["y"].clone()
    buf = torch.full((24, 128), 7.0, dtype=BF16, device=DEV)
    out, n, rstd = M.moe_postnorm(x, y, out=x, n=buf[2:22], **kw)
    assert out is x and torch.equal(x, ref[0]) and torch.equal(n, ref[1]) and (buf[:2] == 7).all() and (buf[22:] == 7).all()
    out, _, _ = M.moe_postnorm(d["x"], y, out=y, **kw)
    assert torch.equal(y, ref[0])
    g = d["grad_out"].clone()
    size = M.moe_norm_bwd_workspace_size(BF16, 20, 128, 4)
    ws = torch.full((size + 512,), 171, dtype=torch.uint8, device=DEV)
    got = names(M.moe_postnorm_bwd(g, d["grad_n"], d["x"], d["y"], rstd, grad_x=g, workspace=ws, **kw))
    assert all(torch.equal(got[k], ref[3][k]) for k in got) and (ws[size:] == 171).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_an_empty_batch(dtype):
    x = torch.empty(0, 64, dtype=dtype, device=DEV)
    w, gate = torch.ones(64, dtype=dtype, device=DEV), torch.ones(3, 64, dtype=dtype, device=DEV)
    out, n, rstd = M.moe_postnorm(x, x, w, gate, next_weight=w)
    assert out.shape == n.shape == (0, 64) and rstd.shape == (0, 2)
    got = M.moe_postnorm_bwd(x, x, x, x, rstd, w, gate, next_weight=w)
    assert got[0].shape == (0, 64) and all((t == 0).all() for t in got[2:]) and got[3].shape == (3, 64)
    n, rstd = M.moe_prenorm(x, w)
    assert (M.moe_prenorm_bwd(n, x, rstd, w)[1] == 0).all()
    assert M.moe_prenorm(x, w, quantize=True)[0].shape == (0, 64)


def test_gradient_against_differences():
    """Central differences of a weighted sum of out and n in float64; h^2/6 |f'''| is below 1e-5 at h = 1e-3."""
    d = make(4, 16, F32, 6, 2)
    _, _, _, got = run_all(d, 0.5)

    def value(e):
        r = reference({k: e[k] for k in ("x", "y", "weight", "gate", "next_weight")}, 0.5, 1e-6, 0.0)
        return float((r["out"][0] * up(d["grad_out"])).sum() + (r["n"][0] * up(d["grad_n"])).sum())

    for name, at in (("x", (1, 3)), ("y", (2, 5)), ("weight", (4,)), ("gate", (1, 9)), ("next_weight", (15,))):
        two = []
        for h in (1e-3, -1e-3):
            e = dict(d)
            e[name] = d[name].double()
            e[name][at] += h
            two.append(value(e))
        assert abs((two[0] - two[1]) / 2e-3 - float(got["grad_" + name][at])) < 1e-4, name


def test_rows_past_32_bit_offsets():
    """2^21 rows of 1024 bfloat16 (4 GiB): the last rows are what they are alone."""
    T, H = (1 << 21) + 3, 1024
    x = torch.zeros(T, H, dtype=BF16, device=DEV)
    d = make(3, H, BF16, 1)
    x[-3:] = d["x"]
    n, _ = M.moe_prenorm(x, d["next_weight"])
    one, _ = M.moe_prenorm(d["x"], d["next_weight"])
    assert torch.equal(n[-3:], one) and (n[:-3:100003] == 0).all()
    q, s = M.moe_quant_rows(x)
    q1, s1 = M.moe_quant_rows(d["x"])
    assert torch.equal(q[-3:], q1) and torch.equal(s[-3:], s1)
    out, n, rstd = M.moe_postnorm(x, x, d["weight"], next_weight=d["next_weight"], out=n)
    o1, n1, r1 = M.moe_postnorm(d["x"], d["x"], d["weight"], next_weight=d["next_weight"])
    assert torch.equal(out[-3:], o1) and torch.equal(n[-3:], n1) and torch.equal(rstd[-3:], r1)
    got = M.moe_postnorm_bwd(x, x, x, x, rstd, d["weight"], next_weight=d["next_weight"])
    ref = M.moe_postnorm_bwd(d["x"], d["x"], d["x"], d["x"], r1, d["weight"], next_weight=d["next_weight"])
    assert torch.equal(got[0][-3:], ref[0]) and torch.equal(got[1][-3:], ref[1])


def test_the_most_rows():
    """2^26 rows of one chunk: more workgroups than one dimension of a grid holds threads for."""
    T = 1 << 26
    x = torch.zeros(T, 8, dtype=BF16, device=DEV)
    d = make(3, 8, BF16, 2)
    at = torch.tensor([0, (1 << 25) + 1, T - 1], device=DEV)
    x[at] = d["x"]
    n, rstd = M.moe_prenorm(x, d["next_weight"])
    one, r1 = M.moe_prenorm(d["x"], d["next_weight"])
    assert torch.equal(n[at], one) and torch.equal(rstd[at], r1) and int((n != 0).any(1).sum()) == 3
    gx, gw = M.moe_prenorm_bwd(x, x, rstd, d["next_weight"])
    g1, w1 = M.moe_prenorm_bwd(d["x"], d["x"], r1, d["next_weight"])
    assert torch.equal(gx[at], g1) and torch.allclose(gw.float(), w1.float(), rtol=2 ** -7)


def test_refusals():
    d = make(12, 64, F32, 1, 3)
    kw = dict(x=d["x"], y=d["y"], weight=d["weight"], gate=d["gate"], next_weight=d["next_weight"])
    for bad in (dict(y=d["y"][:6]), dict(x=d["x"].t()), dict(weight=d["weight"][:32]), dict(gate=d["gate"][0]),
                dict(next_weight=d["weight"].bfloat16()), dict(y=d["y"].cpu()), dict(out=d["x"][:3]),
                dict(next_weight=None, n=torch.empty_like(d["x"])), dict(gate=d["gate"].new_ones(5, 64)), dict(eps=0.0),
                dict(topk_weights=torch.ones(12, 1, device=DEV))):
        with pytest.raises((ValueError, M.api.MoeError)):
            M.moe_postnorm(**(kw | bad))
    with pytest.raises(RuntimeError):
        M.moe_postnorm(**kw, handle=M.Handle())
    with pytest.raises(ValueError):
        M.moe_prenorm(d["x"], d["weight"], scale=torch.ones(12, device=DEV))
    rstd = torch.ones(12, 2, device=DEV)
    with pytest.raises(ValueError):
        M.moe_postnorm_bwd(d["x"], None, d["x"], d["y"], rstd, grad_weight=True)
    with pytest.raises(M.api.MoeError):
        M.moe_postnorm_bwd(None, None, d["x"], d["y"], rstd, d["weight"])
    with pytest.raises(M.api.MoeError):
        M.moe_prenorm_bwd(d["x"], d["x"], rstd[:, 0].contiguous(), d["weight"], grad_x=False, grad_weight=False)
