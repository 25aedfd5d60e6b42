"""The expert layer for a few tokens against its formula in float64.

Bound, with u = 2^-24 and n terms in a float32 sum in any order: n u times the
sum of magnitudes.  Per pair: dg <= H u sum|Wg x|, du <= H u sum|Wu x|;
|f'| <= 1.13 for both activations, so the activation is off by
  da <= 1.13 |u| dg + |f(g)| du + dg du + 16 u |g| |u|
(the last for exp, tanh, their arguments and products), and for bfloat16 by
2^-16 |a|, what its two parts leave.  The output adds  sum_k |w| (sum |W2| da + I u sum
|W2 a|),  (K + 2) u sum_k |w| |y| and, for bfloat16, eps/2 |out|.
"""
import math

import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def make(T, K, E, H, I, dtype, seed, itype=torch.int32, of=None):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(T, H, generator=g).to(dtype).to(DEV)
    w13 = (torch.randn(E, 2 * I, H, generator=g) * H ** -0.5).to(dtype).to(DEV)
    w2 = (torch.randn(E, H, I, generator=g) * I ** -0.5).to(dtype).to(DEV)
    idx = torch.randint(0, of or E, (T, K), generator=g).to(itype).to(DEV)
    w = torch.randn(T, K, generator=g).to(DEV)
    return x, idx, w, w13, w2


def reference(x, idx, w, w13, w2, act, rounded=False):
    """(out, bound) in float64 on the CPU; rounded: of a computation that rounds act to the dtype (eps/2 |a|)."""
    dtype = x.dtype
    half, split = (torch.finfo(dtype).eps / 2, 2.0 ** -16) if dtype == BF16 else (0.0, 0.0)
    split = half if rounded else split
    x, w13, w2 = x.cpu().double(), w13.cpu().double(), w2.cpu().double()
    T, H = x.shape
    E, _, I = w2.shape
    out = torch.zeros(T, H, dtype=torch.float64)
    tol = torch.zeros(T, H, dtype=torch.float64)
    K = idx.shape[1]
    for t in range(T):
        for k in range(K):
            e = int(idx[t, k])
            if not 0 <= e < E:
                continue
            g, u = w13[e, :I] @ x[t], w13[e, I:] @ x[t]
            dg, du = H * U * (w13[e, :I].abs() @ x[t].abs()), H * U * (w13[e, I:].abs() @ x[t].abs())
            if act == "silu":
                f = g / (1 + torch.exp(-g))
            else:
                f = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
            a = f * u
            da = 1.13 * u.abs() * dg + f.abs() * du + dg * du + 16 * U * g.abs() * u.abs()
            da = da + split * (a.abs() + da)
            wt = 1.0 if w is None else float(w[t, k])
            y = w2[e] @ a
            size = w2[e].abs() @ a.abs()
            out[t] += wt * y
            tol[t] += abs(wt) * (w2[e].abs() @ da + I * U * size + (K + 2) * U * size)
    return out, tol + half * (out.abs() + tol) + 1e-37


def compare(x, idx, w, w13, w2, act="silu"):
    got = M.moe_few(x, idx, w, w13, w2, activation=act)
    assert got.dtype == x.dtype and got.shape == x.shape
    ref, tol = reference(x, idx, w, w13, w2, act)
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), float((err - tol).max())
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("T,K,E,H,I", [
    (1, 1, 1, 8, 8), (1, 8, 128, 256, 96), (1, 2, 4, 1000, 40), (3, 8, 16, 136, 200), (7, 2, 8, 504, 168),
    (17, 1, 1, 64, 48), (64, 8, 32, 72, 24), (512, 1, 3, 40, 16), (65, 2, 200, 128, 64), (9, 7, 9, 2048, 768),
    (100, 5, 1, 32, 32), (16, 32, 64, 24, 104), (5, 3, 1024, 16, 8)])
def test_against_the_formula(dtype, act, T, K, E, H, I):
    x, idx, w, w13, w2 = make(T, K, E, H, I, dtype, T + K + E)
    compare(x, idx, w, w13, w2, act)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,E", [(16, 2, 16), (17, 2, 16), (32, 2, 16), (33, 2, 16), (64, 2, 16), (65, 2, 16)])
def test_both_sides_of_the_borders_between_tile_counts(dtype, T, K, E):
    """2, 4 and 8 pairs an expert; experts whose load is far from the average among them."""
    x, idx, w, w13, w2 = make(T, K, E, 328, 136, dtype, T)
    compare(x, idx, w, w13, w2)
    idx[:, 0] = 3
    idx[0, 0], idx[1, 0] = 4, -1
    compare(x, idx, w, w13, w2)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_ids_outside_the_experts_add_nothing(dtype, itype):
    x, idx, w, w13, w2 = make(20, 4, 12, 64, 40, dtype, 3, itype, of=48)
    idx[0] = -1
    idx[1] = 12
    idx[2, 0], idx[2, 1] = idx[2, 2], idx[2, 2]  # one expert three times
    idx[3] = torch.iinfo(itype).max
    idx[4] = torch.iinfo(itype).min
    got = compare(x, idx, w, w13, w2)
    for t in (0, 1, 3, 4):
        assert (got[t] == 0).all()
    idx[:] = -1
    assert (M.moe_few(x, idx, w, w13, w2) == 0).all()
    if itype == torch.int64:  # ids whose low half is a valid one
        idx[:] = (1 << 32) + 3
        assert (M.moe_few(x, idx, w, w13, w2) == 0).all()


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [3, 40])
def test_without_weights_and_nothing_leaks(dtype, E):
    """Experts that nobody chose hold NaN, and so does one token: no other row
    sees either."""
    x, idx, _, w13, w2 = make(11, 2, E, 72, 56, dtype, E)
    used = torch.zeros(E, dtype=torch.bool)
    idx = idx.clamp(max=E - 2)
    used[idx.flatten().long().cpu()] = True
    for e in range(E):
        if not used[e]:
            w13[e], w2[e] = math.nan, math.inf
    ref = compare(x, idx, None, w13, w2)
    x2 = x.clone()
    x2[5] = math.nan
    x2[6] = math.inf
    got = M.moe_few(x2, idx, None, w13, w2)
    keep = [t for t in range(11) if t not in (5, 6)]
    assert torch.equal(got[keep], ref[keep]) and torch.isnan(got[5]).all()


def test_rows_around_the_output_stay_and_results_repeat():
    x, idx, w, w13, w2 = make(6, 4, 10, 88, 48, BF16, 1)
    buf = torch.full((10, 88), 7.0, dtype=BF16, device=DEV)
    ws = torch.zeros(M.moe_few_workspace_size(BF16, 6, 4, 48) + 512, dtype=torch.uint8, device=DEV)
    ws[-512:] = 171
    a = M.moe_few(x, idx, w, w13, w2, out=buf[2:8], workspace=ws)
    assert a.data_ptr() == buf[2:8].data_ptr()
    assert (buf[:2] == 7).all() and (buf[8:] == 7).all() and (ws[-512:] == 171).all()
    for _ in range(5):
        assert torch.equal(M.moe_few(x, idx, w, w13, w2), buf[2:8])


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,E", [(512, 1, 1), (64, 8, 3), (170, 3, 40)])
def test_many_pairs_an_expert_repeat(dtype, T, K, E):
    """Which column of a tile a pair takes is left to chance; its values are not."""
    args = make(T, K, E, 136, 72, dtype, 4)
    ref = M.moe_few(*args)
    for _ in range(20):
        assert torch.equal(M.moe_few(*args), ref)


def test_empty_batch():
    x, idx, w, w13, w2 = make(1, 4, 10, 88, 48, BF16, 1)
    assert M.moe_few(x[:0], idx[:0], w[:0], w13, w2).shape == (0, 88)


def test_two_streams_at_once():
    """Calls that overlap, each with its own workspace."""
    sets = [make(8, 4, 16, 512, 256, BF16, s) for s in range(4)]
    refs = [M.moe_few(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    for _ in range(5):
        got = []
        for s, st in zip(sets, streams):
            with torch.cuda.stream(st):
                got.append(M.moe_few(*s))
        torch.cuda.synchronize()
        assert all(torch.equal(g, r) for g, r in zip(got, refs))


def test_graph_replays_with_new_routing():
    x, idx, w, w13, w2 = make(12, 4, 24, 256, 136, BF16, 2)
    out = torch.empty_like(x)
    ws = torch.empty(M.moe_few_workspace_size(BF16, 12, 4, 136), dtype=torch.uint8, device=DEV)

    def step():
        M.moe_few(x, idx, w, w13, w2, out=out, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for seed in range(4):
        x2, idx2, w2_, _, _ = make(12, 4, 24, 256, 136, BF16, 50 + seed, of=30)
        x.copy_(x2), idx.copy_(idx2), w.copy_(w2_)
        ref = M.moe_few(x, idx, w, w13, w2)
        torch.cuda.synchronize()
        out.zero_(), ws.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ref)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_router_layer_and_exchange_agree(dtype):
    """A decode step as a program runs it, router then layer, against the long
    way: layout, dispatch, the experts' products in torch, combine."""
    T, K, E, H, I = 24, 4, 16, 128, 72
    x, _, _, w13, w2 = make(T, K, E, H, I, dtype, 9)
    logits = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(DEV)
    idx, w = M.moe_route(logits, K)
    got = M.moe_few(x, idx, w, w13, w2)
    h = M.moe_layout(idx, E, 1)
    recv, _ = M.moe_dispatch(h, x)
    off = h.field("expert_offset").tolist()
    y = torch.empty(T * K, H, device=DEV)
    for e in range(E):
        r = recv[off[e]:off[e + 1]].float()
        gu = r @ w13[e].float().t().contiguous()
        a = (torch.nn.functional.silu(gu[:, :I]) * gu[:, I:]).to(dtype).float()
        y[off[e]:off[e + 1]] = a @ w2[e].float().t().contiguous()
    out = M.moe_combine(h, y, w)
    # two computations, each within its bound of the formula; the long way rounds act
    tol = sum(reference(x, idx, w, w13, w2, "silu", rounded)[1] for rounded in (False, True))
    assert bool(((got.double() - out.double()).abs().cpu() <= tol).all())


def test_refusals():
    x, idx, w, w13, w2 = make(4, 2, 6, 64, 32, F32, 1)
    for bad in (lambda: M.moe_few(x, idx, w[:3].contiguous(), w13, w2), lambda: M.moe_few(x, idx, w, w13[:5], w2),
                lambda: M.moe_few(x, idx, w, w13, w2.to(BF16)), lambda: M.moe_few(x.cpu(), idx, w, w13, w2),
                lambda: M.moe_few(x, idx, w, w13, w2, activation="relu"), lambda: M.moe_few(x, idx[:3], w, w13, w2),
                lambda: M.moe_few(x, idx, w, w13.transpose(1, 2), w2), lambda: M.moe_few(x[0], idx, w, w13, w2)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(TypeError):
        M.moe_few(x, idx.short(), w, w13, w2)
    with pytest.raises(TypeError):
        M.moe_few(x.half(), idx, w, w13.half(), w2.half())
    big = make(257, 2, 6, 64, 32, F32, 1)
    with pytest.raises(M.MoeError) as e:
        M.moe_few(*big)
    assert e.value.code == -3
    odd = make(4, 2, 6, 66, 32, F32, 1)
    with pytest.raises(M.MoeError) as e:
        M.moe_few(*odd)
    assert e.value.code == -2
    with pytest.raises(M.MoeError) as e:
        M.moe_few(x, idx, w, w13, w2, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.code == -5


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,E", [(1, 1, 1), (3, 2, 40), (33, 2, 16), (70, 3, 16), (150, 2, 16)])
def test_every_bit_of_act_counts(dtype, T, K, E):
    """Columns of act in pairs, 1 + 2^-9 + 2^-s and 1 + 2^-9 with s = 10 ... 23,
    subtracted by the second product, which leaves exactly 2^-s.  Every step is
    exact: the gate is 64, whose sigmoid is 1 in 24 bits; the up products have three
    terms with 24 bits between them, the other sums two; the results, powers of two,
    need no rounding."""
    H, I, steps = 64, 40, range(10, 24)
    x = torch.zeros(T, H)
    x[:, 0], x[:, 1], x[:, 2] = 1.0, 2.0 ** -4, 2.0 ** -4
    w13, w2 = torch.zeros(E, 2 * I, H), torch.zeros(E, H, I)
    w13[:, :I, 0] = 64.0
    want = torch.zeros(H)
    for n, s in enumerate(steps):
        sign = -1.0 if n % 2 else 1.0
        w13[:, I + 2 * n, 0] = w13[:, I + 2 * n + 1, 0] = sign
        w13[:, I + 2 * n, 2] = w13[:, I + 2 * n + 1, 2] = sign * 2.0 ** -5
        w13[:, I + 2 * n, 1] = sign * 2.0 ** (4 - s)
        w2[:, n, 2 * n], w2[:, n, 2 * n + 1] = 1.0, -1.0
        want[n] = sign * 64.0 * 2.0 ** -s
    idx = (torch.arange(T * K) % E).view(T, K).to(torch.int32)
    w = torch.ones(T, K)
    w[:, 1:] = 0.0
    got = M.moe_few(x.to(dtype).to(DEV), idx.to(DEV), w.to(DEV), w13.to(dtype).to(DEV), w2.to(dtype).to(DEV))
    assert torch.equal(got.cpu().float(), want.expand(T, H))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,K,E,H,I", [(1, 2, 6, 64, 40), (9, 3, 12, 520, 264), (40, 2, 16, 2056, 72), (64, 4, 16, 72, 136),
                                       (128, 2, 9, 2048, 48)])
def test_infinities_where_they_count(dtype, T, K, E, H, I):
    """Single infinities in chosen weights and in act come out as the formula in
    float64 has them; everything finite stays within its bound."""
    x, idx, w, w13, w2 = make(T, K, E, H, I, dtype, T + I)
    e = [int(v) for v in idx.flatten()[:3]]
    places = [(e[0], 1, 3, math.inf), (e[-1], H - 1, I - 1, -math.inf), (e[0], 5, 0, -math.inf), (e[0], 5, 1, 1.0)]
    for a, h, i, v in places:
        w2[a, h, i] = v
    if E > 6:  # an infinite column of act: every output of that expert
        w13[int(idx[T - 1, K - 1]), I + 2, 0] = math.inf
    ref, tol = reference(x, idx, w, w13, w2, "silu")
    got = M.moe_few(x, idx, w, w13, w2).cpu().double()
    assert torch.isinf(ref).any()
    fin = torch.isfinite(ref)
    assert torch.equal(torch.isnan(got), torch.isnan(ref))
    assert torch.equal(got[torch.isinf(ref)], ref[torch.isinf(ref)])
    assert bool(((got - ref).abs() <= tol)[fin].all())


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_weights_past_four_gib(dtype):
    """Experts whose weights lie past 32-bit offsets, against a call's formula on
    those experts alone."""
    E, H, I = 1024, 2048, (768 if dtype == BF16 else 400)
    g = torch.Generator(device=DEV).manual_seed(1)
    new = lambda scale, *s: torch.empty(s, dtype=dtype, device=DEV).normal_(0, scale, generator=g)  # noqa: E731
    x, w13, w2 = new(1.0, 5, H), new(H ** -0.5, E, 2 * I, H), new(I ** -0.5, E, H, I)
    assert w13.numel() * w13.element_size() > 1 << 32
    used = torch.tensor([0, 513, 1000, 1022, 1023], device=DEV)
    small = torch.tensor([[4, 0], [3, 4], [2, 1], [4, 3], [0, 2]], device=DEV)
    w = torch.rand((5, 2), generator=g, device=DEV)
    got = M.moe_few(x, used[small], w, w13, w2)
    ref, tol = reference(x, small, w, w13[used], w2[used], "silu")
    assert bool(((got.cpu().double() - ref).abs() <= tol).all())
