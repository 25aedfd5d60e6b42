"""The router on the GPU against its definition in float64 (numpy): the choice
has to be the same, weights and gradients lie within derived bounds.

Bounds (u = 2^-24).  A weight is a quotient of exponentials of z - m: with
|z - m| <= 64 here, the rounded difference moves an exponential by at most
64 u relative, expf by 2 u, a sum of E <= 1024 positive terms by at most
(E/64 + 6) u <= 22 u on 64 lanes' partial sums (each lane's terms in a row,
then six folds); two quotients and products, 4 u.  Twice that, for numerator
and denominator: 2 * (64 + 2 + 22 + 2) u < 192 u = 1.2e-5.  A gradient is such
a weight times a difference of at most K + 1 bounded products: its bound is
the same factor times the sum of the products' magnitudes.
"""
import math

import numpy as np
import pytest
import torch

import combine_moe_layout_04_amd as M
from devutil import to_host

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
REL = 192 * 2.0 ** -24
F32, BF16 = torch.float32, torch.bfloat16


def draw(T, E, dtype, seed, spread=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(T, E, generator=g) * spread).to(dtype).to(DEV)


def scores64(z, score):
    """Scores in float64, as the definition says: NaN spreads over a softmax row."""
    z = np.asarray(z, np.float64)
    with np.errstate(all="ignore"):
        if score == "sigmoid":
            return 1.0 / (1.0 + np.exp(-z))
        m = np.max(np.where(np.isnan(z), -np.inf, z), axis=1, keepdims=True)
        m = np.where(np.isneginf(m), 0.0, m)
        p = np.exp(z - m)
        s = p.sum(1, keepdims=True)
        return np.where(s == 0, 0.0, p / np.where(s == 0, 1.0, s))


def choice64(z, K, score, bias, groups, keep):
    z = np.asarray(z, np.float64)
    zc = np.where(np.isnan(z), -np.inf, z)
    if bias is None and groups == keep:
        c = zc
    else:
        c = scores64(zc, score) + (0.0 if bias is None else np.asarray(bias, np.float64))
    if keep < groups:
        T, E = c.shape
        top = -np.sort(-c.reshape(T, groups, E // groups), axis=2)[:, :, :2]
        order = np.argsort(-top.sum(2), axis=1, kind="stable")[:, :keep]
        mask = np.zeros((T, groups), bool)
        np.put_along_axis(mask, order, True, 1)
        # a masked expert ranks below a -inf one that takes part
        rank = np.where(np.repeat(mask, E // groups, 1), np.where(np.isneginf(c), -1e300, c), -np.inf)
        return np.argsort(-rank, axis=1, kind="stable")[:, :K]
    return np.argsort(-c, axis=1, kind="stable")[:, :K]


def weights64(z, idx, score, renormalize, scale):
    s = np.take_along_axis(scores64(z, score), idx, 1)
    if renormalize:
        total = s.sum(1, keepdims=True)
        with np.errstate(all="ignore"):
            return np.where(total == 0, 0.0, scale * s / np.where(total == 0, 1.0, total))
    return scale * s


def check(z, K, score, renormalize, scale=1.0, bias=None, groups=1, keep=1):
    idx, w = M.moe_route(z, K, bias, score, renormalize, groups, keep, scale)
    assert idx.dtype == torch.int32 and w.dtype == F32
    z64 = z.double().cpu().numpy()
    ref = choice64(z64, K, score, None if bias is None else bias.cpu().numpy(), groups, keep)
    assert np.array_equal(idx.cpu().numpy(), ref)
    ref_w = weights64(z64, ref, score, renormalize, scale)
    got = w.double().cpu().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(ref_w))
    ok = ~np.isnan(ref_w)
    assert np.all(np.abs(got[ok] - ref_w[ok]) <= REL * np.abs(ref_w[ok]) + 1e-37), np.abs(got[ok] / ref_w[ok] - 1).max()
    return idx


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 128, 8), (5, 60, 4), (3, 63, 63 // 2), (130, 64, 8), (1000, 129, 6),
                                   (257, 256, 8), (33, 500, 32), (65, 1024, 16), (7, 1023, 10)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_choice_and_weights(dtype, T, E, K, score, renormalize):
    check(draw(T, E, dtype, T * E + K, 3.0), min(K, 32, E), score, renormalize, 1.0 if E % 2 else 2.5)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,groups,keep,bias", [
    (64, 256, 8, 8, 4, True), (33, 128, 6, 4, 1, False), (9, 60, 4, 3, 2, True), (17, 64, 8, 64, 9, True),
    (5, 1023, 7, 33, 4, True), (12, 1024, 16, 16, 16, True), (31, 40, 5, 1, 1, True), (3, 992, 32, 31, 2, False),
    (2, 1, 1, 1, 1, True), (101, 64, 8, 1, 1, True), (50, 256, 15, 16, 8, True), (1000, 128, 8, 1, 1, True),
    (333, 256, 8, 8, 4, False), (5, 64, 3, 4, 2, True), (1, 256, 15, 1, 1, True), (19, 64, 4, 16, 16, True)])
def test_bias_and_groups(dtype, score, T, E, K, groups, keep, bias):
    z = draw(T, E, dtype, T + E, 2.0)
    b = torch.randn(E, generator=torch.Generator().manual_seed(7)).mul_(0.1).to(DEV) if bias else None
    check(z, K, score, True, 1.0, b, groups, keep)
    check(z, K, score, False, 2.5, b, groups, keep)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("E", [8, 130, 600])
def test_ties_go_to_the_lower_index(dtype, E):
    z = torch.randint(-2, 3, (50, E), generator=torch.Generator().manual_seed(E)).to(dtype).to(DEV)
    z[3] = 0.0
    z[3, ::2] = -0.0  # one value
    for groups in (1, 2):
        check(z, 8 if groups == 1 else 4, "sigmoid", True, 1.0, None, groups, 1)
    check(z, 5, "softmax", False, 1.0, torch.zeros(E, device=DEV))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,groups,keep", [(96, 1, 1), (96, 8, 3), (128, 1, 1), (128, 8, 3)])
def test_choices_next_to_a_border(score, E, groups, keep):
    """Biases that lift every expert to the same value but for their own float32
    rounding: only 64 bits tell the experts (and groups) apart, and the choice
    has to be the one that they tell."""
    for seed in range(40):
        z = draw(1, E, F32, seed, 1.5)
        s = scores64(z.cpu().numpy(), score)[0]
        b = torch.from_numpy((1.0 - s).astype(np.float32)).to(DEV)
        spread = np.abs(s + b.double().cpu().numpy() - 1.0).max()
        assert 0 < spread < 2.0 ** -24
        check(z, 6, score, True, 1.0, b, groups, keep)
        # among tokens that are told apart easily
        rows = draw(7, E, F32, 1000 + seed, 1.5)
        rows[seed % 7] = z[0]
        check(rows, 6, score, True, 1.0, b, groups, keep)


def test_masked_rows_and_nan():
    z = draw(40, 96, F32, 5, 2.0)
    z[0] = -math.inf                       # nothing left
    z[1, 5:] = -math.inf                   # fewer than K left
    z[2, 7] = math.nan
    z[3, :] = torch.finfo(F32).min
    z[4, ::2] = -math.inf
    z[5, :] = math.nan
    z[6, :] = torch.finfo(F32).min
    z[6, 90] = torch.finfo(F32).max / 2
    for score in ("softmax", "sigmoid"):
        for renormalize in (True, False):
            idx = check(z, 8, score, renormalize)
            assert idx[0].tolist() == list(range(8))
    zero = torch.zeros(96, device=DEV)
    for score in ("softmax", "sigmoid"):
        check(z, 8, score, True, 1.0, zero, 8, 3)
        check(torch.cat([z, z[:, :32]], 1), 8, score, True, 1.0, torch.zeros(128, device=DEV), 8, 3)
        check(torch.cat([z, z[:, :32]], 1), 8, score, False, 1.0, torch.zeros(128, device=DEV))
    _, w = M.moe_route(z, 8, score="softmax")
    assert (w[0] == 0).all() and torch.isnan(w[2]).all() and not torch.isnan(w[3:5]).any()


def grad64(z, idx, gw, score, renormalize, scale):
    """The formulas in float64, with the magnitudes that the bound multiplies."""
    z = np.asarray(z, np.float64)
    T, E = z.shape
    K = idx.shape[1]
    G = scale * np.asarray(gw, np.float64)
    s = scores64(z, score)
    g, mag = np.zeros((T, E)), np.zeros((T, E))
    for t in range(T):
        ok = [(k, e) for k, e in enumerate(idx[t]) if 0 <= e < E]
        if score == "softmax" and not renormalize:
            dot = sum(s[t, e] * G[t, k] for k, e in ok)
            size = sum(s[t, e] * abs(G[t, k]) for k, e in ok)
            up, upm = np.zeros(E), np.zeros(E)
            for k, e in ok:
                up[e] += G[t, k]
                upm[e] += abs(G[t, k])
            g[t], mag[t] = s[t] * (up - dot), s[t] * (upm + size)
            continue
        total = sum(s[t, e] for _, e in ok) if renormalize else 1.0
        total = total if total else 1.0
        mean = sum(s[t, e] / total * G[t, k] for k, e in ok) if renormalize else 0.0
        size = sum(s[t, e] / total * abs(G[t, k]) for k, e in ok) if renormalize else 0.0
        for k, e in ok:
            f = s[t, e] / total * (1.0 if score == "softmax" else 1.0 / (1.0 + math.exp(z[t, e])))
            g[t, e] += f * (G[t, k] - mean)
            mag[t, e] += f * (abs(G[t, k]) + size)
    return g, mag


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
@pytest.mark.parametrize("T,E,K", [(1, 1, 1), (1, 128, 8), (37, 60, 4), (130, 129, 32), (5, 1024, 8), (9, 1000, 1)])
def test_gradient_against_the_formula(dtype, score, renormalize, T, E, K):
    z = draw(T, E, dtype, E + K, 2.0)
    idx, _ = M.moe_route(z, K, score=score, renormalize=renormalize, scale=1.5)
    gw = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).to(DEV)
    if T > 20:
        idx = idx.clone()
        idx[3, 1] = idx[3, 0]      # the same expert twice
        idx[4, 2] = -1             # no expert
        idx[5, 0] = E
        idx[6, :] = -7
    got = M.moe_route_bwd(z, idx, gw, score, renormalize, 1.5)
    assert got.dtype == dtype
    ref, mag = grad64(z.double().cpu().numpy(), idx.cpu().numpy(), gw.cpu().numpy(), score, renormalize, 1.5)
    tol = REL * mag + (torch.finfo(dtype).eps / 2 * np.abs(ref) * (1 + REL) if dtype == BF16 else 0.0) + 1e-37
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), (err - tol).max()


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [True, False])
def test_gradient_against_differences(score, renormalize):
    """Central differences of the float64 weights at the kernel's choice, step
    h = 1e-5: their error is h^2/6 of a third derivative (below 10 for these
    scores and |G| <= 4) and 1e-16/h from rounding, 1e-9 together."""
    z = draw(6, 24, F32, 11)
    idx, _ = M.moe_route(z, 4, score=score, renormalize=renormalize)
    gw = torch.randn(6, 4, generator=torch.Generator().manual_seed(2)).clamp_(-4, 4).to(DEV)
    got = M.moe_route_bwd(z, idx, gw, score, renormalize).double().cpu().numpy()
    z64, i, g = z.double().cpu().numpy(), idx.cpu().numpy(), gw.double().cpu().numpy()
    _, mag = grad64(z64, i, g, score, renormalize, 1.0)
    h = 1e-5
    for j in range(24):
        d = np.zeros_like(z64)
        d[:, j] = h
        up = (weights64(z64 + d, i, score, renormalize, 1.0) * g).sum(1)
        down = (weights64(z64 - d, i, score, renormalize, 1.0) * g).sum(1)
        assert np.all(np.abs((up - down) / (2 * h) - got[:, j]) <= REL * mag[:, j] + 1e-8)


def test_autograd_route_reaches_the_logits():
    z = draw(20, 32, F32, 3).requires_grad_()
    idx, w = M.autograd.route(z, 4, score="sigmoid", scale=2.0)
    assert not idx.requires_grad
    g = torch.randn(20, 4, generator=torch.Generator().manual_seed(4)).to(DEV)
    w.backward(g)
    assert torch.equal(z.grad, M.moe_route_bwd(z.detach(), idx, g, "sigmoid", True, 2.0))


def test_empty_batch_and_given_outputs():
    z = torch.empty((0, 16), device=DEV)
    idx, w = M.moe_route(z, 4)
    assert idx.shape == (0, 4) and w.shape == (0, 4)
    assert M.moe_route_bwd(z, idx, w).shape == (0, 16)
    z = draw(9, 16, F32, 1)
    oi = torch.full((11, 4), -5, dtype=torch.int32, device=DEV)
    ow = torch.full((11, 4), 9.0, device=DEV)
    i2, w2 = M.moe_route(z, 4, topk_idx=oi[1:10], topk_weights=ow[1:10])
    ref = M.moe_route(z, 4)
    assert torch.equal(i2, ref[0]) and torch.equal(w2, ref[1])
    assert (oi[0] == -5).all() and (oi[10] == -5).all() and (ow[0] == 9).all() and (ow[10] == 9).all()


def test_refusals():
    z = draw(4, 16, F32, 1)
    with pytest.raises(ValueError, match="score"):
        M.moe_route(z, 2, score="tanh")
    for kw, code in ((dict(num_groups=3, topk_groups=1), -2), (dict(num_groups=4, topk_groups=5), -2),
                     (dict(num_groups=8, topk_groups=1), -2), (dict(scale=math.inf), -1), (dict(num_groups=0), -2)):
        with pytest.raises(M.MoeError) as e:
            M.moe_route(z, 4, **kw)
        assert e.value.code == code, kw
    with pytest.raises(M.MoeError):
        M.moe_route(z, 17)
    with pytest.raises(ValueError):
        M.moe_route(z.t(), 2)
    with pytest.raises(ValueError):
        M.moe_route(z, 2, bias=torch.zeros(15, device=DEV))
    with pytest.raises(ValueError):
        M.moe_route(z.cpu(), 2)
    with pytest.raises(TypeError):
        M.moe_route(z.half(), 2)
    idx, w = M.moe_route(z, 2)
    with pytest.raises(ValueError):
        M.moe_route_bwd(z, idx.long(), w)
    with pytest.raises(ValueError):
        M.moe_route_bwd(z, idx, w[:, :1].contiguous())


def test_graph_replays_match_eager():
    z = draw(300, 128, BF16, 8)
    gw = torch.randn(300, 8, generator=torch.Generator().manual_seed(3)).to(DEV)
    idx = torch.empty((300, 8), dtype=torch.int32, device=DEV)
    w = torch.empty((300, 8), device=DEV)
    gz = torch.empty_like(z)

    def step():
        M.moe_route(z, 8, renormalize=False, topk_idx=idx, topk_weights=w)
        M.moe_route_bwd(z, idx, gw, renormalize=False, grad_logits=gz)

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
        z.copy_(draw(300, 128, BF16, 100 + seed))
        ri, rw = M.moe_route(z, 8, renormalize=False)
        rg = M.moe_route_bwd(z, ri, gw, renormalize=False)
        torch.cuda.synchronize()
        idx.zero_(), w.zero_(), gz.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(idx, ri) and torch.equal(w, rw) and torch.equal(gz, rg)


def shares64(z, idx, score):
    """Renormalised scores of the chosen experts in float64, formed from their
    logarithms, so that no score is too small; sigmoids below 2^-1022 count as zero."""
    z = np.take_along_axis(np.asarray(z, np.float64), idx, 1)
    log = z if score == "softmax" else np.where(z < -708.0, -np.inf, -np.logaddexp(0.0, -z))
    top = log.max(1, keepdims=True)
    s = np.exp(log - np.where(np.isneginf(top), 0.0, top))
    return s / np.maximum(s.sum(1, keepdims=True), 1e-300)


def check_shares(z, K, score, scale, bias=None, groups=1, keep=1):
    """Weights and gradients of a renormalised router against shares64.  With logits
    d <= 104 below the largest chosen one (further ones' shares are below 1e-45) the
    module's bound is 2 * (104 + 2 + 22 + 2) u, and 2 * 3 u more for the sigmoid's
    other factor: below 272 u.  1e-37: what is rounded below the normal numbers."""
    rel = 272 * 2.0 ** -24
    idx, w = M.moe_route(z, K, bias, score, True, groups, keep, scale)
    z64 = z.double().cpu().numpy()
    ref = choice64(z64, K, score, None if bias is None else bias.cpu().numpy(), groups, keep)
    assert np.array_equal(idx.cpu().numpy(), ref)
    q = shares64(z64, ref, score)
    assert np.all(np.abs(w.double().cpu().numpy() - scale * q) <= rel * scale * q + 1e-37)
    gw = torch.randn(*w.shape, generator=torch.Generator().manual_seed(5)).to(DEV)
    G = scale * gw.double().cpu().numpy()
    rest = 1.0 if score == "softmax" else 1.0 / (1.0 + np.exp(np.take_along_axis(z64, ref, 1)))
    g = np.zeros(z64.shape)
    mag = np.zeros(z64.shape)
    np.put_along_axis(g, ref, (G - (q * G).sum(1, keepdims=True)) * q * rest, 1)
    np.put_along_axis(mag, ref, (np.abs(G) + (q * np.abs(G)).sum(1, keepdims=True)) * q * rest, 1)
    got = M.moe_route_bwd(z, idx, gw, score, True, scale).double().cpu().numpy()
    half = torch.finfo(z.dtype).eps / 2 if z.dtype == BF16 else 0.0
    assert np.all(np.abs(got - g) <= rel * mag + half * np.abs(g) * (1 + rel) + 1e-37)
    return w


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [1, 8])
@pytest.mark.parametrize("scale", [1.0, 2.5, 1e-3])
@pytest.mark.parametrize("lo,hi", [(-110, -85), (-95, -80), (-700, -60), (-130, 3)])
def test_renormalised_sigmoids_far_below_zero(dtype, K, scale, lo, hi):
    """Scores whose sum, or its quotient with the scale, 32 bits do not hold."""
    g = torch.Generator().manual_seed(K - lo)
    z = torch.empty(60, 64).uniform_(lo, hi, generator=g).to(dtype).to(DEV)
    z[0] = -88.2
    b = torch.randn(64, generator=g).to(DEV)
    for bias, groups, keep in ((None, 1, 1), (b, 1, 1), (b, 4, 2)):
        w = check_shares(z, K, "sigmoid", scale, bias, groups, keep)
        assert float((w.sum(1) - scale).abs().max()) <= 2e-5 * scale


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("K", [1, 8])
@pytest.mark.parametrize("scale", [1.0, 2.5])
@pytest.mark.parametrize("depth", [60, 85, 100, 600])
def test_softmax_with_a_bias_towards_experts_far_below_the_largest(dtype, K, scale, depth):
    g = torch.Generator().manual_seed(depth)
    z = torch.empty(60, 64).uniform_(-35 - depth, -depth, generator=g)
    z[:, ::8] = torch.randn(60, 8, generator=g)
    b = torch.rand(64, generator=g)
    b[::8] = -3.0
    for groups, keep in ((1, 1), (4, 2)):
        w = check_shares(z.to(dtype).to(DEV), K, "softmax", scale, b.to(DEV), groups, keep)
        assert float((w.sum(1) - scale).abs().max()) <= 2e-5 * scale


def test_scores_that_count_as_zero():
    """Sigmoids below 2^-1022, as of a mask of the type's lowest value, and -inf."""
    z = torch.full((4, 32), -800.0)
    z[1, 3] = -600.0
    z[2] = torch.finfo(F32).min
    z[3] = -math.inf
    for bias in (None, torch.zeros(32, device=DEV)):
        w = check_shares(z.to(DEV), 4, "sigmoid", 2.0, bias)
        assert (w[[0, 2, 3]] == 0).all() and w[1].sum() == 2


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_nan_in_the_gradient(score):
    """A NaN among the chosen logits reaches its token's gradient, every element of
    it where the softmax is not renormalised; renormalised, the logits that were not
    chosen have no part in it."""
    z = draw(6, 40, F32, 3, 2.0)
    z[:, 39] = -20.0
    idx, _ = M.moe_route(z, 4, score=score)
    gw = torch.randn(6, 4, generator=torch.Generator().manual_seed(2)).to(DEV)
    clean = {r: M.moe_route_bwd(z, idx, gw, score, r) for r in (True, False)}
    z[1, 39] = math.nan                 # not chosen
    z[2, int(idx[2, 1])] = math.nan     # chosen
    for r in (True, False):
        g = M.moe_route_bwd(z, idx, gw, score, r)
        other = [0, 3, 4, 5]
        assert torch.equal(g[other], clean[r][other])
        if score == "softmax" and not r:
            assert torch.isnan(g[[1, 2]]).all()
            continue
        assert torch.equal(g[1], clean[r][1])
        hit = torch.zeros(40, dtype=torch.bool, device=DEV)
        hit[(idx[2] if r else idx[2, 1:2]).long()] = True
        assert torch.equal(torch.isnan(g[2]), hit)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_biases_keep_the_group_limit(score):
    """A bias of +inf puts its expert, and so its group, in front, also where the
    rest of the group is at -inf; one of -inf puts its expert last."""
    z = draw(9, 16, F32, 1)
    b = torch.zeros(16, device=DEV)
    b[4:8] = -math.inf
    b[5] = math.inf
    b[15] = -math.inf
    idx, _ = M.moe_route(z, 4, b, score, True, 4, 1)
    assert (idx == torch.tensor([5, 4, 6, 7], dtype=torch.int32, device=DEV)).all()
    idx, _ = M.moe_route(z, 8, b, score, True, 4, 2)  # and the best other group
    assert (idx[:, 0] == 5).all()
    c = scores64(z.double().cpu().numpy(), score) + np.where(np.isinf(b.cpu().numpy()), -np.inf, 0.0)
    for t in range(9):
        value = [-np.sort(-c[t, 4 * g:4 * g + 4])[:2].sum() for g in range(4)]
        best = max((g for g in range(4) if g != 1), key=lambda g: value[g])
        assert set(idx[t].tolist()) == set(range(4, 8)) | set(range(4 * best, 4 * best + 4))
    idx, _ = M.moe_route(z, 2, b, score)
    assert (idx[:, 0] == 5).all() and not torch.isin(idx[:, 1], torch.tensor([4, 6, 7, 15], device=DEV)).any()


def test_the_most_tokens():
    """One expert: nothing to choose, every weight 1; 2^26 - 4 tokens fill the largest grid."""
    z = torch.zeros((2 ** 26 - 4, 1), dtype=BF16, device=DEV)
    idx = torch.full((z.shape[0], 1), 7, dtype=torch.int32, device=DEV)
    w = torch.zeros(z.shape, device=DEV)
    M.moe_route(z, 1, topk_idx=idx, topk_weights=w)
    assert int((idx != 0).sum()) == 0 and int((w != 1).sum()) == 0
    g = M.moe_route_bwd(z, idx, w, renormalize=False)
    assert int((g != 0).sum()) == 0
    more = torch.zeros((2 ** 26 - 3, 1), dtype=BF16, device=DEV)
    with pytest.raises(M.MoeError) as e:
        M.moe_route(more, 1)
    assert e.value.code == -3


def test_logits_past_four_gib():
    """2^31 logits and more: the last tokens get what they get in a call of their own."""
    T, E, K = 2 ** 21 + 77, 1024, 2
    z = torch.empty((T, E), dtype=BF16, device=DEV).normal_(generator=torch.Generator(device=DEV).manual_seed(1))
    assert z.numel() > 1 << 31
    bias = torch.rand(E, device=DEV)
    for kw in (dict(), dict(bias=bias, score="sigmoid", num_groups=8, topk_groups=2)):
        idx, w = M.moe_route(z, K, **kw)
        ref = M.moe_route(z[-500:], K, **kw)
        assert torch.equal(idx[-500:], ref[0]) and torch.equal(w[-500:], ref[1])
    for renormalize in (True, False):
        g = M.moe_route_bwd(z, idx, w, renormalize=renormalize)
        assert torch.equal(g[-500:], M.moe_route_bwd(z[-500:], ref[0], ref[1], renormalize=renormalize))
