"""The balance loss where sums are long, logits far apart and sequences many, against values known exactly or in
float64."""
import math

import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_tokens_that_do_not_count_change_nothing(score):
    """The kept tokens' gradients are the same bits whatever the others hold."""
    g = torch.Generator().manual_seed(3)
    z = torch.randn(90, 24, generator=g).to(DEV)
    idx = torch.randint(0, 24, (90, 3), generator=g).to(torch.int32).to(DEV)
    seq = torch.tensor([7, 20, 20, 61, 80], dtype=torch.int32, device=DEV)
    keep = (torch.rand(90, generator=g) > 0.3).to(DEV)
    mask = keep.clone()
    keep[:7] = False
    keep[80:] = False
    gl = torch.tensor([0.7, 1.3], device=DEV)
    got = []
    for other in (1.0, math.nan, math.inf, -math.inf, 3e38):
        z2, idx2 = z.clone(), idx.clone()
        z2[~keep], idx2[~keep] = other, 1 << 30
        loss, counts, probs, tokens = M.moe_balance(z2, idx2, seq, mask, score)
        got.append((loss, counts, probs, tokens, M.moe_balance_bwd(z2, counts, tokens, gl, 3, seq, mask, score)))
    for other in got[1:]:
        assert all(torch.equal(a, b) for a, b in zip(got[0], other))
    assert (got[0][4][~keep] == 0).all() and (got[0][4][keep] != 0).any()


@pytest.mark.parametrize("E", [64, 200, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_far_logits_keep_their_digits(score, E):
    """Scores of logits up to 80 below the largest, each token a sequence of its own, so that probs are the
    scores.

    Logits are multiples of 2^-10 below 2^7, so z - max is exact.  u = 2^-24: an exponential is off by 3 u, a
    sum of at most 16 + 6 terms by 22 u more, the quotient by 2 u, so a softmax by 30 u; a sigmoid relative
    to the largest is an exponential, a sum with another, a quotient and a product, 9 u, so its share is off by
    9 + 31 + 2 u.  The gradient of loss[1] is 2/n lse softmax: 30 u, 3 u for the products, and lse to
    4 u (|lse| + max) + 32 u."""
    T = 48
    g = torch.Generator().manual_seed(E)
    z = -torch.floor(torch.rand(T, E, generator=g) * 80 * 1024) / 1024
    z += torch.floor(torch.rand(T, 1, generator=g) * 40 * 1024 - 20 * 1024) / 1024
    idx = torch.randint(0, E, (T, 2), generator=g).to(torch.int32).to(DEV)
    seq = torch.arange(T + 1, dtype=torch.int32, device=DEV)
    loss, counts, probs, tokens = M.moe_balance(z.to(DEV), idx, seq, None, score)
    grad = M.moe_balance_bwd(z.to(DEV), counts, tokens, torch.tensor([0.0, 1.0], device=DEV), 2, seq, None, score)
    zd = z.double()
    soft, lse = torch.softmax(zd, 1), torch.logsumexp(zd, 1, keepdim=True)
    ref = soft
    if score == "sigmoid":
        ref = torch.sigmoid(zd)
        ref = ref / ref.sum(1, keepdim=True)
    err = ((probs.cpu().double() - ref).abs() / ref).max()
    assert err <= (30 if score == "softmax" else 42) * U, float(err / U)
    want = 2 / T * lse * soft
    dl = 4 * U * (lse.abs() + zd.amax(1, keepdim=True).abs()) + 32 * U
    tol = 33 * U * want.abs() + 2 / T * soft * dl + 1e-37
    bad = (grad.cpu().double() - want).abs() - tol
    assert bool((bad <= 0).all()), float(bad.max())


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_an_infinite_logit_has_an_infinite_z_loss(score):
    """lse of a token with +inf is +inf, and so is the mean of lse^2; with NaN beside it it is NaN."""
    for E in (5, 64, 300):
        z = torch.randn(40, E, generator=torch.Generator().manual_seed(E)).to(DEV)
        idx = torch.zeros(40, 1, dtype=torch.int32, device=DEV)
        z[3, E // 2] = math.inf
        assert M.moe_balance(z, idx, score=score)[0][1] == math.inf
        z[3, 0] = math.inf
        z[3, E - 1] = -math.inf
        assert M.moe_balance(z, idx, score=score)[0][1] == math.inf
        z[3, 1] = math.nan
        assert torch.isnan(M.moe_balance(z, idx, score=score)[0][1])


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,dtype", [((1 << 23) + 5, 13, F32), ((1 << 21) + 3, 300, BF16)])
def test_sums_over_many_equal_tokens(score, T, E, dtype):
    """Equal logits, whose scores 1/E are not dyadic: a long sum in 32 bits rounds to the same side again and again.

    u = 2^-24: a score is off by 4 u, at most 128 of them are added in a wave and 16 waves' sums of them in a run,
    144 u; the rest is in 64 bits, and rounded once.  lse is off by 4 u, its square by 9 u."""
    z = torch.full((T, E), 0.5, dtype=dtype, device=DEV)
    idx = (torch.arange(T, device=DEV) % E).to(torch.int32).view(-1, 1)
    loss, counts, probs, tokens = M.moe_balance(z, idx, score=score)
    assert torch.equal(counts[0].long(), torch.bincount(idx.view(-1), minlength=E)) and tokens.tolist() == [T]
    err = float((probs.double() * (E / T) - 1).abs().max())
    assert err <= 149 * U, err / U
    assert abs(float(loss[0]) - 1) <= 150 * U, float(loss[0] - 1) / U
    lse2 = (0.5 + math.log(E)) ** 2
    assert abs(float(loss[1]) / lse2 - 1) <= 155 * U, (float(loss[1]) / lse2 - 1) / U
