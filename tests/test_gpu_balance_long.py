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


def packed(T, lengths):
    off = torch.cat([torch.zeros(1, dtype=torch.int64), torch.cumsum(torch.tensor(lengths), 0)])
    assert off[-1] == T
    return off.to(torch.int32).to(DEV)


MANY = {  # lengths of 65535 sequences: one token each; all empty but one in the middle; runs of empty ones between
    "one token each": [1] * 65535,
    "one of all": [0] * 40000 + [5000] + [0] * 25534,
    "empty runs": ([3, 0, 1] + [0] * 997) * 65 + [0] * 534 + [700],
    "empty first and last": [0] * 30000 + [2] * 5000 + [0] * 30535,
}


@pytest.mark.parametrize("kind", list(MANY))
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_the_most_sequences(kind, score):
    """65535 sequences.  Equal logits: each score is 1/E to 4 u of itself, and with one expert a token, chosen in
    turn, a sequence of n tokens has counts c_e and the loss E/n^2 sum_e c_e n/E = 1; the gradient of the
    balance loss is 1/E (a_e - mean a), a_e = E c_e / (S' n^2)."""
    lengths = MANY[kind]
    assert len(lengths) == 65535
    T, E = sum(lengths), 16
    seq = packed(T, lengths)
    n = torch.tensor(lengths, device=DEV)
    which = torch.repeat_interleave(torch.arange(len(lengths), device=DEV), n)
    z = torch.full((T, E), 0.25, device=DEV)
    idx = (torch.arange(T, device=DEV) % E).to(torch.int32).view(-1, 1)
    loss, counts, probs, tokens = M.moe_balance(z, idx, seq, None, score)
    want = torch.zeros(65535, E, dtype=torch.int32, device=DEV).index_put_((which, idx.view(-1).long()), torch.ones((), dtype=torch.int32, device=DEV), accumulate=True)
    assert torch.equal(counts, want) and torch.equal(tokens, n.int())
    ref = (n.double() / E)[:, None].expand(-1, E)
    assert bool(((probs.double() - ref).abs() <= 160 * U * ref).all())
    assert abs(float(loss[0]) - 1) <= 160 * U and abs(float(loss[1]) / (0.25 + math.log(E)) ** 2 - 1) <= 160 * U
    grad = M.moe_balance_bwd(z, counts, tokens, torch.tensor([1.0, 0.0], device=DEV), 1, seq, None, score).double()
    some = int((n > 0).sum())
    a = E * want[which].double() / (some * n[which].double() ** 2)[:, None]
    slope = 1 / E if score == "softmax" else 1 / E * (1 - 1 / (1 + math.exp(-0.25)))
    m = a.mean(1, keepdim=True)
    tol = 32 * U * slope * (a + m)
    assert bool(((grad - slope * (a - m)).abs() <= tol).all())


def test_sequences_cost_what_is_in_them():
    """4096 tokens with 65535 sequences, nearly all empty, against one sequence: kernels of 120 and 17 us against 11
    and 4.5 (2850 and 120 when every wave walked the empty sequences and read every sequence's tokens)."""
    T, E, K, S = 4096, 128, 8, 65535
    z = torch.randn(T, E, generator=torch.Generator().manual_seed(1)).to(BF16).to(DEV)
    idx = torch.topk(z, K, 1)[1].to(torch.int32)
    many = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    many[S // 2:], many[-1] = T // 2, T
    gl = torch.ones(2, device=DEV)

    def fastest(f):
        f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            for _ in range(5):
                f()
        times = []
        for _ in range(8):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            graph.replay()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)

    took = []
    for seq in (None, many):
        _, counts, _, tokens = M.moe_balance(z, idx, seq)
        took.append((fastest(lambda: M.moe_balance(z, idx, seq)), fastest(lambda: M.moe_balance_bwd(z, counts, tokens, gl, K, seq))))
    assert took[1][0] < 60 * took[0][0] and took[1][1] < 14 * took[0][1], took
