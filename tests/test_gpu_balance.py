"""The balance and z losses, their counts and their gradient against the formulas in float64.

Bound, with u = 2^-24 and logits of |z| <= 16: a score is off by C u of itself, C = 128 (the
exponent's rounding |z - max| <= 32, the exponential and the division 4, sums of at most 16 + 6
terms, twice for sigmoids), and so is a softmax value.  A partial sum over a run's tokens adds at
most (run + 8) u; the rest is in 64 bits.  lse is off by 4 u (|lse| + |max|) + 32 u.  A gradient is
off by 200 u s (|a| + sum s |a|) plus g1 2/n (|lse| C u + dlse) soft, and eps/2 of itself for the
rounding to the logits' type.
"""
import math

import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24
C = 128


def make(T, E, K, dtype, seed, S=None, masked=False, itype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    z = (torch.randn(T, E, generator=g) * 2).clamp(-16, 16).to(dtype)
    idx = torch.randint(0, E, (T, K), generator=g).to(itype)
    seq = None
    if S is not None:
        seq = torch.cat([torch.zeros(1), torch.sort(torch.randint(0, T + 1, (S - 1,), generator=g))[0], torch.tensor([T])])
        seq = seq.to(torch.int32)
    mask = torch.rand(T, generator=g) > 0.3 if masked else None
    return tuple(None if t is None else t.to(DEV) for t in (z, idx, seq, mask))


def reference(z, idx, seq, mask, score, grad_loss, base=None):
    """Results and their bounds, in float64 on the CPU: (value, bound) by name."""
    dtype = z.dtype
    z, idx, grad_loss = z.cpu().double(), idx.cpu().long(), grad_loss.cpu().double()
    T, E = z.shape
    K = idx.shape[1]
    seq = [0, T] if seq is None else seq.tolist()
    S = len(seq) - 1
    keep = torch.zeros(T, dtype=torch.bool)
    which = torch.zeros(T, dtype=torch.long)
    for q in range(S):
        keep[seq[q]:seq[q + 1]] = True
        which[seq[q]:seq[q + 1]] = q
    if mask is not None:
        keep &= mask.cpu().bool()
    soft, lse = torch.softmax(z, 1), torch.logsumexp(z, 1)
    dead = lse == -math.inf
    soft[dead], lse[dead] = 0.0, 0.0
    if score == "softmax":
        s, slope = soft, soft
    else:
        sig = torch.where(z < -708, 0.0, torch.sigmoid(z))
        total = sig.sum(1, keepdim=True)
        s = torch.where(total > 0, sig / total, 0.0)
        slope = s * torch.sigmoid(-z)
    member = torch.zeros(S, T, dtype=torch.float64)
    member[which[keep], torch.nonzero(keep)[:, 0]] = 1.0
    good = (idx >= 0) & (idx < E)
    chosen = torch.zeros(T, E, dtype=torch.float64).scatter_add_(1, idx.clamp(0, E - 1), good.double())
    counts, n = member @ chosen, member.sum(1)
    # values that do not count may be anything
    sk, zk = torch.where(keep[:, None], s, 0.0), torch.where(keep, lse, 0.0)
    probs = member @ sk
    some = int((n > 0).sum())
    share = torch.where(n > 0, E / (K * max(1, some) * n.clamp(min=1) ** 2), 0.0)[:, None]
    alln = max(1.0, float(n.sum()))
    loss = torch.stack([(share * counts * probs).sum(), (zk ** 2).sum() / alln])
    run = max(4, (T + 511) // 512)
    rel = (C + run + 16) * U
    dl = 4 * U * (lse.abs() + torch.where(torch.isfinite(z), z, 0.0).abs().amax(1)) + 32 * U
    dz_loss = float((keep * (2 * lse.abs() * dl + dl * dl)).sum() / alln) + (run + 16) * U * float(loss[1])
    a = grad_loss[0] * (member.t() @ (share * counts))
    dot, size = (s * a).sum(1, keepdim=True), (s * a.abs()).sum(1, keepdim=True)
    g1 = grad_loss[1] * 2 / alln
    grad = slope * (a - dot) + g1 * (lse[:, None] * soft)
    tol = 200 * U * slope * (a.abs() + size) + abs(g1) * soft * (lse.abs() * C * U + dl)[:, None]
    grad, tol = torch.where(keep[:, None], grad, 0.0), torch.where(keep[:, None], tol, 0.0)
    if base is not None:
        grad = grad + base.cpu().double()
        tol = tol + U * grad.abs()
    half = torch.finfo(dtype).eps / 2
    return {"loss": (loss, torch.stack([loss[0].abs() * rel, torch.tensor(dz_loss)]) + 1e-37),
            "counts": (counts, torch.zeros(())), "probs": (probs, probs * rel + 1e-37), "tokens": (n, torch.zeros(())),
            "grad": (grad, tol + half * (grad.abs() + tol) + 1e-37)}


def compare(z, idx, seq, mask, score, base=None, seed=0):
    gl = (torch.rand(2, generator=torch.Generator().manual_seed(seed)) + 0.5).to(DEV)
    loss, counts, probs, tokens = M.moe_balance(z, idx, seq, mask, score)
    grad = M.moe_balance_bwd(z, counts, tokens, gl, idx.shape[1], seq, mask, score, grad_base=base)
    assert grad.dtype == z.dtype
    got = {"loss": loss, "counts": counts, "probs": probs, "tokens": tokens, "grad": grad}
    for name, (ref, tol) in reference(z, idx, seq, mask, score, gl, base).items():
        err = (got[name].cpu().double() - ref).abs()
        assert got[name].shape == ref.shape and bool((err <= tol).all()), (name, float((err - tol).max()))
    return got


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K", [
    (1, 1, 1), (1, 8, 2), (2, 64, 8), (5, 65, 1), (17, 3, 3), (256, 8, 2), (1000, 128, 8), (777, 129, 12), (300, 256, 8),
    (33, 257, 4), (40, 513, 32), (9, 1024, 7), (2049, 16, 2), (5000, 60, 4)])
def test_against_the_formulas(dtype, score, T, E, K):
    z, idx, _, _ = make(T, E, K, dtype, T + E)
    compare(z, idx, None, None, score)


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,K,S", [(1, 8, 2, 3), (64, 16, 2, 64), (65, 100, 4, 65), (700, 128, 8, 24), (3000, 40, 3, 5),
                                     (2500, 70, 2, 900), (4, 5, 1, 5000), (600, 9, 2, 130)])
def test_sequences_and_masks(dtype, score, T, E, K, S):
    """Sequences of any length, empty ones among them, that begin and end inside a run of tokens."""
    z, idx, seq, mask = make(T, E, K, dtype, T + S, S, True)
    compare(z, idx, seq, mask, score)
    compare(z, idx, seq, None, score)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_tokens_that_do_not_count_are_not_read(score):
    """NaN in masked tokens, before the first sequence and behind the last; all masked; empty sequences alone."""
    z, idx, _, mask = make(90, 24, 3, F32, 5, masked=True)
    seq = torch.tensor([7, 20, 20, 61, 80], dtype=torch.int32, device=DEV)
    ref = compare(z, idx, seq, mask, score)
    keep = mask.clone()
    keep[:7] = False
    keep[80:] = False
    z2, idx2 = z.clone(), idx.clone()
    z2[~keep], idx2[~keep] = math.nan, 1 << 30
    got = compare(torch.where(keep[:, None], z, z), idx, seq, mask, score)
    l2 = M.moe_balance(z2, idx2, seq, mask, score)
    for a, b in zip(l2, (ref["loss"], ref["counts"], ref["probs"], ref["tokens"])):
        assert torch.equal(a, b)
    gl = torch.ones(2, device=DEV)
    grad = M.moe_balance_bwd(z2, l2[1], l2[3], gl, 3, seq, mask, score)
    assert (grad[~keep] == 0).all() and torch.isfinite(grad).all() and got is not None
    none = torch.zeros(90, dtype=torch.uint8, device=DEV)
    loss, counts, probs, tokens = M.moe_balance(z2, idx2, seq, none, score)
    assert (loss == 0).all() and (counts == 0).all() and (probs == 0).all() and (tokens == 0).all()
    assert (M.moe_balance_bwd(z2, counts, tokens, gl, 3, seq, none, score) == 0).all()
    behind = torch.tensor([90, 90, 90], dtype=torch.int32, device=DEV)
    assert all((t == 0).all() for t in M.moe_balance(z2, idx2, behind, None, score))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_masked_experts_and_far_logits(dtype, score):
    """-inf and the type's lowest value in some places; tokens with nothing but -inf; far negative logits."""
    z, idx, _, _ = make(40, 70, 4, dtype, 8)
    z[:, 3:40:5] = -math.inf
    z[5:9, 10:60] = torch.finfo(dtype).min
    z[11] = -math.inf
    z[12, 1:] = -math.inf
    z[13] -= 300.0  # sigmoids below float32's range, each with its share
    if score == "sigmoid":
        z[14] = -800.0  # no score: no probability, and the z loss as ever
    got = compare(z, idx, None, None, score)
    assert torch.isfinite(got["grad"]).all() and (got["grad"][11] == 0).all()


def test_nan_and_infinity_spread():
    for bad in (math.nan, math.inf):
        z, idx, _, _ = make(30, 20, 2, F32, 9)
        z[4, 3] = bad
        seq = torch.tensor([0, 10, 30], dtype=torch.int32, device=DEV)
        loss, counts, probs, tokens = M.moe_balance(z, idx, seq)
        assert torch.isnan(loss[0]) and not torch.isfinite(loss[1])
        assert torch.isnan(probs[0]).all() and torch.isfinite(probs[1]).all()
        grad = M.moe_balance_bwd(z, counts, tokens, torch.ones(2, device=DEV), 2, seq)
        assert torch.isnan(grad[4]).any() and torch.isfinite(grad[:4]).all() and torch.isfinite(grad[5:]).all()


@pytest.mark.parametrize("itype", [torch.int32, torch.int64])
def test_ids_outside_the_experts_and_repeated_ones(itype):
    z, idx, _, _ = make(50, 12, 4, BF16, 3, itype=itype)
    idx[0], idx[1] = -1, 12
    idx[2] = torch.iinfo(itype).max
    idx[3] = torch.iinfo(itype).min
    idx[4] = 5
    if itype == torch.int64:
        idx[5] = (1 << 32) + 3
    compare(z, idx, None, None, "softmax")


def test_an_even_choice_has_loss_one():
    T, E, K = 64, 16, 4
    z = torch.zeros(T, E, device=DEV)
    idx = ((torch.arange(T, device=DEV)[:, None] * K + torch.arange(K, device=DEV)) % E).to(torch.int32)
    loss, counts, probs, tokens = M.moe_balance(z, idx)
    assert loss[0] == 1 and (counts == T * K // E).all() and (probs == T / E).all() and tokens[0] == T


def test_an_empty_batch():
    z, idx = torch.empty(0, 8, device=DEV), torch.empty(0, 2, dtype=torch.int32, device=DEV)
    for seq in (None, torch.zeros(4, dtype=torch.int32, device=DEV)):
        out = M.moe_balance(z, idx, seq)
        assert all((t == 0).all() for t in out) and out[1].shape == (1 if seq is None else 3, 8)
        assert M.moe_balance_bwd(z, out[1], out[3], torch.ones(2, device=DEV), 2, seq).shape == (0, 8)


def test_gradient_against_differences():
    """Central differences of the loss in float64: truncation h^2/6 |f'''|, with values of order 1 below 1e-5 at h = 1e-3."""
    for score in ("softmax", "sigmoid"):
        z, idx, seq, mask = make(13, 9, 3, F32, 4, 3, True)
        gl = torch.tensor([1.5, 0.25], device=DEV)
        _, counts, _, tokens = M.moe_balance(z, idx, seq, mask, score)
        grad = M.moe_balance_bwd(z, counts, tokens, gl, 3, seq, mask, score).cpu().double()
        h = 1e-3
        for t, e in ((0, 0), (3, 4), (7, 8), (12, 2)):
            two = []
            for d in (h, -h):
                zz = z.double()
                zz[t, e] += d
                two.append(float((reference(zz, idx, seq, mask, score, gl)["loss"][0] * gl.cpu().double()).sum()))
            assert abs((two[0] - two[1]) / (2 * h) - float(grad[t, e])) < 1e-5


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_base_gradient_in_place_and_results_repeat(dtype):
    z, idx, seq, mask = make(400, 40, 4, dtype, 6, 7, True)
    base = torch.randn(400, 40, device=DEV).to(dtype)
    got = compare(z, idx, seq, mask, "softmax", base)
    again = base.clone()
    out = M.moe_balance_bwd(z, got["counts"], got["tokens"], (torch.rand(2, generator=torch.Generator().manual_seed(0)) + 0.5).to(DEV),
                            4, seq, mask, grad_base=again, grad_logits=again)
    assert out is again and torch.equal(again, got["grad"])
    for _ in range(5):
        loss, counts, probs, tokens = M.moe_balance(z, idx, seq, mask)
        assert torch.equal(loss, got["loss"]) and torch.equal(probs, got["probs"]) and torch.equal(counts, got["counts"])


def test_given_buffers_and_what_lies_around_them():
    z, idx, seq, mask = make(100, 20, 2, F32, 7, 4, True)
    ref = M.moe_balance(z, idx, seq, mask)
    size = M.moe_balance_workspace_size(100, 20, 4)
    ws = torch.full((size + 512,), 171, dtype=torch.uint8, device=DEV)
    bufs = [torch.full((n + 8,), 7, dtype=d, device=DEV) for n, d in ((2, F32), (80, torch.int32), (80, F32), (4, torch.int32))]
    views = [bufs[0][:2], bufs[1][:80].view(4, 20), bufs[2][:80].view(4, 20), bufs[3][:4]]
    got = M.moe_balance(z, idx, seq, mask, "softmax", *views, workspace=ws)
    for a, b, v, buf in zip(got, ref, views, bufs):
        assert a is v and torch.equal(a, b) and (buf[-8:] == 7).all()
    assert (ws[size:] == 171).all()


def test_a_batch_of_many_tokens():
    """Offsets past 32 bits in the logits: 2^21 tokens of 1024 experts in bfloat16 (4 GiB)."""
    T, E, K = (1 << 21) + 5, 1024, 2
    z = torch.zeros(T, E, dtype=BF16, device=DEV)
    idx = torch.zeros(T, K, dtype=torch.int32, device=DEV)
    seq = torch.tensor([0, T - 6, T], dtype=torch.int32, device=DEV)
    tail, tidx, _, _ = make(6, E, K, BF16, 1)
    z[T - 6:], idx[T - 6:] = tail, tidx
    loss, counts, probs, tokens = M.moe_balance(z, idx, seq)
    one = M.moe_balance(tail, tidx)
    assert torch.equal(counts[1], one[1][0]) and tokens.tolist() == [T - 6, 6] and counts[0, 0] == K * (T - 6)
    assert torch.allclose(probs[1], one[2][0], rtol=64 * U, atol=0)
    assert torch.allclose(probs[0], torch.full_like(probs[0], (T - 6) / E), rtol=0.0, atol=0.0)  # powers of two: exact sums
    grad = M.moe_balance_bwd(z, counts, tokens, torch.tensor([2.0, 0.0], device=DEV), K, seq)
    ref = M.moe_balance_bwd(tail, one[1], one[3], torch.tensor([1.0, 0.0], device=DEV), K)  # one of two sequences: half
    assert torch.equal(grad[T - 6:], ref)


def test_refusals():
    z, idx, seq, mask = make(10, 8, 2, F32, 1, 2, True)
    with pytest.raises(ValueError):
        M.moe_balance(z, idx, seq, mask, "tanh")
    with pytest.raises(ValueError):
        M.moe_balance(z, idx[:5])
    with pytest.raises(ValueError):
        M.moe_balance(z, idx, seq.long())
    with pytest.raises(ValueError):
        M.moe_balance(z, idx, seq[:1])
    with pytest.raises(TypeError):
        M.moe_balance(z, idx, seq, mask.float())
    with pytest.raises(ValueError):
        M.moe_balance(z.t(), idx)
    with pytest.raises(ValueError):
        M.moe_balance(z.cpu(), idx)
    with pytest.raises(TypeError):
        M.moe_balance(z.half(), idx)
    with pytest.raises(M.api.MoeError):
        M.moe_balance(z, idx, workspace=torch.empty(16, dtype=torch.uint8, device=DEV))
