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
