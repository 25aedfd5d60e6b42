"""Gradients of the norms' weights and gates as sums over many tokens, against values known exactly."""
import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32 = torch.float32
U = 2.0 ** -24
# a number whose sum in 32 bits rounds to the same side again and again: 2048 of them are off by 511 u
STEP = 0.98614501953125


def ones(T, H):
    """Rows whose mean square is 1 and whose root mean square with eps = 1e-30 is 1: every term below is STEP."""
    return torch.ones(T, H, device=DEV), torch.full((T, H), STEP, device=DEV), torch.ones(H, device=DEV)


def near(t, n):
    """n terms of STEP: at most 256 are added in 32 bits, their sums in 64, and the result is rounded once."""
    err = float((t.double() / (n * STEP) - 1).abs().max())
    assert err <= 257 * U, err / U


@pytest.mark.parametrize("T,H", [(1 << 21, 4), ((1 << 21) + 300, 8), (1 << 20, 260), (1 << 19, 1028)])
def test_before_a_block(T, H):
    x, gn, w = ones(T, H)
    _, rstd = M.moe_prenorm(x, w, 1e-30)
    assert (rstd == 1).all()
    near(M.moe_prenorm_bwd(gn, x, rstd, w, grad_x=False)[1], T)


@pytest.mark.parametrize("T,H,G", [(1 << 21, 4, 1), (1 << 21, 8, 0), (1 << 20, 260, 2), (1 << 21, 4, 1 << 12), (1 << 21, 4, 1 << 18),
                                   (257 * 70000, 4, 70000), (1 << 18, 8200, 1)])
def test_after_a_block(T, H, G):
    """Also more gates of several parts than one dimension of a grid has workgroups."""
    x, g, w = ones(T, H)
    gate = torch.ones(G, H, device=DEV) if G else None
    _, _, rstd = M.moe_postnorm(x, x, w, gate, 1.0, eps=1e-30, out=x)
    x.fill_(1.0)
    assert (rstd == 1).all()
    _, _, gw, gg, _ = M.moe_postnorm_bwd(g, None, x, x, rstd, w, gate, grad_x=False, grad_y=False)
    near(gw, T)
    if G:
        near(gg, T // G)
