"""The balance loss's C ABI without a GPU: host validation refuses bad arguments
with the exact codes before anything is launched."""
import ctypes

import pytest

from test_abi_cpu import C, FAKE, L  # noqa: F401  (L is a fixture)

ORDER = ("z", "dtype", "T", "E", "idx", "itype", "K", "seq", "S", "mask", "score", "loss", "counts", "probs", "tokens",
         "ws", "ws_bytes")
GOOD = dict(z=FAKE, dtype=1, T=4, E=6, idx=FAKE, itype=0, K=2, seq=FAKE, S=3, mask=FAKE, score=0, loss=FAKE, counts=FAKE,
            probs=FAKE, tokens=FAKE, ws=FAKE, ws_bytes=1 << 20)
BORDER = ("z", "dtype", "T", "E", "K", "seq", "S", "mask", "score", "counts", "tokens", "grad_loss", "base", "grad")
BGOOD = dict(z=FAKE, dtype=1, T=4, E=6, K=2, seq=FAKE, S=3, mask=FAKE, score=0, counts=FAKE, tokens=FAKE, grad_loss=FAKE,
             base=FAKE, grad=FAKE)

SHARED = [
    (dict(T=-1), "MOE_ERR_INVALID_ARG"), (dict(S=-1), "MOE_ERR_INVALID_ARG"), (dict(score=2), "MOE_ERR_INVALID_ARG"),
    (dict(K=0), "MOE_ERR_SHAPE"), (dict(E=0), "MOE_ERR_SHAPE"), (dict(S=0), "MOE_ERR_SHAPE"),
    (dict(seq=None), "MOE_ERR_SHAPE"), (dict(K=33), "MOE_ERR_UNSUPPORTED"), (dict(E=1025), "MOE_ERR_UNSUPPORTED"),
    (dict(S=65536), "MOE_ERR_UNSUPPORTED"), (dict(T=(1 << 26) - 3), "MOE_ERR_UNSUPPORTED"),
    (dict(dtype=2), "MOE_ERR_UNSUPPORTED"), (dict(z=None), "MOE_ERR_INVALID_ARG"), (dict(z=FAKE + 1), "MOE_ERR_ALIGNMENT"),
    (dict(dtype=0, z=FAKE + 2), "MOE_ERR_ALIGNMENT"), (dict(seq=FAKE + 2), "MOE_ERR_ALIGNMENT"),
    (dict(counts=None), "MOE_ERR_INVALID_ARG"), (dict(tokens=None), "MOE_ERR_INVALID_ARG"),
    (dict(counts=FAKE + 2), "MOE_ERR_ALIGNMENT"), (dict(tokens=FAKE + 2), "MOE_ERR_ALIGNMENT")]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(itype=2), "MOE_ERR_UNSUPPORTED"), (dict(idx=None), "MOE_ERR_INVALID_ARG"), (dict(loss=None), "MOE_ERR_INVALID_ARG"),
    (dict(probs=None), "MOE_ERR_INVALID_ARG"), (dict(ws=None), "MOE_ERR_INVALID_ARG"),
    (dict(idx=FAKE + 2), "MOE_ERR_ALIGNMENT"), (dict(itype=1, idx=FAKE + 4), "MOE_ERR_ALIGNMENT"),
    (dict(loss=FAKE + 2), "MOE_ERR_ALIGNMENT"), (dict(probs=FAKE + 2), "MOE_ERR_ALIGNMENT"),
    (dict(ws=FAKE + 128), "MOE_ERR_ALIGNMENT"), (dict(ws_bytes=1), "MOE_ERR_WORKSPACE"),
    (dict(T=0, z=None, idx=None, loss=None), "MOE_ERR_INVALID_ARG")])
def test_balance_refusals(L, kw, code):  # noqa: F811
    a = dict(GOOD, **kw)
    assert L.moe_balance(*(a[n] for n in ORDER), None) == C[code]


@pytest.mark.parametrize("kw,code", SHARED + [
    (dict(grad_loss=None), "MOE_ERR_INVALID_ARG"), (dict(grad=None), "MOE_ERR_INVALID_ARG"),
    (dict(grad_loss=FAKE + 2), "MOE_ERR_ALIGNMENT"), (dict(base=FAKE + 1), "MOE_ERR_ALIGNMENT"),
    (dict(grad=FAKE + 1), "MOE_ERR_ALIGNMENT")])
def test_balance_bwd_refusals(L, kw, code):  # noqa: F811
    a = dict(BGOOD, **kw)
    assert L.moe_balance_bwd(*(a[n] for n in BORDER), None) == C[code]


def test_balance_empty_and_workspace(L):  # noqa: F811
    a = dict(BGOOD, T=0, z=None, counts=None, tokens=None, grad_loss=None, base=None, grad=None)
    assert L.moe_balance_bwd(*(a[n] for n in BORDER), None) == C["MOE_OK"]
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    f = L.moe_balance_workspace_size
    assert f(4096, 128, 1, ctypes.byref(n)) == 0 and n.value >= 128 * 8  # a count and a sum of every expert
    assert f(4096, 128, 64, ctypes.byref(m)) == 0 and m.value > n.value
    exact = dict(GOOD, T=4096, E=128, S=64, K=1, ws_bytes=m.value - 1)
    assert L.moe_balance(*(exact[n] for n in ORDER), None) == C["MOE_ERR_WORKSPACE"]
    assert f(0, 1, 1, ctypes.byref(n)) == 0 and n.value > 0
    assert f(4, 1025, 1, ctypes.byref(n)) == C["MOE_ERR_UNSUPPORTED"]
    assert f(4, 8, 0, ctypes.byref(n)) == C["MOE_ERR_SHAPE"]
    assert f(4, 8, 1, None) == C["MOE_ERR_INVALID_ARG"]
