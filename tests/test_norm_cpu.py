"""The norms' C ABI without a GPU: host validation refuses bad arguments with
the exact codes before anything is launched."""
import ctypes
import math

import pytest

from test_abi_cpu import C, FAKE, L  # noqa: F401  (L is a fixture)

PRE = dict(x=FAKE, dtype=1, T=3, H=32, w=FAKE, offset=0.0, eps=1e-6, n=FAKE, q=None, scale=None, rstd=FAKE)
POST = dict(h=None, x=FAKE, y=FAKE, dtype=1, T=6, H=32, tw=None, w=FAKE, gate=FAKE, G=2, a=1.0, nw=FAKE, offset=0.0, eps=1e-6,
            out=FAKE, n=FAKE, rstd=FAKE)
PRE_BWD = dict(gn=FAKE, x=FAKE, dtype=1, T=3, H=32, w=FAKE, offset=0.0, rstd=FAKE, base=FAKE, gx=FAKE, gw=FAKE, ws=FAKE,
               ws_bytes=1 << 20)
POST_BWD = dict(g=FAKE, gn=FAKE, x=FAKE, y=FAKE, dtype=1, T=6, H=32, rstd=FAKE, w=FAKE, gate=FAKE, G=2, a=1.0, nw=FAKE,
                offset=0.0, gx=FAKE, gy=FAKE, gw=FAKE, gg=FAKE, gnw=FAKE, ws=FAKE, ws_bytes=1 << 20)

ROWS = [(dict(T=-1), "MOE_ERR_INVALID_ARG"), (dict(H=0), "MOE_ERR_SHAPE"), (dict(H=20), "MOE_ERR_SHAPE"),
        (dict(dtype=0, H=6), "MOE_ERR_SHAPE"), (dict(dtype=2), "MOE_ERR_UNSUPPORTED"),
        (dict(T=(1 << 26) + 1), "MOE_ERR_UNSUPPORTED"), (dict(H=32776), "MOE_ERR_UNSUPPORTED"),
        (dict(dtype=0, H=16388), "MOE_ERR_UNSUPPORTED"), (dict(offset=math.inf), "MOE_ERR_INVALID_ARG"),
        (dict(x=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(w=FAKE + 8), "MOE_ERR_ALIGNMENT")]
EPS = [(dict(eps=0.0), "MOE_ERR_INVALID_ARG"), (dict(eps=-1.0), "MOE_ERR_INVALID_ARG"),
       (dict(eps=math.nan), "MOE_ERR_INVALID_ARG"), (dict(eps=math.inf), "MOE_ERR_INVALID_ARG"),
       (dict(x=None), "MOE_ERR_INVALID_ARG")]


@pytest.mark.parametrize("kw,code", ROWS + EPS + [
    (dict(w=None), "MOE_ERR_INVALID_ARG"), (dict(n=None), "MOE_ERR_INVALID_ARG"), (dict(q=FAKE), "MOE_ERR_INVALID_ARG"),
    (dict(n=None, q=FAKE), "MOE_ERR_INVALID_ARG"), (dict(n=None, q=FAKE, scale=FAKE, H=24), "MOE_ERR_SHAPE"),
    (dict(n=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(rstd=FAKE + 2), "MOE_ERR_ALIGNMENT"),
    (dict(n=None, q=FAKE + 8, scale=FAKE), "MOE_ERR_ALIGNMENT"), (dict(n=None, q=FAKE, scale=FAKE + 2), "MOE_ERR_ALIGNMENT")])
def test_prenorm_refusals(L, kw, code):  # noqa: F811
    assert L.moe_prenorm(*dict(PRE, **kw).values(), None) == C[code]


@pytest.mark.parametrize("kw,code", ROWS + EPS + [
    (dict(a=math.nan), "MOE_ERR_INVALID_ARG"), (dict(G=-1), "MOE_ERR_INVALID_ARG"), (dict(G=4), "MOE_ERR_SHAPE"),
    (dict(G=12), "MOE_ERR_SHAPE"), (dict(G=0), "MOE_ERR_INVALID_ARG"), (dict(gate=None), "MOE_ERR_INVALID_ARG"),
    (dict(n=None), "MOE_ERR_INVALID_ARG"), (dict(nw=None), "MOE_ERR_INVALID_ARG"), (dict(y=None), "MOE_ERR_INVALID_ARG"),
    (dict(out=None), "MOE_ERR_INVALID_ARG"), (dict(tw=FAKE), "MOE_ERR_INVALID_ARG"), (dict(y=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(gate=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(nw=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(out=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(n=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(rstd=FAKE + 4), "MOE_ERR_ALIGNMENT")])
def test_postnorm_refusals(L, kw, code):  # noqa: F811
    assert L.moe_postnorm(*dict(POST, **kw).values(), None) == C[code]


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(gn=None), "MOE_ERR_INVALID_ARG"), (dict(x=None), "MOE_ERR_INVALID_ARG"), (dict(w=None), "MOE_ERR_INVALID_ARG"),
    (dict(rstd=None), "MOE_ERR_INVALID_ARG"), (dict(gx=None, gw=None), "MOE_ERR_INVALID_ARG"),
    (dict(ws=None), "MOE_ERR_INVALID_ARG"), (dict(ws_bytes=3 * 32 * 4 - 1), "MOE_ERR_WORKSPACE"),
    (dict(gn=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(base=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(gx=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(gw=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(ws=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(rstd=FAKE + 2), "MOE_ERR_ALIGNMENT")])
def test_prenorm_bwd_refusals(L, kw, code):  # noqa: F811
    assert L.moe_prenorm_bwd(*dict(PRE_BWD, **kw).values(), None) == C[code]


@pytest.mark.parametrize("kw,code", ROWS + [
    (dict(a=math.inf), "MOE_ERR_INVALID_ARG"), (dict(G=-1), "MOE_ERR_INVALID_ARG"), (dict(G=4), "MOE_ERR_SHAPE"),
    (dict(G=0, gate=None), "MOE_ERR_INVALID_ARG"), (dict(gate=None), "MOE_ERR_INVALID_ARG"),
    (dict(g=None, gn=None), "MOE_ERR_INVALID_ARG"), (dict(nw=None), "MOE_ERR_INVALID_ARG"), (dict(x=None), "MOE_ERR_INVALID_ARG"),
    (dict(y=None), "MOE_ERR_INVALID_ARG"), (dict(w=None), "MOE_ERR_INVALID_ARG"),
    (dict(gn=None, nw=None), "MOE_ERR_INVALID_ARG"), (dict(rstd=None), "MOE_ERR_INVALID_ARG"),
    (dict(gx=None, gy=None, gw=None, gg=None, gnw=None), "MOE_ERR_INVALID_ARG"), (dict(ws=None), "MOE_ERR_INVALID_ARG"),
    (dict(ws_bytes=64), "MOE_ERR_WORKSPACE"), (dict(g=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(gn=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(y=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(gy=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(gg=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(gnw=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(rstd=FAKE + 4), "MOE_ERR_ALIGNMENT"), (dict(ws=FAKE + 8), "MOE_ERR_ALIGNMENT")])
def test_postnorm_bwd_refusals(L, kw, code):  # noqa: F811
    assert L.moe_postnorm_bwd(*dict(POST_BWD, **kw).values(), None) == C[code]


def test_wide_rows_need_the_workspace(L):  # noqa: F811
    """Rows past MOE_NORM_WIDE after a block go backward in two kernels, which meet in the workspace."""
    one = dict(POST_BWD, H=8200, gw=None, gg=None, gnw=None)
    assert L.moe_postnorm_bwd(*dict(one, ws=None).values(), None) == C["MOE_ERR_INVALID_ARG"]
    assert L.moe_postnorm_bwd(*dict(one, ws_bytes=64).values(), None) == C["MOE_ERR_WORKSPACE"]
    n, m = ctypes.c_size_t(), ctypes.c_size_t()
    f = L.moe_norm_bwd_workspace_size
    assert f(1, 4096, 8200, 1, ctypes.byref(n)) == 0 and n.value >= 64 * 8200 * 12 + 4096 * 8
    assert f(1, 4096, 8192, 1, ctypes.byref(m)) == 0 and m.value == 256 * 8192 * 12


def test_handles_empty_calls_and_workspace(L):  # noqa: F811
    h = ctypes.c_void_p()
    assert L.moe_handle_create(ctypes.byref(h), None) == C["MOE_OK"]
    assert L.moe_postnorm(*dict(POST, h=h).values(), None) == C["MOE_ERR_HANDLE"]
    L.moe_handle_destroy(h)
    none = dict.fromkeys(("x", "w", "n", "rstd"))
    assert L.moe_prenorm(*dict(PRE, T=0, **none).values(), None) == C["MOE_OK"]
    none = dict.fromkeys(("x", "y", "w", "gate", "nw", "out", "n", "rstd"))
    assert L.moe_postnorm(*dict(POST, T=0, **none).values(), None) == C["MOE_OK"]
    none = dict.fromkeys(("g", "gn", "x", "y", "rstd", "w", "gate", "nw", "gx", "gy", "gw", "gg", "gnw", "ws"))
    assert L.moe_postnorm_bwd(*dict(POST_BWD, T=0, **none).values(), None) == C["MOE_OK"]
    n = ctypes.c_size_t()
    f = L.moe_norm_bwd_workspace_size
    assert f(1, 4096, 2048, 8, ctypes.byref(n)) == 0 and n.value >= 3 * 8 * 2048 * 4
    assert f(0, 0, 2048, 0, ctypes.byref(n)) == 0 and n.value == 0
    assert f(1, 10, 2048, 4, ctypes.byref(n)) == C["MOE_ERR_SHAPE"]
    assert f(1, 10, 2048, -1, ctypes.byref(n)) == C["MOE_ERR_INVALID_ARG"]
    assert f(1, 10, 2044, 1, ctypes.byref(n)) == C["MOE_ERR_SHAPE"]
    assert f(1, 0, 2048, 65534, ctypes.byref(n)) == C["MOE_ERR_UNSUPPORTED"]
    assert f(2, 10, 2048, 1, ctypes.byref(n)) == C["MOE_ERR_UNSUPPORTED"]
    assert f(1, 10, 2048, 1, None) == C["MOE_ERR_INVALID_ARG"]
