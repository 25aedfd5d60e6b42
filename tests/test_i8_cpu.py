"""The 8-bit products' C ABI without a GPU: host validation refuses bad
arguments with the exact codes before anything is launched."""
import ctypes

import pytest

from test_abi_cpu import C, FAKE, L  # noqa: F401  (L is a fixture)

QORDER = ("x", "dtype", "rows", "width", "q", "scale")
QGOOD = dict(x=FAKE, dtype=1, rows=3, width=32, q=FAKE, scale=FAKE)
ORDER = ("h", "q", "scale", "rows", "width", "tokens", "w", "w_scale", "E", "first", "N", "act", "out", "dtype")
GOOD = dict(h=None, q=FAKE, scale=FAKE, rows=3, width=32, tokens=0, w=FAKE, w_scale=FAKE, E=1, first=0, N=32, act=-1,
            out=FAKE, dtype=1)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "MOE_ERR_INVALID_ARG"), (dict(width=0), "MOE_ERR_SHAPE"), (dict(width=24), "MOE_ERR_SHAPE"),
    (dict(dtype=2), "MOE_ERR_UNSUPPORTED"), (dict(width=131072), "MOE_ERR_UNSUPPORTED"),
    (dict(rows=(1 << 26) - 3), "MOE_ERR_UNSUPPORTED"), (dict(x=None), "MOE_ERR_INVALID_ARG"),
    (dict(q=None), "MOE_ERR_INVALID_ARG"), (dict(scale=None), "MOE_ERR_INVALID_ARG"),
    (dict(x=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(q=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(scale=FAKE + 2), "MOE_ERR_ALIGNMENT")])
def test_quant_refusals(L, kw, code):  # noqa: F811
    a = dict(QGOOD, **kw)
    assert L.moe_quant_rows(*(a[n] for n in QORDER), None) == C[code]


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), "MOE_ERR_INVALID_ARG"), (dict(tokens=2), "MOE_ERR_INVALID_ARG"), (dict(tokens=1), "MOE_ERR_INVALID_ARG"),
    (dict(act=2), "MOE_ERR_INVALID_ARG"), (dict(act=-2), "MOE_ERR_INVALID_ARG"), (dict(dtype=2), "MOE_ERR_UNSUPPORTED"),
    (dict(E=0), "MOE_ERR_SHAPE"), (dict(E=2), "MOE_ERR_SHAPE"), (dict(first=1), "MOE_ERR_SHAPE"),
    (dict(first=-1), "MOE_ERR_SHAPE"), (dict(width=0), "MOE_ERR_SHAPE"), (dict(width=40), "MOE_ERR_SHAPE"),
    (dict(N=0), "MOE_ERR_SHAPE"), (dict(N=12), "MOE_ERR_SHAPE"), (dict(N=24, act=0), "MOE_ERR_SHAPE"),
    (dict(N=33, act=0), "MOE_ERR_SHAPE"), (dict(dtype=0, N=6), "MOE_ERR_SHAPE"),
    (dict(width=131072), "MOE_ERR_UNSUPPORTED"), (dict(N=(1 << 20) + 8), "MOE_ERR_UNSUPPORTED"),
    (dict(N=1 << 16, width=1 << 15), "MOE_ERR_UNSUPPORTED"), (dict(rows=(1 << 26) + 1), "MOE_ERR_UNSUPPORTED"),
    (dict(q=None), "MOE_ERR_INVALID_ARG"), (dict(scale=None), "MOE_ERR_INVALID_ARG"), (dict(w=None), "MOE_ERR_INVALID_ARG"),
    (dict(w_scale=None), "MOE_ERR_INVALID_ARG"), (dict(out=None), "MOE_ERR_INVALID_ARG"),
    (dict(q=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(w=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(out=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(scale=FAKE + 2), "MOE_ERR_ALIGNMENT"),
    (dict(w_scale=FAKE + 2), "MOE_ERR_ALIGNMENT")])
def test_matmul_refusals(L, kw, code):  # noqa: F811
    a = dict(GOOD, **kw)
    assert L.moe_matmul_i8(*(a[n] for n in ORDER), None) == C[code]


def test_a_handle_without_a_layout_and_empty_calls(L):  # noqa: F811
    h = ctypes.c_void_p()
    assert L.moe_handle_create(ctypes.byref(h), None) == C["MOE_OK"]
    a = dict(GOOD, h=h)
    assert L.moe_matmul_i8(*(a[n] for n in ORDER), None) == C["MOE_ERR_HANDLE"]
    L.moe_handle_destroy(h)
    a = dict(GOOD, rows=0, q=None, scale=None, w=None, w_scale=None, out=None)
    assert L.moe_matmul_i8(*(a[n] for n in ORDER), None) == C["MOE_OK"]
    a = dict(QGOOD, rows=0, x=None, q=None, scale=None)
    assert L.moe_quant_rows(*(a[n] for n in QORDER), None) == C["MOE_OK"]
