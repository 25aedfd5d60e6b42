"""The few-token expert layer's C ABI without a GPU: host validation refuses
bad arguments with the exact codes before anything is launched."""
import ctypes

import pytest

from test_abi_cpu import C, FAKE, L  # noqa: F401  (L is a fixture)

ORDER = ("x", "dtype", "T", "H", "idx", "itype", "K", "w", "w13", "w2", "E", "I", "act", "out", "ws", "ws_bytes")
GOOD = dict(x=FAKE, dtype=1, T=4, H=64, idx=FAKE, itype=0, K=2, w=FAKE, w13=FAKE, w2=FAKE, E=6, I=32, act=0, out=FAKE,
            ws=FAKE, ws_bytes=4 * 2 * 32 * 2)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), "MOE_ERR_INVALID_ARG"), (dict(K=0), "MOE_ERR_SHAPE"), (dict(E=0), "MOE_ERR_SHAPE"),
    (dict(H=0), "MOE_ERR_SHAPE"), (dict(I=0), "MOE_ERR_SHAPE"), (dict(H=60), "MOE_ERR_SHAPE"),
    (dict(I=36), "MOE_ERR_SHAPE"), (dict(dtype=0, I=34), "MOE_ERR_SHAPE"), (dict(dtype=2), "MOE_ERR_UNSUPPORTED"),
    (dict(K=33), "MOE_ERR_UNSUPPORTED"), (dict(E=1025), "MOE_ERR_UNSUPPORTED"), (dict(T=257), "MOE_ERR_UNSUPPORTED"),
    (dict(T=1 << 62), "MOE_ERR_UNSUPPORTED"), (dict(H=1 << 21), "MOE_ERR_UNSUPPORTED"),
    (dict(I=1 << 21), "MOE_ERR_UNSUPPORTED"), (dict(itype=2), "MOE_ERR_UNSUPPORTED"),
    (dict(act=2), "MOE_ERR_INVALID_ARG"), (dict(x=None), "MOE_ERR_INVALID_ARG"), (dict(idx=None), "MOE_ERR_INVALID_ARG"),
    (dict(w13=None), "MOE_ERR_INVALID_ARG"), (dict(w2=None), "MOE_ERR_INVALID_ARG"),
    (dict(out=None), "MOE_ERR_INVALID_ARG"), (dict(ws=None), "MOE_ERR_INVALID_ARG"),
    (dict(x=FAKE + 8), "MOE_ERR_ALIGNMENT"), (dict(w13=FAKE + 8), "MOE_ERR_ALIGNMENT"),
    (dict(w2=FAKE + 2), "MOE_ERR_ALIGNMENT"), (dict(out=FAKE + 4), "MOE_ERR_ALIGNMENT"),
    (dict(ws=FAKE + 128), "MOE_ERR_ALIGNMENT"), (dict(idx=FAKE + 2), "MOE_ERR_ALIGNMENT"),
    (dict(idx=FAKE + 4, itype=1), "MOE_ERR_ALIGNMENT"), (dict(w=FAKE + 2), "MOE_ERR_ALIGNMENT"),
    (dict(ws_bytes=511), "MOE_ERR_WORKSPACE")])
def test_few_refusals(L, kw, code):  # noqa: F811
    a = dict(GOOD, **kw)
    assert L.moe_few(*(a[n] for n in ORDER), None) == C[code]


def test_few_empty_and_workspace(L):  # noqa: F811
    a = dict(GOOD, T=0, x=None, idx=None, w=None, w13=None, w2=None, out=None, ws=None, ws_bytes=0)
    assert L.moe_few(*(a[n] for n in ORDER), None) == C["MOE_OK"]
    n = ctypes.c_size_t()
    assert L.moe_few_workspace_size(1, 4, 2, 32, ctypes.byref(n)) == 0 and n.value == 1024
    assert L.moe_few_workspace_size(0, 512, 1, 4, ctypes.byref(n)) == 0 and n.value == 8192
    assert L.moe_few_workspace_size(0, 513, 1, 4, ctypes.byref(n)) == C["MOE_ERR_UNSUPPORTED"]
    assert L.moe_few_workspace_size(3, 4, 1, 4, ctypes.byref(n)) == C["MOE_ERR_UNSUPPORTED"]
    assert L.moe_few_workspace_size(1, 4, 2, 32, None) == C["MOE_ERR_INVALID_ARG"]
