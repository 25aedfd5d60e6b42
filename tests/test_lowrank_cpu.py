"""The low-rank adapters' C ABI without a GPU: a handle that has no layout,
or is none, is refused before anything is launched."""
import ctypes

from test_abi_cpu import C, FAKE, L  # noqa: F401  (L is a fixture)


def test_lowrank_needs_a_layout(L):  # noqa: F811
    h = ctypes.c_void_p()
    assert L.moe_handle_create(ctypes.byref(h), None) == 0
    try:
        for handle, code in ((h, "MOE_ERR_HANDLE"), (None, "MOE_ERR_INVALID_ARG")):
            assert L.moe_lowrank(handle, FAKE, 1, 64, FAKE, FAKE, 2, 16, 64, None, None, FAKE, FAKE, None) == C[code]
            assert L.moe_lowrank_bwd(handle, FAKE, 1, 64, FAKE, FAKE, FAKE, 2, 16, 64, None, FAKE, None, FAKE, FAKE, FAKE,
                                     None, FAKE, 1 << 30, None) == C[code]
    finally:
        L.moe_handle_destroy(h)
