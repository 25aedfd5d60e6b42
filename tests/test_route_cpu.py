"""The router's C ABI without a GPU: host validation refuses bad arguments
with the exact codes before anything is launched."""
import ctypes

import pytest

from test_abi_cpu import C, FAKE, L  # noqa: F401  (L is a fixture)


def options(**kw):
    from combine_moe_layout_04_amd._lib import MoeRouteOptions
    o = dict(score=0, renormalize=1, num_groups=1, topk_groups=1, scale=1.0)
    o.update(kw)
    return ctypes.byref(MoeRouteOptions(*[o[n] for n, _ in MoeRouteOptions._fields_]))


CASES = [
    (dict(T=-1), {}, "MOE_ERR_INVALID_ARG"), (dict(K=0), {}, "MOE_ERR_SHAPE"), (dict(K=17), {}, "MOE_ERR_SHAPE"),
    (dict(E=0), {}, "MOE_ERR_SHAPE"), (dict(E=1025), {}, "MOE_ERR_UNSUPPORTED"),
    (dict(E=64, K=33), {}, "MOE_ERR_UNSUPPORTED"), (dict(T=1 << 31), {}, "MOE_ERR_UNSUPPORTED"),
    (dict(T=1 << 29), {}, "MOE_ERR_UNSUPPORTED"), (dict(T=1 << 26, K=1), {}, "MOE_ERR_UNSUPPORTED"), (dict(dtype=2), {}, "MOE_ERR_UNSUPPORTED"),
    ({}, dict(score=2), "MOE_ERR_INVALID_ARG"), ({}, dict(renormalize=2), "MOE_ERR_INVALID_ARG"),
    ({}, dict(scale=float("nan")), "MOE_ERR_INVALID_ARG"), ({}, dict(num_groups=0), "MOE_ERR_SHAPE"),
    ({}, dict(num_groups=4, topk_groups=5), "MOE_ERR_SHAPE"), ({}, dict(num_groups=3), "MOE_ERR_SHAPE"),
    ({}, dict(num_groups=8, topk_groups=1), "MOE_ERR_SHAPE"), ({}, dict(topk_groups=0), "MOE_ERR_SHAPE"),
    (dict(E=1024), dict(num_groups=128, topk_groups=64), "MOE_ERR_UNSUPPORTED"),
    (dict(z=None), {}, "MOE_ERR_INVALID_ARG"), (dict(idx=None), {}, "MOE_ERR_INVALID_ARG"),
    (dict(w=None), {}, "MOE_ERR_INVALID_ARG"), (dict(z=FAKE + 2), {}, "MOE_ERR_ALIGNMENT"),
    (dict(idx=FAKE + 1), {}, "MOE_ERR_ALIGNMENT"), (dict(w=FAKE + 2), {}, "MOE_ERR_ALIGNMENT"),
]


@pytest.mark.parametrize("kw,opt,code", CASES)
def test_route_refusals(L, kw, opt, code):  # noqa: F811
    a = dict(z=FAKE, dtype=0, T=4, E=16, K=4, idx=FAKE, w=FAKE)
    a.update(kw)
    head = (a["z"], a["dtype"], a["T"], a["E"], a["K"], options(**opt))
    assert L.moe_route(*head, None, a["idx"], a["w"], None) == C[code]
    assert L.moe_route_bwd(*head, a["idx"], a["w"], FAKE, None) == C[code]


def test_route_null_options_bias_and_empty(L):  # noqa: F811
    assert L.moe_route(FAKE, 0, 4, 16, 4, None, None, FAKE, FAKE, None) == C["MOE_ERR_INVALID_ARG"]
    assert L.moe_route(FAKE, 0, 4, 16, 4, options(), FAKE + 2, FAKE, FAKE, None) == C["MOE_ERR_ALIGNMENT"]
    assert L.moe_route_bwd(FAKE, 0, 4, 16, 4, options(), FAKE, FAKE, None, None) == C["MOE_ERR_INVALID_ARG"]
    assert L.moe_route(None, 0, 0, 16, 4, options(), None, None, None, None) == C["MOE_OK"]
    assert L.moe_route_bwd(None, 0, 0, 16, 4, options(), None, None, None, None) == C["MOE_OK"]


def test_options_go_by_value():
    import torch
    from combine_moe_layout_04_amd import api

    def scale(o):
        return o._obj.scale

    s = torch.tensor(1.5)
    assert scale(api._route_options("softmax", True, 1, 1, s)) == 1.5
    s += 1
    assert scale(api._route_options("softmax", True, 1, 1, s)) == 2.5
    for bad in (2 ** 32 + 1, -1):
        with pytest.raises(ValueError):
            api._route_options("softmax", True, bad, 1, 1.0)


def test_the_most_tokens(L):  # noqa: F811
    for T, code in ((2 ** 26 - 4, "MOE_OK"), (2 ** 26 - 3, "MOE_ERR_UNSUPPORTED"), (2 ** 26 - 1, "MOE_ERR_UNSUPPORTED")):
        # a bad pointer is refused after the sizes are
        want = C["MOE_ERR_INVALID_ARG"] if code == "MOE_OK" else C[code]
        assert L.moe_route(None, 0, T, 1, 1, options(), None, FAKE, FAKE, None) == want
        assert L.moe_route_bwd(None, 0, T, 1, 1, options(), FAKE, FAKE, FAKE, None) == want
