"""Products in 8-bit integers in every size of tile: segments of every length around the tiles' edges, several
column tiles, whole and partial steps, rows gathered by token, every activation and output type.

Sums and scales as in test_gpu_i8: without an activation outputs are equal to float32 arithmetic of known order,
bit for bit; with one they are off by 24 u |g up| (u = 2^-24), and eps/2 of themselves for the rounding.
"""
import math

import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24

# rows of each expert: none, one, and both sides of 16, 32, 64, 128, 256 and of what three row parts hold
ROWS = [0, 1, 15, 16, 17, 31, 48, 64, 65, 112, 127, 128, 129, 0, 240, 255, 256, 257, 300, 288, 289, 383, 384, 385, 513]
E, R = len(ROWS), sum(ROWS)


def tiles(rows, N, width, experts):
    """The rule by which the library takes its tiles (128 x 256, 64 x 128, 64 x 64), in whole numbers."""
    def most(bm, bn):
        return (rows // bm + (min(rows, experts) if experts else 1)) * -(-N // bn)
    if most(128, 256) >= (192 if width >= 2048 else 400):
        return "large"
    return "middle" if most(64, 128) >= 256 else "small"


def operands(rows, width, banks, N, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    q = torch.randint(-128, 128, (rows, width), generator=g, dtype=torch.int8, device=DEV)
    w = torch.randint(-128, 128, (banks, N, width), generator=g, dtype=torch.int8, device=DEV)
    s = (torch.rand(rows, generator=g, device=DEV) + 0.5) / 64
    ws = (torch.rand(banks, N, generator=g, device=DEV) + 0.5) * (width ** -0.5 / 64)
    return q, s, w, ws


def expected(q, s, w, ws, act, dtype):
    """(value, bound) of one expert's rows; sums in float64, exact below 2^53."""
    acc = torch.mm(q.double(), w.double().t().contiguous())
    if act is None:
        return ((acc.float() * s[:, None]) * ws).to(dtype), 0.0
    y = acc * s.double()[:, None] * ws.double()
    g, up = y.chunk(2, 1)
    if act == "silu":
        f = g / (1 + torch.exp(-g))
    else:
        f = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    ref, tol = f * up, 24 * U * (g * up).abs()
    return ref, tol + torch.finfo(dtype).eps / 2 * (ref.abs() + tol) + 1e-37


def check(got, ref, tol, what):
    if isinstance(tol, float):
        assert torch.equal(got, ref), what
    else:
        err = (got.double() - ref).abs()
        assert bool((err <= tol).all()), (what, float((err - tol).max()))


KINDS = [(None, F32), ("silu", BF16), ("gelu_tanh", F32), (None, BF16), ("silu", F32), ("gelu_tanh", BF16)]
SHAPES = [(16, 2064, "large"), (128, 2064, "large"), (272, 2304, "large"), (1024, 2304, "large"), (1040, 2064, "large"),
          (1280, 2064, "large"), (2064, 1040, "large"), (144, 1040, "middle"), (1040, 1040, "middle"), (1152, 1040, "middle"),
          (1280, 1040, "middle"), (2064, 656, "middle"), (144, 144, "small"), (1040, 144, "small"), (2064, 144, "small")]


@pytest.mark.parametrize("tokens", [True, False])
@pytest.mark.parametrize("width,N,size", SHAPES)
def test_segments_of_every_length(tokens, width, N, size):
    assert tiles(R, N, width, E) == size
    g = torch.Generator().manual_seed(width + N)
    idx = torch.repeat_interleave(torch.arange(E), torch.tensor(ROWS))[torch.randperm(R, generator=g)]
    h = M.moe_layout(idx.to(torch.int32).view(-1, 1).to(DEV), E, 1)
    q, s, w, ws = operands(R, width, E, N, width)
    token, off = h.field("recv_token").long(), h.field("expert_offset").tolist()
    assert [b - a for a, b in zip(off, off[1:])] == ROWS
    outs = []
    for act, dtype in KINDS:
        out = torch.full((R, N if act is None else N // 2), math.nan, dtype=dtype, device=DEV)
        outs.append(M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=tokens, activation=act, out=out))
    for e in range(E):
        at = slice(off[e], off[e + 1])
        rows = token[at] if tokens else torch.arange(off[e], off[e + 1], device=DEV)
        for (act, dtype), out in zip(KINDS, outs):
            ref, tol = expected(q[rows], s[rows], w[e], ws[e], act, dtype)
            check(out[at], ref, tol, (e, ROWS[e], act, dtype))


@pytest.mark.parametrize("width,N,size", [(400, 2064, "large"), (1040, 2064, "large"), (400, 656, "middle"), (1168, 656, "middle")])
def test_several_experts_a_token(width, N, size):
    """Each token's row is read by four experts, of very different numbers of tokens."""
    T, K, experts = 1000, 4, 16
    assert tiles(T * K, N, width, experts) == size
    g = torch.Generator().manual_seed(width)
    z = torch.randn(T, experts, generator=g) - 0.3 * torch.arange(experts)
    idx = torch.topk(z, K, 1)[1].to(torch.int32).to(DEV)
    h = M.moe_layout(idx, experts, 1)
    q, s, w, ws = operands(T, width, experts, N, width)
    token, off = h.field("recv_token").long(), h.field("expert_offset").tolist()
    assert min(b - a for a, b in zip(off, off[1:])) < 64 and max(b - a for a, b in zip(off, off[1:])) > 300
    for act, dtype in KINDS[:4]:
        out = M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True, activation=act, dtype=dtype)
        for e in range(experts):
            rows = token[off[e]:off[e + 1]]
            ref, tol = expected(q[rows], s[rows], w[e], ws[e], act, dtype)
            check(out[off[e]:off[e + 1]], ref, tol, (e, act, dtype))


@pytest.mark.parametrize("rows,width,N,size", [(4099, 400, 3344, "large"), (4099, 1296, 3344, "large"), (4099, 2192, 1552, "large"),
                                               (1030, 1040, 2064, "middle"), (1030, 2064, 2064, "middle")])
def test_without_a_layout(rows, width, N, size):
    assert tiles(rows, N, width, 0) == size
    q, s, w, ws = operands(rows, width, 1, N, rows)
    for act, dtype in KINDS:
        out = M.moe_matmul_i8(q, s, w[0], ws[0], activation=act, dtype=dtype)
        ref, tol = expected(q, s, w[0], ws[0], act, dtype)
        check(out, ref, tol, (act, dtype))


@pytest.mark.parametrize("N,size", [(2064, "large"), (1040, "middle"), (144, "small")])
@pytest.mark.parametrize("act", [None, "silu", "gelu_tanh"])
def test_padding_rows_are_zero_whatever_the_weights_scales(N, size, act):
    """Channels whose weights were not finite have an infinity or NaN as their scale: NaN in every token's row,
    and still zero in a row without a token."""
    h = M.Handle(pad_multiple=16)
    idx = torch.repeat_interleave(torch.arange(E), torch.tensor(ROWS)).to(torch.int32).view(-1, 1).to(DEV)
    M.moe_layout(idx, E, 1, handle=h)
    assert tiles(h.R, N, 144, E) == size
    q, s, w, ws = operands(R, 144, E, N, 5)
    plain = M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True, activation=act, dtype=F32)
    w[:, 3], ws[:, 3] = 0, math.inf
    w[:, N - 1], ws[:, N - 1] = 0, math.nan
    out = M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True, activation=act, dtype=F32)
    there = h.field("expert_offset")[-1]
    token = h.field("recv_token")[:there]
    out, plain = out[:there], plain[:there]
    assert int((token < 0).sum()) > 100 and (out[token < 0] == 0).all()
    bad = [3, N - 1] if act is None else [3, N // 2 - 1]
    keep = [n for n in range(out.shape[1]) if n not in bad]
    assert torch.isnan(out[token >= 0][:, bad]).all() and torch.equal(out[:, keep], plain[:, keep])


def test_far_gates_keep_their_digits():
    """silu(g) of whole g down to -80 to 9 u of itself: the exponential is off by 4 u of itself, the sum by u, the
    reciprocal by 2 u, the products with g and with up = 1 by u each."""
    q = torch.zeros(1, 16, dtype=torch.int8, device=DEV)
    q[0, 0] = 1
    g = torch.arange(-80, 48, device=DEV)
    w = torch.zeros(256, 16, dtype=torch.int8, device=DEV)
    w[:128, 0], w[128:, 0] = g.to(torch.int8), 1
    one = torch.ones(256, device=DEV)
    out = M.moe_matmul_i8(q, one[:1], w, one, activation="silu", dtype=F32)[0].double()
    ref = g.double() / (1 + torch.exp(-g.double()))
    assert bool(((out - ref).abs() <= 9 * U * ref.abs()).all()), float(((out - ref).abs() / ref.abs().clamp(min=1e-300)).max() / U)
