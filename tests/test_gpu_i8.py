"""Rows in 8 bits and the products with them against exact arithmetic.

The rows' scales and integers are equal to the definition's.  A product's sum is exact in integers;
what follows is float32 arithmetic of known order (the sum's conversion, times the row's scale, times
the channel's), so without an activation outputs are equal to it, bit for bit.  With one, u = 2^-24:
gate and up are off by 3 u of themselves, |f'| <= 1.13, |f(g)| <= |g| and 16 u |g| for the
exponential or tanh with their arguments, so the result is off by 24 u |g up|, and eps/2 of itself
for the rounding.
"""
import math

import pytest
import torch

import combine_moe_layout_04_amd as M

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
F32, BF16 = torch.float32, torch.bfloat16
U = 2.0 ** -24


def exact_quant(x):
    """On the CPU: the scale is one float32 division; a float64 quotient of two float32 numbers is
    not rounded onto a half that it is not."""
    x = x.cpu()
    top = x.abs().amax(-1).float()
    s = torch.maximum(top / 127, torch.tensor(2.0 ** -126))
    return torch.round(x.double() / s.double()[..., None]).to(torch.int8), s


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,width", [(1, 16), (3, 32), (5, 624), (257, 768), (64, 2048), (7, 2064), (3, 7168), (2, 16400),
                                        (2, 131056), (1025, 48), (4, 1008), (4, 1024), (4, 1040)])
def test_rows_are_the_definitions(dtype, rows, width):
    g = torch.Generator().manual_seed(rows + width)
    x = (torch.randn(rows, width, generator=g) * torch.exp(4 * torch.randn(rows, 1, generator=g))).to(dtype)
    q, s = M.moe_quant_rows(x.to(DEV))
    rq, rs = exact_quant(x)
    assert q.dtype == torch.int8 and q.shape == x.shape and torch.equal(s.cpu(), rs) and torch.equal(q.cpu(), rq)


def test_values_next_to_a_half():
    """Rows with scale 1, 1/3 and others, and values at and one step beside every half."""
    for top in (127.0, 127 / 3, 1e-30, 3e38, 5.25, 2.0 ** -119, 1.17e-38):
        s = torch.maximum(torch.tensor(top) / 127, torch.tensor(2.0 ** -126))
        half = ((torch.arange(-127, 127) + 0.5).double() * s.double()).float()
        up, down = torch.nextafter(half, torch.tensor(math.inf)), torch.nextafter(half, torch.tensor(-math.inf))
        x = torch.cat([torch.tensor([top, -top]), half, up, down])
        x = x[x.abs() <= top]
        x = torch.cat([x, torch.zeros(-len(x) % 16)])[None]
        q, sc = M.moe_quant_rows(x.to(DEV))
        rq, rs = exact_quant(x)
        assert torch.equal(sc.cpu(), rs) and torch.equal(q.cpu(), rq), top


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_zeros_the_smallest_and_what_is_not_finite(dtype):
    x = torch.zeros(8, 32, dtype=dtype)
    x[1] = torch.finfo(dtype).tiny
    x[2, 3] = torch.finfo(dtype).max
    x[3, 4] = -math.inf
    x[4, 5] = math.nan
    x[5, 6], x[5, 7] = math.inf, math.nan
    x[6, 0] = 1.0
    x[7] = 2.0 ** -133
    q, s = (t.cpu() for t in M.moe_quant_rows(x.to(DEV)))
    rq, rs = exact_quant(x)
    for r in (0, 1, 2, 6, 7):
        assert torch.equal(q[r], rq[r]) and s[r] == rs[r]
    assert s[3] == math.inf and torch.isnan(s[4]) and torch.isnan(s[5]) and (q[3:6] == 0).all()
    w = torch.ones(16, 32, dtype=torch.int8, device=DEV)
    y = M.moe_matmul_i8(q.to(DEV), s.to(DEV), w, torch.ones(16, device=DEV), dtype=F32)
    assert torch.isnan(y[3:6]).all() and torch.isfinite(y[[0, 1, 6, 7]]).all()
    # float32's largest number m: m / 127 is rounded up, so 127 of them lie above m + ulp(m) / 2 and are
    # infinite in float32; bfloat16's largest is 2^120 below m, where there is room
    m = torch.finfo(torch.float32).max
    s2 = torch.tensor(m) / 127
    assert 127 * float(s2) >= m + 2.0 ** 103 and s2 * 127 == math.inf
    assert torch.equal(y[2].cpu(), (127.0 * s[2]).expand(16)) and (dtype == F32 or torch.isfinite(y[2]).all())


def bank(E, N, width, seed):
    g = torch.Generator().manual_seed(seed)
    w = torch.randint(-128, 128, (E, N, width), generator=g, dtype=torch.int8)
    return w.to(DEV), (torch.rand(E, N, generator=g) + 0.5).to(DEV) * width ** -0.5 / 64


def rows8(M_, width, seed):
    g = torch.Generator().manual_seed(seed)
    q = torch.randint(-128, 128, (M_, width), generator=g, dtype=torch.int8)
    return q.to(DEV), (torch.rand(M_, generator=g) + 0.5).to(DEV) / 64


def scaled(acc, s, ws):
    """float(acc) * s * ws in float32, each rounded on its own."""
    return (acc.to(torch.float32) * s[:, None]) * ws


def check(got, q, s, w, ws, act, dtype, what=""):
    """got [n, cols] against rows q [n, width] with one expert's weights, on the CPU."""
    acc = (q.cpu().double() @ w.cpu().double().t()).round().long()  # below 2^53: exact
    y = scaled(acc, s.cpu(), ws.cpu())
    if act is None:
        ref = y.to(dtype)
        assert torch.equal(got.cpu(), ref), what
        return
    n = y.shape[1] // 2
    y = (acc.double() * s.cpu().double()[:, None]) * ws.cpu().double()
    g, up = y[:, :n], y[:, n:]
    if act == "silu":
        f = g / (1 + torch.exp(-g))
    else:
        f = 0.5 * g * (1 + torch.tanh(math.sqrt(2 / math.pi) * (g + 0.044715 * g ** 3)))
    ref = f * up
    tol = 24 * U * (g * up).abs()
    tol = tol + torch.finfo(dtype).eps / 2 * (ref.abs() + tol) + 1e-37
    err = (got.cpu().double() - ref).abs()
    assert bool((err <= tol).all()), (what, float((err - tol).max()))


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("act", [None, "silu", "gelu_tanh"])
@pytest.mark.parametrize("rows,width,N", [
    (1, 16, 16), (1, 2048, 1536), (3, 32, 48), (15, 48, 80), (16, 128, 128), (17, 144, 272), (33, 624, 664 - 8), (65, 256, 144),
    (127, 112, 400), (130, 272, 304), (255, 1040, 256), (257, 64, 512), (300, 768, 2048), (515, 2064, 176)])
def test_one_expert_without_a_layout(dtype, act, rows, width, N):
    q, s = rows8(rows, width, rows)
    w, ws = bank(1, N, width, N)
    got = M.moe_matmul_i8(q, s, w[0], ws[0], activation=act, dtype=dtype)
    assert got.dtype == dtype and got.shape == (rows, N if act is None else N // 2)
    check(got, q, s, w[0], ws[0], act, dtype)


def routed(T, K, E, seed, skew=0.0, pad=1, itype=torch.int32):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(T, E, generator=g) - skew * torch.arange(E)
    idx = torch.topk(z, K, 1)[1].to(itype).to(DEV)
    return idx, M.moe_layout(idx, E, 1, handle=M.Handle(pad_multiple=pad))


@pytest.mark.parametrize("tokens", [True, False])
@pytest.mark.parametrize("T,K,E,width,N,skew,pad", [
    (1, 1, 1, 16, 16, 0, 1), (1, 8, 128, 256, 96, 0, 1), (4, 2, 8, 1008, 48, 0, 1), (64, 8, 32, 144, 80, 0, 1),
    (33, 3, 5, 624, 160, 1.0, 1), (200, 2, 4, 128, 272, 3.0, 1), (333, 2, 5, 272, 336, 0.5, 16), (700, 4, 16, 96, 144, 0.3, 1),
    (600, 1, 1024, 32, 32, 0, 1), (1100, 8, 64, 64, 128, 0.1, 128), (2000, 1, 3, 80, 64, 0, 1), (130, 7, 9, 512, 256, 2.0, 3)])
def test_every_receive_row(tokens, T, K, E, width, N, skew, pad):
    """Each segment against its expert's weights; empty experts; padding rows; rows past the last as they were."""
    idx, h = routed(T, K, E, T + E, skew, pad)
    q, s = rows8(T, width, T)
    w, ws = bank(E, N, width, E)
    token = h.field("recv_token").cpu().long()
    off = h.field("expert_offset").cpu().tolist()
    qr, sr = q, s
    if not tokens:
        qr = torch.full((h.R, width), 55, dtype=torch.int8, device=DEV)
        sr = torch.full((h.R,), math.nan, device=DEV)
        at = torch.nonzero(token >= 0)[:, 0]
        pads = torch.nonzero(token[:off[-1]] < 0)[:, 0]
        qr[at.to(DEV)], sr[at.to(DEV)] = q[token[at].to(DEV)], s[token[at].to(DEV)]
        qr[pads.to(DEV)], sr[pads.to(DEV)] = 0, 2.0 ** -126
    for act, dtype in ((None, BF16), ("silu", F32), ("gelu_tanh", BF16)):
        out = torch.full((h.R, N if act is None else N // 2), 7.0, dtype=dtype, device=DEV)
        M.moe_matmul_i8(qr, sr, w, ws, handle=h, tokens=tokens, activation=act, out=out)
        assert (out[off[-1]:] == 7).all()
        for e in range(E):
            a, b = off[e], off[e + 1]
            if a == b:
                continue
            mine = token[a:b]
            qe = torch.where((mine >= 0)[:, None], q.cpu()[mine.clamp(min=0)], torch.zeros((), dtype=torch.int8))
            se = torch.where(mine >= 0, s.cpu()[mine.clamp(min=0)], torch.zeros(()))
            check(out[a:b], qe, se, w[e], ws[e], act, dtype, (e, act))


def test_some_of_the_layouts_experts():
    """A partition's own weights: rows of the other experts stay as they were; the parts make up the whole."""
    T, K, E, width, N = 150, 3, 12, 160, 48
    idx, h = routed(T, K, E, 2, 0.2)
    q, s = rows8(T, width, 1)
    w, ws = bank(E, N, width, 1)
    whole = M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True)
    off = h.field("expert_offset").cpu().tolist()
    parts = torch.full_like(whole, 9.0)
    for first, n in ((4, 4), (0, 4), (8, 4)):
        one = torch.full_like(whole, 9.0)
        M.moe_matmul_i8(q, s, w[first:first + n], ws[first:first + n], handle=h, tokens=True, first_expert=first, out=one)
        assert torch.equal(one[off[first]:off[first + n]], whole[off[first]:off[first + n]])
        assert (one[:off[first]] == 9).all() and (one[off[first + n]:] == 9).all()
        M.moe_matmul_i8(q, s, w[first:first + n], ws[first:first + n], handle=h, tokens=True, first_expert=first, out=parts)
    assert torch.equal(parts, whole)


@pytest.mark.parametrize("n", [15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 288, 289, 512, 513])
def test_segments_around_the_sizes_of_tiles(n):
    """One expert of n rows beside small ones, in layouts of few and of many rows an expert."""
    for others in (0, 40):
        idx = torch.cat([torch.full((n,), 1), torch.arange(others) % 40 + 2, torch.tensor([0])]).to(torch.int32).view(-1, 1).to(DEV)
        E = 2 + others
        h = M.moe_layout(idx, E, 1)
        q, s = rows8(len(idx), 192, n)
        w, ws = bank(E, 144, 192, 3)
        out = M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True, activation="silu", dtype=F32)
        check(out[1:1 + n], q[:n], s[:n], w[1], ws[1], "silu", F32)
        check(out[:1], q[-1:], s[-1:], w[0], ws[0], "silu", F32)
        for j in range(others):
            check(out[1 + n + j:2 + n + j], q[n + j:n + j + 1], s[n + j:n + j + 1], w[2 + j], ws[2 + j], "silu", F32)


def test_the_largest_sums():
    """Every product -128 * -128 at the greatest width: 2^31 - 2^18 fits 32 bits."""
    width = 131056
    q = torch.full((3, width), -128, dtype=torch.int8, device=DEV)
    w = torch.full((16, width), -128, dtype=torch.int8, device=DEV)
    w[3] = 127
    y = M.moe_matmul_i8(q, torch.ones(3, device=DEV), w, torch.ones(16, device=DEV), dtype=F32)
    assert (y[:, 0] == 128.0 * 128 * width).all() and (y[:, 3] == torch.tensor(-128.0 * 127 * width).float()).all()


def test_weights_and_rows_past_32_bit_offsets():
    """A bank of 5 GiB, and an output of 2^31 values: the last expert and the last rows."""
    E, N, width = 40, 4096, 32768
    w = torch.zeros(E, N, width, dtype=torch.int8, device=DEV)
    one, ws1 = bank(1, N, width, 1)
    w[E - 1] = one[0]
    ws = torch.ones(E, N, device=DEV)
    ws[E - 1] = ws1[0]
    q, s = rows8(5, width, 2)
    idx = torch.full((5, 1), E - 1, dtype=torch.int32, device=DEV)
    out = M.moe_matmul_i8(q, s, w, ws, handle=M.moe_layout(idx, E, 1), tokens=True)
    check(out, q, s, one[0], ws1[0], None, BF16)
    del w
    rows = (1 << 19) + 3
    q = torch.zeros(rows, 16, dtype=torch.int8, device=DEV)
    s = torch.ones(rows, device=DEV)
    w, ws = bank(1, 4096, 16, 3)
    tail, ts = rows8(4, 16, 4)
    q[-4:], s[-4:] = tail, ts
    out = M.moe_matmul_i8(q, s, w[0], ws[0])
    check(out[-4:], tail, ts, w[0], ws[0], None, BF16)
    assert (out[:-4:4001] == 0).all()


def test_many_wide_rows():
    """2^23 rows that take a workgroup of 512 threads each: more than one dimension of a grid holds."""
    rows, width = (1 << 23) + 5, 1040
    x = torch.zeros(rows, width, device=DEV)
    tail = torch.randn(3, width, generator=torch.Generator().manual_seed(1)).to(DEV)
    at = torch.tensor([0, (1 << 22) + 1, rows - 1], device=DEV)
    x[at] = tail
    q, s = M.moe_quant_rows(x)
    rq, rs = exact_quant(tail)
    assert torch.equal(q[at].cpu(), rq) and torch.equal(s[at].cpu(), rs)
    s[at] = 2.0 ** -126
    assert (s == 2.0 ** -126).all()
    # the most rows at all, several of them a wave
    rows = (1 << 26) - 4
    del x, q, s
    x = torch.zeros(rows, 16, dtype=BF16, device=DEV)
    x[-1] = torch.arange(16)
    q, s = M.moe_quant_rows(x)
    assert torch.equal(q[-1].cpu(), exact_quant(x[-1:])[0][0]) and (q[:-1:100003] == 0).all() and (s[:-1] == 2.0 ** -126).all()


@pytest.mark.parametrize("rows,N", [(6500, 4096), (2700, 1024), (700, 512)])
@pytest.mark.parametrize("width", [16, 128, 144, 256, 272, 384, 400, 512, 640, 752, 768, 896])
def test_many_tiles_of_few_steps(rows, N, width):
    """Every size of tile, one to seven steps each, several tiles a workgroup.

    Sums stay below 2^24 (896 * 127^2 = 14.5e6), so a float32 product has them exactly in any
    order, and float(acc) * scale * w_scale is formed as the kernel forms it: equal in all bits."""
    g = torch.Generator(device=DEV).manual_seed(width)
    q = torch.randint(-127, 128, (rows, width), generator=g, device=DEV, dtype=torch.int8)
    w = torch.randint(-127, 128, (N, width), generator=g, device=DEV, dtype=torch.int8)
    s = torch.rand(rows, generator=g, device=DEV) + 0.5
    ws = torch.rand(N, generator=g, device=DEV) + 0.5
    want = (q.float() @ w.float().T) * s[:, None] * ws
    for _ in range(3):
        out = torch.full((rows, N), math.nan, dtype=torch.float32, device=DEV)
        assert torch.equal(M.moe_matmul_i8(q, s, w, ws, dtype=torch.float32, out=out), want)
    assert torch.equal(M.moe_matmul_i8(q, s, w, ws, dtype=torch.bfloat16), want.to(torch.bfloat16))


def test_results_repeat_and_an_empty_batch():
    idx, h = routed(500, 4, 16, 1)
    q, s = rows8(500, 304, 1)
    w, ws = bank(16, 208, 304, 1)
    ref = M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True, activation="silu")
    for _ in range(5):
        assert torch.equal(M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True, activation="silu"), ref)
    h0 = M.moe_layout(torch.empty(0, 4, dtype=torch.int32, device=DEV), 16, 1)
    q0, s0 = M.moe_quant_rows(torch.empty(0, 304, device=DEV))
    assert M.moe_matmul_i8(q0, s0, w, ws, handle=h0, tokens=True).shape == (0, 208)
    assert M.moe_matmul_i8(q0, s0, w[0], ws[0]).shape == (0, 208)


def test_a_bank_laid_out_and_a_whole_layer():
    """Weights laid out by moe_quant_rows; the layer in 8 bits against itself in float64 on the same integers."""
    T, K, E, H, I = 70, 4, 8, 128, 96
    g = torch.Generator().manual_seed(1)
    x = torch.randn(T, H, generator=g).to(BF16).to(DEV)
    w13 = torch.randn(E, 2 * I, H, generator=g).to(BF16).to(DEV)
    q13, s13 = M.moe_quant_rows(w13)
    rq, rs = exact_quant(w13)
    assert q13.shape == w13.shape and s13.shape == (E, 2 * I) and torch.equal(q13.cpu(), rq) and torch.equal(s13.cpu(), rs)
    idx, h = routed(T, K, E, 4)
    q, s = M.moe_quant_rows(x)
    act = M.moe_matmul_i8(q, s, q13, s13, handle=h, tokens=True, activation="silu")
    token, off = h.field("recv_token").cpu().long(), h.field("expert_offset").cpu().tolist()
    for e in range(E):
        t = token[off[e]:off[e + 1]]
        if len(t):
            check(act[off[e]:off[e + 1]], q.cpu()[t], s.cpu()[t], rq[e], rs[e], "silu", BF16)


def test_refusals():
    idx, h = routed(10, 2, 4, 1)
    q, s = rows8(10, 64, 1)
    w, ws = bank(4, 32, 64, 1)
    for bad in (dict(q=q[:9]), dict(q=q.t()), dict(scale=s[:9]), dict(scale=s.double()), dict(w=w[0]), dict(w=w.float()),
                dict(w_scale=ws[:3]), dict(activation="relu"), dict(out=torch.empty(3, 32, device=DEV)), dict(q=q.cpu())):
        kw = dict(q=q, scale=s, w=w, w_scale=ws, handle=h, tokens=True) | bad
        with pytest.raises((ValueError, M.api.MoeError)):
            M.moe_matmul_i8(**kw)
    with pytest.raises(M.api.MoeError):
        M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True, first_expert=1)
    with pytest.raises(M.api.MoeError):
        M.moe_matmul_i8(q, s, w, ws, handle=h)  # token rows, taken for receive rows
    with pytest.raises(TypeError):
        M.moe_matmul_i8(q, s, w, ws, handle=h, tokens=True, dtype=torch.float16)
    with pytest.raises(RuntimeError):
        M.moe_matmul_i8(q, s, w, ws, handle=M.Handle(), tokens=True)
    with pytest.raises(TypeError):
        M.moe_quant_rows(torch.zeros(2, 32, device=DEV, dtype=torch.float16))
    with pytest.raises(M.api.MoeError):
        M.moe_quant_rows(torch.zeros(2, 40, device=DEV))
