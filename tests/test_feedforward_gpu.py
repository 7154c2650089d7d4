"""The gated feed-forward block and the 8-bit products on the GPU against their formulas in 64 bits."""

import math
import sys

import pytest
import torch

import feedforward_oracle as F
import operator_oracle as O
from allreduce_emulated_peer_amd import mscl as M

pytestmark = pytest.mark.gpu
DTYPES = O.DTYPES
ACTS = sorted(M.ACTIVATION_CODES)


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


def note(*what):
    print("[gpu-case]", *what, file=sys.stderr, flush=True)


def normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def integers(gen, *shape):
    return torch.randint(-128, 128, shape, generator=gen, dtype=torch.int8)


def placed(t, form):
    """t on the GPU: as it is, as a block of columns of a wider matrix, or off 16-byte alignment."""
    if t is None or form == "plain":
        return None if t is None else t.cuda()
    fill = 77 if t.dtype == torch.int8 else math.nan
    if t.dim() == 1:
        room = torch.full((t.shape[0] + 3,), fill, dtype=t.dtype, device="cuda")
        room[1:-2] = t.cuda()
        return room[1:-2]
    pad = {"columns": (16, 16), "odd": (3, 2)}[form]
    room = torch.full((t.shape[0], t.shape[1] + sum(pad)), fill, dtype=t.dtype, device="cuda")
    view = room[:, pad[0]:pad[0] + t.shape[1]]
    view.copy_(t)
    return view


# From one row to several tiles, k from one to many blocks; no size a multiple of what a kernel works in, and some that are.
SIZES = [(1, 1, 1), (1, 256, 128), (2, 40, 3), (5, 1000, 33), (16, 64, 64), (31, 8, 100), (33, 129, 65), (64, 512, 256),
         (65, 72, 136), (100, 2049, 70), (127, 31, 257), (128, 128, 128), (256, 256, 512), (300, 96, 520), (513, 320, 264)]


def gated_case(gen, m, k, n, t, bias=True):
    x = normal(gen, m, k, dtype=t)
    wg, wu = (normal(gen, n, k, scale=max(k, 1) ** -0.5, dtype=t) for _ in range(2))
    bg, bu = (normal(gen, n, scale=0.5, dtype=t) if bias else None for _ in range(2))
    return x, wg, wu, bg, bu


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", ["plain", "columns", "odd"])
def test_gated_linear(dtype, form):
    gen = torch.Generator().manual_seed(51)
    t = DTYPES[dtype]
    for i, (m, k, n) in enumerate(SIZES):
        act = ACTS[i % len(ACTS)]
        args = gated_case(gen, m, k, n, t, bias=i % 3 != 0)
        note("gated linear", dtype, form, m, k, n, act)
        there = [placed(v, form) for v in args]
        got = M.gated_linear_tensors(*there, act, return_preacts=True)
        alone = M.gated_linear_tensors(*there, act)
        for g, want, name in zip(got, F.gated_linear(*args, act), ("y", "gate", "up")):
            F.assert_within(g, want, f"{name} {m}x{k}x{n} {act}")
        assert torch.equal(alone, got[0])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", ["plain", "columns", "odd"])
def test_gated_linear_backward(dtype, form):
    gen = torch.Generator().manual_seed(52)
    t = DTYPES[dtype]
    for i, (m, k, n) in enumerate(SIZES):
        act = ACTS[(i + 2) % len(ACTS)]
        x, wg, wu, _, _ = gated_case(gen, m, k, n, t, bias=False)
        dy, z, v = (normal(gen, m, n, scale=s, dtype=t) for s in (1.0, 1.5, 1.0))
        note("gated linear backward", dtype, form, m, k, n, act)
        args = [placed(a, form) for a in (dy, x, wg, wu, z, v)] + [act]
        got = M.gated_linear_backward_tensors(*args)
        for g, want, name in zip(got, F.gated_linear_backward(dy, x, wg, wu, z, v, act), ("dx", "dwg", "dwu", "dbg", "dbu")):
            F.assert_within(g, want, f"{name} {m}x{k}x{n} {act}")
        for only, at in (("dx", (0,)), ("dw", (1, 2)), ("db", (3, 4))):
            one = M.gated_linear_backward_tensors(*args, **{f"need_{o}": o == only for o in ("dx", "dw", "db")})
            assert [i for i, g in enumerate(one) if g is not None] == list(at)
            assert all(torch.equal(one[i], got[i]) for i in at)


@pytest.mark.parametrize("dtype", DTYPES)
def test_quantize(dtype):
    gen = torch.Generator().manual_seed(53)
    t = DTYPES[dtype]
    for i, (m, k) in enumerate([(1, 1), (3, 16), (5, 17), (1, 1000), (70, 1024), (9, 2049), (33, 4096), (600, 130),
                                (520, 1030), (515, 4097), (513, 8200), (4, 8200), (2, 16400), (514, 16385), (3, 33000)]):
        x = normal(gen, m, k, dtype=t)
        x[0] = 0
        if m > 1 and dtype != "fp16":
            x[1] *= 2.0 ** -110  # below the least size
        for form in ("plain", "columns", "odd"):
            note("quantize", dtype, m, k, form)
            q, scale = M.quantize_tensors(placed(x, form))
            want_q, want_scale = F.quantize(x)
            assert torch.equal(q.cpu(), want_q) and torch.equal(scale.cpu(), want_scale), (m, k, form)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", ["plain", "columns", "odd"])
def test_linear_quantized(dtype, form):
    gen = torch.Generator().manual_seed(54)
    t = DTYPES[dtype]
    for i, (m, k, n) in enumerate(SIZES):
        act = ACTS[(i + 1) % len(ACTS)]
        x, w = integers(gen, m, k), integers(gen, n, k)
        sx, sw = torch.rand(m, generator=gen) * 0.02 + 1e-3, torch.rand(n, generator=gen) * 0.02 / k ** 0.5 + 1e-5
        b = normal(gen, n, scale=0.5, dtype=t) if i % 3 else None
        r = normal(gen, m, n, dtype=t) if i % 4 else None
        note("linear int8", dtype, form, m, k, n, act)
        y = M.linear_quantized_tensors(placed(x, form), sx.cuda(), placed(w, form), sw.cuda(), placed(b, form), placed(r, form),
                                  act, dtype=t)
        F.assert_within(y, F.linear_quantized(x, sx, w, sw, b, r, act, t), f"y {m}x{k}x{n} {act}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", ["plain", "columns", "odd"])
def test_gated_linear_quantized(dtype, form):
    gen = torch.Generator().manual_seed(55)
    t = DTYPES[dtype]
    for i, (m, k, n) in enumerate(SIZES):
        act = ACTS[(i + 3) % len(ACTS)]
        x, wg, wu = integers(gen, m, k), integers(gen, n, k), integers(gen, n, k)
        sx = torch.rand(m, generator=gen) * 0.02 + 1e-3
        sg, su = (torch.rand(n, generator=gen) * 0.02 / k ** 0.5 + 1e-5 for _ in range(2))
        bg, bu = (normal(gen, n, scale=0.5, dtype=t) if i % 3 else None for _ in range(2))
        note("gated linear int8", dtype, form, m, k, n, act)
        y = M.gated_linear_quantized_tensors(placed(x, form), sx.cuda(), placed(wg, form), sg.cuda(), placed(wu, form), su.cuda(),
                                        placed(bg, form), placed(bu, form), act, dtype=t)
        F.assert_within(y, F.gated_linear_quantized(x, sx, wg, sg, wu, su, bg, bu, act, t), f"y {m}x{k}x{n} {act}")


# Large products (256 x 256 tiles): edges inside a tile, k that ends inside a block, odd and even numbers of blocks, and
# operands that have to be laid out anew.
LARGE = [(2304, 1024, 2048, "plain"), (2100, 1040, 2000, "plain"), (2100, 1040, 2000, "columns"), (2300, 1027, 1955, "odd"),
         (4097, 576, 1040, "plain"), (1030, 4100, 3960, "odd")]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n,form", LARGE)
def test_large_gated_products(dtype, m, k, n, form):
    gen = torch.Generator().manual_seed(56)
    t = DTYPES[dtype]
    args = gated_case(gen, m, k, n, t)
    there, c = [placed(v, form) for v in args], [v.cuda() for v in args]  # the oracle's 64 bits on the GPU
    note("large gated linear", dtype, m, k, n, form)
    got = M.gated_linear_tensors(*there, "silu", return_preacts=True)
    for g, want, name in zip(got, F.gated_linear(*c, "silu"), ("y", "gate", "up")):
        F.assert_within(g, want, name)
    assert torch.equal(M.gated_linear_tensors(*there, "silu"), got[0])


# k and n large enough that the input gradient, the weights' gradients or both run by large tiles
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n,form", [(2304, 4096, 512, "plain"), (300, 4096, 2304, "plain"), (2100, 4000, 2056, "columns"),
                                        (2300, 4099, 1955, "odd"), (2200, 4104, 200, "plain")])
def test_large_gated_gradients(dtype, m, k, n, form):
    gen = torch.Generator().manual_seed(57)
    t = DTYPES[dtype]
    x, wg, wu, _, _ = gated_case(gen, m, k, n, t, bias=False)
    dy, z, v = (normal(gen, m, n, scale=s, dtype=t) for s in (1.0, 1.5, 1.0))
    args = (dy, x, wg, wu, z, v)
    there, c = [placed(a, form) for a in args], [a.cuda() for a in args]
    note("large gated gradients", dtype, m, k, n, form)
    got = M.gated_linear_backward_tensors(*there, "gelu")
    for g, want, name in zip(got, F.gated_linear_backward(*c, "gelu"), ("dx", "dwg", "dwu", "dbg", "dbu")):
        F.assert_within(g, want, name)
    for a, b in zip(got, M.gated_linear_backward_tensors(*there, "gelu")):
        assert torch.equal(a, b)


def test_large_binary32_products_with_infinities_nan_and_far_values():
    """What the bfloat16 parts of a value cannot hold: the tiles with such sums are summed again in binary32."""
    gen = torch.Generator().manual_seed(59)
    m, k, n = 2100, 4100, 1030
    x, wg, wu, _, _ = gated_case(gen, m, k, n, torch.float32, bias=False)
    x[5, 3], x[7, k - 1], wu[11, 40] = math.inf, math.nan, -math.inf
    x[9] *= 2.0 ** 108
    x[300:, 40] = x[300:, 40].abs() + 1
    x[:300, 40] = -x[:300, 40].abs() - 1
    note("large binary32 product with infinities")
    y, gate, up = M.gated_linear_tensors(x.cuda(), wg.cuda(), wu.cuda(), activation="none", return_preacts=True)
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[[5, 7]] = True
    assert not bool(torch.isfinite(gate.cpu()[bad]).any()) and bool(torch.isnan(gate[7]).all())
    assert torch.equal(up[300:, 11].cpu(), torch.full((m - 300,), -math.inf))
    ok = [i for i in range(m) if i not in (5, 7)]
    cols = [i for i in range(n) if i != 11]
    c = x[ok].cuda(), wg[cols].cuda(), wu[cols].cuda()
    _, want_gate, want_up = F.gated_linear(*c, None, None, "none")
    F.assert_within(gate[ok][:, cols], want_gate, "gate")
    F.assert_within(up[ok][:, cols], want_up, "up")

    note("large binary32 gradients with infinities")
    dy, z, v = (normal(gen, m, n, scale=s) for s in (1.0, 1.5, 1.0))
    dy[5, 3], dy[7, 12] = math.inf, math.nan
    dy[9] *= 2.0 ** 108
    x, wg, wu, _, _ = gated_case(gen, m, k, n, torch.float32, bias=False)
    got = M.gated_linear_backward_tensors(*[t.cuda() for t in (dy, x, wg, wu, z, v)], "none")
    assert not bool(torch.isfinite(got[0][[5, 7]]).any()) and not bool(torch.isfinite(got[1][[3, 12]]).any())
    c = [t.cuda() for t in (dy[ok], x, wg, wu, z[ok], v[ok])]
    F.assert_within(got[0][ok], F.gated_linear_backward(c[0], x[ok].cuda(), *c[2:], "none")[0], "dx")
    cols = [i for i in range(n) if i not in (3, 12)]
    c = [t.cuda() for t in (dy[:, cols], x, wg[cols], wu[cols], z[:, cols], v[:, cols])]
    for g, want, name in zip(got[1:], F.gated_linear_backward(*c, "none")[1:], ("dwg", "dwu", "dbg", "dbu")):
        F.assert_within(g[cols], want, name)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("m,k,n,form", [(2304, 2048, 4096, "plain"), (2100, 2064, 4000, "plain"), (2100, 2064, 4000, "columns"),
                                        (2300, 2051, 3907, "odd"), (4097, 1152, 2056, "plain")])
def test_large_int8_products(dtype, m, k, n, form):
    gen = torch.Generator().manual_seed(58)
    t = DTYPES[dtype]
    x, w, v = integers(gen, m, k), integers(gen, n, k), integers(gen, n, k)
    sx = torch.rand(m, generator=gen) * 0.02 + 1e-3
    sw, sv = (torch.rand(n, generator=gen) * 0.02 / k ** 0.5 + 1e-5 for _ in range(2))
    b, r = normal(gen, n, scale=0.5, dtype=t), normal(gen, m, n, dtype=t)
    c = [a.cuda() for a in (x, sx, w, sw, v, sv, b, r)]
    xg, wg, vg, bg, rg = (placed(a, form) for a in (x, w, v, b, r))
    note("large int8 product", dtype, m, k, n, form)
    y = M.linear_quantized_tensors(xg, c[1], wg, c[3], bg, rg, "gelu", dtype=t)
    F.assert_within(y, F.linear_quantized(*c[:4], c[6], c[7], "gelu", t), "y")
    note("large gated int8 product", dtype, m, k, n, form)
    y = M.gated_linear_quantized_tensors(xg, c[1], wg, c[3], vg, c[5], bg, None, "silu", dtype=t)
    F.assert_within(y, F.gated_linear_quantized(*c[:6], c[6], None, "silu", t), "gated y")


def test_int8_sums_are_exact_to_their_largest():
    """The largest sums that are allowed, of both signs, with scales of powers of two: nothing rounds but the sum."""
    k = 131071
    x, w = torch.full((3, k), -128, dtype=torch.int8), torch.full((5, k), -128, dtype=torch.int8)
    x[1] = 127
    x[2, ::2] = 127
    w[4, 1:] = 0
    note("largest integer sums")
    sx, sw = torch.tensor([1.0, 0.5, 4.0]), torch.tensor([1.0, 2.0, 0.25, 8.0, 1.0])
    y = M.linear_quantized_tensors(x.cuda(), sx.cuda(), w.cuda(), sw.cuda(), dtype=torch.float32).cpu()
    want = (x.double() @ w.double().t()).float() * sx[:, None] * sw
    assert torch.equal(y, want)
    with pytest.raises(M.MsclError, match="131071"):
        M.linear_quantized_tensors(torch.zeros(1, k + 1, dtype=torch.int8, device="cuda"), sx[:1].cuda(),
                              torch.zeros(1, k + 1, dtype=torch.int8, device="cuda"), sw[:1].cuda())
