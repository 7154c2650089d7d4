"""The gated feed-forward block and the 8-bit products on the GPU at the edges of what a call may be."""

import math
import os
import subprocess
import sys

import pytest
import torch

import feedforward_oracle as F
import operator_oracle as O
from allreduce_emulated_peer_amd import mscl as M
from test_feedforward_gpu import ACTS, DTYPES, gated_case, integers, normal, note, placed

pytestmark = pytest.mark.gpu
CODES = {torch.float32: M.FLOAT32, torch.float16: M.FLOAT16, torch.bfloat16: M.BFLOAT16}


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


def scales(gen, n, size=0.02):
    return torch.rand(n, generator=gen) * size + size / 20


def within(got, want, names):
    for g, w, name in zip(got, want, names):
        F.assert_within(g, w, name)


BACK = ("dx", "dwg", "dwu", "dbg", "dbu")


# ---------------------------------------------------------------- shapes

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n,form", [(1, 8200, 70, "plain"), (3, 4100, 200, "odd"), (9, 12289, 33, "columns"),
                                        (17, 8192, 48, "plain"), (32, 5003, 130, "odd"), (12, 640, 8300, "plain"),
                                        (32, 100, 8200, "columns"), (2, 15, 40, "odd"), (20, 131, 5, "odd")])
def test_few_rows(dtype, m, k, n, form):
    """Up to 32 rows: k split over workgroups and waves, ends of k inside a step, one and two tiles of rows."""
    gen = torch.Generator().manual_seed(71)
    t = DTYPES[dtype]
    args = gated_case(gen, m, k, n, t)
    note("few rows, gated", dtype, m, k, n, form)
    got = M.gated_linear_tensors(*[placed(a, form) for a in args], "gelu_tanh", return_preacts=True)
    within(got, F.gated_linear(*args, "gelu_tanh"), ("y", "gate", "up"))
    x, w, v = integers(gen, m, k), integers(gen, n, k), integers(gen, n, k)
    sx, sw, sv = scales(gen, m), scales(gen, n, 0.02 / k ** 0.5), scales(gen, n, 0.02 / k ** 0.5)
    b, r = normal(gen, n, dtype=t), normal(gen, m, n, dtype=t)
    xg, wg, vg, bg, rg = (placed(a, form) for a in (x, w, v, b, r))
    note("few rows, 8 bits", dtype, m, k, n, form)
    y = M.linear_quantized_tensors(xg, sx.cuda(), wg, sw.cuda(), bg, rg, "silu", dtype=t)
    F.assert_within(y, F.linear_quantized(x, sx, w, sw, b, r, "silu", t), "8-bit y")
    y = M.gated_linear_quantized_tensors(xg, sx.cuda(), wg, sw.cuda(), vg, sv.cuda(), bg, None, "gelu", dtype=t)
    F.assert_within(y, F.gated_linear_quantized(x, sx, w, sw, v, sv, b, None, "gelu", t), "gated 8-bit y")


# rows x outputs that few tiles cover and k that is long: shares of k
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n,form", [(40, 6001, 50, "odd"), (130, 4096, 70, "plain"), (70, 3000, 200, "columns")])
def test_few_tiles_of_long_sums(dtype, m, k, n, form):
    gen = torch.Generator().manual_seed(72)
    t = DTYPES[dtype]
    args = gated_case(gen, m, k, n, t)
    note("long sums, gated", dtype, m, k, n, form)
    got = M.gated_linear_tensors(*[placed(a, form) for a in args], "silu", return_preacts=True)
    within(got, F.gated_linear(*args, "silu"), ("y", "gate", "up"))
    x, w, v = integers(gen, m, k), integers(gen, n, k), integers(gen, n, k)
    sx, sw, sv = scales(gen, m), scales(gen, n, 0.02 / k ** 0.5), scales(gen, n, 0.02 / k ** 0.5)
    xg, wg, vg = (placed(a, form) for a in (x, w, v))
    note("long sums, 8 bits", dtype, m, k, n, form)
    y = M.linear_quantized_tensors(xg, sx.cuda(), wg, sw.cuda(), dtype=t)
    F.assert_within(y, F.linear_quantized(x, sx, w, sw, None, None, "none", t), "8-bit y")
    y = M.gated_linear_quantized_tensors(xg, sx.cuda(), wg, sw.cuda(), vg, sv.cuda(), dtype=t)
    F.assert_within(y, F.gated_linear_quantized(x, sx, w, sw, v, sv, None, None, "silu", t), "gated 8-bit y")
    # the backward pass's long sums are over rows (weights) and over outputs (input)
    for rows, k2, n2 in ((6001, 40, 50), (60, 70, 5000)):
        x, wg, wu, _, _ = gated_case(gen, rows, k2, n2, t, bias=False)
        dy, z, u = (normal(gen, rows, n2, dtype=t) for _ in range(3))
        note("long sums, gated backward", dtype, rows, k2, n2, form)
        got = M.gated_linear_backward_tensors(*[placed(a, form) for a in (dy, x, wg, wu, z, u)])
        within(got, F.gated_linear_backward(dy, x, wg, wu, z, u, "silu"), BACK)


def test_leading_dimensions():
    gen = torch.Generator().manual_seed(73)
    x, wg, wu, bg, bu = gated_case(gen, 30, 24, 40, torch.bfloat16)
    dy = normal(gen, 30, 40, dtype=torch.bfloat16)
    c = [t.cuda() for t in (wg, wu, bg, bu)]
    note("leading dimensions")
    y, gate, up = M.gated_linear_tensors(x.view(2, 3, 5, 24).cuda(), *c, return_preacts=True)
    assert y.shape == gate.shape == up.shape == (2, 3, 5, 40)
    within([t.view(30, 40) for t in (y, gate, up)], F.gated_linear(x, wg, wu, bg, bu, "silu"), ("y", "gate", "up"))
    got = M.gated_linear_backward_tensors(dy.view(2, 3, 5, 40).cuda(), x.view(2, 3, 5, 24).cuda(), c[0], c[1], gate, up)
    assert [g.shape for g in got] == [(2, 3, 5, 24), (40, 24), (40, 24), (40,), (40,)]
    want = F.gated_linear_backward(dy, x, wg, wu, gate.view(30, 40).cpu(), up.view(30, 40).cpu(), "silu")
    within([got[0].view(30, 24), *got[1:]], want, BACK)
    one = M.gated_linear_tensors(x[0].cuda(), *c)
    assert one.shape == (40,)
    q, scale = M.quantize_tensors(x.view(2, 3, 5, 24).cuda())
    assert q.shape == (2, 3, 5, 24) and scale.shape == (2, 3, 5)
    flat, flat_scale = M.quantize_tensors(x[0].cuda())
    assert flat.shape == (24,) and flat_scale.shape == () and torch.equal(flat, q[0, 0, 0]) and flat_scale == scale[0, 0, 0]
    (qg, sg), (qu, su) = M.quantize_tensors(c[0]), M.quantize_tensors(c[1])
    r = dy.view(2, 3, 5, 40).cuda()
    y = M.linear_quantized_tensors(q, scale, qg, sg, c[2], r)
    z = M.gated_linear_quantized_tensors(q, scale, qg, sg, qu, su)
    assert y.shape == z.shape == (2, 3, 5, 40)
    assert torch.equal(M.linear_quantized_tensors(flat, flat_scale, qg, sg, c[2], r[0, 0, 0]), y[0, 0, 0])
    assert torch.equal(M.gated_linear_quantized_tensors(flat, flat_scale, qg, sg, qu, su), z[0, 0, 0])


@pytest.mark.parametrize("dtype", DTYPES)
def test_empty_sizes(dtype):
    t = DTYPES[dtype]
    e = lambda *s: torch.ones(s, dtype=t, device="cuda")  # noqa: E731
    i = lambda *s: torch.ones(s, dtype=torch.int8, device="cuda")  # noqa: E731
    f = lambda *s: torch.ones(s, device="cuda")  # noqa: E731
    note("empty sizes", dtype)
    assert M.gated_linear_tensors(e(0, 5), e(7, 5), e(7, 5)).shape == (0, 7)
    assert M.gated_linear_tensors(e(4, 5), e(0, 5), e(0, 5)).shape == (4, 0)
    y, g, u = M.gated_linear_tensors(e(4, 0), e(7, 0), e(7, 0), e(7), e(7) * 3, "relu", return_preacts=True)
    assert bool((y == 3).all()) and bool((g == 1).all()) and bool((u == 3).all())
    dx, dg, du, bg, bu = M.gated_linear_backward_tensors(e(0, 7), e(0, 5), e(7, 5), e(7, 5), e(0, 7), e(0, 7))
    assert dx.shape == (0, 5) and dg.shape == (7, 5) and not any(v.any() for v in (dg, du, bg, bu))
    dx, dg, du, bg, bu = M.gated_linear_backward_tensors(e(4, 0), e(4, 5), e(0, 5), e(0, 5), e(4, 0), e(4, 0))
    assert dx.shape == (4, 5) and not dx.any() and dg.shape == (0, 5) and bg.shape == (0,)
    dx, dg, du, bg, bu = M.gated_linear_backward_tensors(e(4, 7), e(4, 0), e(7, 0), e(7, 0), e(4, 7), e(4, 7) * 2, "none")
    assert dx.shape == (4, 0) and dg.shape == (7, 0) and bool((bg == 8).all()) and bool((bu == 4).all())
    q, s = M.quantize_tensors(e(0, 5))
    assert q.shape == (0, 5) and s.shape == (0,)
    assert M.linear_quantized_tensors(i(0, 5), f(0), i(7, 5), f(7), dtype=t).shape == (0, 7)
    assert M.linear_quantized_tensors(i(4, 5), f(4), i(0, 5), f(0), dtype=t).shape == (4, 0)
    y = M.linear_quantized_tensors(i(4, 0), f(4), i(7, 0), f(7), e(7), e(4, 7), "relu", dtype=t)
    assert bool((y == 2).all())
    assert M.gated_linear_quantized_tensors(i(0, 5), f(0), i(7, 5), f(7), i(7, 5), f(7), dtype=t).shape == (0, 7)
    y = M.gated_linear_quantized_tensors(i(4, 0), f(4), i(7, 0), f(7), i(7, 0), f(7), e(7), e(7) * 3, "none", dtype=t)
    assert bool((y == 3).all())


# ---------------------------------------------------------------- values

@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(dtype, act):
    """Products with the identity: every value of the activation and its slope, times an even second factor."""
    t = DTYPES[dtype]
    z = torch.cat([torch.linspace(-14, 14, 4000), torch.linspace(-0.01, 0.01, 96)]).to(t).reshape(64, 64)
    eye, twice = torch.eye(64, dtype=t), 2 * torch.eye(64, dtype=t)
    note("gated activation", dtype, act)
    y = M.gated_linear_tensors(z.cuda(), eye.cuda(), twice.cuda(), activation=act)
    F.assert_within(y, F.gated_linear(z, eye, twice, None, None, act)[0], act)
    ones = torch.ones(64, 64, dtype=t)
    got = M.gated_linear_backward_tensors(*[v.cuda() for v in (ones, eye, eye, eye, z, 2 * ones)], act)
    within(got, F.gated_linear_backward(ones, eye, eye, eye, z, 2 * ones, act), BACK)


def test_nan_and_infinity_stay_in_their_rows_and_columns():
    gen = torch.Generator().manual_seed(74)
    for m, k, n in ((20, 70, 50), (40, 70, 50), (300, 320, 512), (2100, 712, 2050)):
        for t in (torch.bfloat16, torch.float32):
            x, wg, wu, bg, bu = gated_case(gen, m, k, n, t)
            x[3, 5], x[7, k - 1], wg[11, 0], wu[13, 1] = math.nan, math.inf, math.nan, -math.inf
            note("gated with NaN and infinity", m, k, n, t)
            y, gate, up = (v.cpu() for v in M.gated_linear_tensors(*[v.cuda() for v in (x, wg, wu, bg, bu)], "none",
                                                                  return_preacts=True))
            bad = torch.zeros(m, n, dtype=torch.bool)
            bad[3], bad[7], bad[:, 11], bad[:, 13] = True, True, True, True
            assert bool(torch.isfinite(y[~bad]).all()) and not bool(torch.isfinite(y[bad]).any())
            assert bool(torch.isnan(gate[:, 11]).all()) and not bool(torch.isfinite(up[:, 13]).any())
            rows = [i for i in range(m) if i not in (3, 7)]
            assert bool(torch.isfinite(gate[rows][:, 13]).all()) and bool(torch.isfinite(up[rows][:, 11]).all())
    for t in DTYPES.values():
        # an activation at -infinity is 0, which an infinite second factor makes NaN, as in the formula
        one = torch.zeros(1, 8, dtype=t, device="cuda")
        w = torch.zeros(3, 8, dtype=t, device="cuda")
        bg = torch.tensor([-math.inf, -math.inf, math.inf], dtype=t, device="cuda")
        bu = torch.tensor([2.0, math.inf, -3.0], dtype=t, device="cuda")
        for act in ("relu", "gelu", "gelu_tanh", "silu"):
            y = M.gated_linear_tensors(one, w, w, bg, bu, act)[0].cpu()
            assert y[0] == 0 and bool(torch.isnan(y[1])) and y[2] == -math.inf


def test_gradients_keep_nan_and_infinity_in_their_rows_and_columns():
    gen = torch.Generator().manual_seed(75)
    for m, k, n, t in ((40, 70, 50, torch.bfloat16), (300, 320, 512, torch.float32), (2100, 4100, 264, torch.bfloat16)):
        x, wg, wu, _, _ = gated_case(gen, m, k, n, t, bias=False)
        dy, z, v = (normal(gen, m, n, dtype=t) for _ in range(3))
        dy[3, 5], z[7, 9], v[11, 2] = math.nan, math.nan, math.nan
        note("gated gradients with NaN", m, k, n, t)
        dx, dwg, dwu, dbg, dbu = (g.cpu() for g in M.gated_linear_backward_tensors(*[a.cuda() for a in (dy, x, wg, wu, z, v)]))
        for g, rows in ((dx, (3, 7, 11)), (dwg, (5, 9, 2)), (dwu, (5, 9))):
            keep = [i for i in range(g.shape[0]) if i not in rows]
            assert bool(torch.isnan(g[list(rows)]).all()) and bool(torch.isfinite(g[keep]).all())
        assert torch.isnan(dbg).nonzero()[:, 0].tolist() == [2, 5, 9] and torch.isnan(dbu).nonzero()[:, 0].tolist() == [5, 9]


def test_rows_that_have_no_scale():
    """A row with an infinity or NaN is marked by its scale and makes its products NaN; rows of zeros are zeros."""
    gen = torch.Generator().manual_seed(76)
    for t in DTYPES.values():
        for k in (40, 1000, 5000, 33000):
            x = normal(gen, 6, k, dtype=t)
            x[1, k - 1], x[2, 0], x[3, 7], x[4] = math.nan, math.inf, -math.inf, 0
            x[5, 3] = torch.finfo(t).max
            note("rows without a scale", t, k)
            q, scale = M.quantize_tensors(x.cuda())
            assert torch.isnan(scale).tolist() == [False, True, True, True, False, False] and not bool(q[1:5].any())
            want_q, want_scale = F.quantize(x[[0, 4, 5]])
            assert torch.equal(q[[0, 4, 5]].cpu(), want_q) and torch.equal(scale[[0, 4, 5]].cpu(), want_scale)
            w, sw = integers(gen, 7, k).cuda(), scales(gen, 7).cuda()
            y = M.linear_quantized_tensors(q, scale, w, sw, dtype=torch.float32)
            z = M.gated_linear_quantized_tensors(q, scale, w, sw, w, sw, activation="none", dtype=torch.float32)
            for out in (y, z):
                assert bool(torch.isnan(out[1:4]).all()) and not bool(out[4].any()) and not bool(torch.isnan(out[[0, 5]]).any())


def test_more_rows_than_a_launch_takes():
    rows, width = 2 ** 21 + 5, 9
    note("many rows", rows, width)
    x = torch.randn(rows, width, generator=torch.Generator(device="cuda").manual_seed(86), device="cuda").bfloat16()
    q, scale = M.quantize_tensors(x)
    for part in (slice(0, 3000), slice(2 ** 21 - 3000, None)):
        want, want_scale = F.quantize(x[part].cpu())
        assert torch.equal(q[part].cpu(), want) and torch.equal(scale[part].cpu(), want_scale)
    values = q.float() * scale[:, None]
    assert bool(((values - x.float()).abs() <= 0.5001 * scale[:, None]).all())


@pytest.mark.parametrize("dtype", DTYPES)
def test_ties_go_to_the_even_integer(dtype):
    """Sizes of 127 times a power of two, so that halves of a step are exact."""
    t = DTYPES[dtype]
    halves = (torch.arange(-126, 127) + 0.5)[:254]
    x = torch.cat([torch.tensor([127.0]), halves]).to(t)
    rows = torch.stack([x * 2.0 ** p for p in (-6, -1, 0, 3)])
    note("ties", dtype)
    q, scale = M.quantize_tensors(rows.cuda())
    want, want_scale = F.quantize(rows)
    assert torch.equal(q.cpu(), want) and torch.equal(scale.cpu(), want_scale)
    exact = halves.to(t).double()
    if bool((exact == halves.double()).all()):
        assert bool((want[:, 1:] % 2 == 0).all())


def test_gradients_against_differences():
    gen = torch.Generator().manual_seed(77)
    m, k, n = 70, 90, 130
    for act in ACTS:
        x, wg, wu, bg, bu = gated_case(gen, m, k, n, torch.float32)
        dy = normal(gen, m, n)
        note("gated differences", act)
        c = [t.cuda() for t in (x, wg, wu, bg, bu)]
        _, z, v = M.gated_linear_tensors(*c, act, return_preacts=True)
        if act == "relu":  # away from the corner, which a difference would step over
            dy = dy * (z.cpu().abs() > 1e-2)
        grads = M.gated_linear_backward_tensors(dy.cuda(), *c[:3], z, v, act)

        def loss(p):
            return float((O.activate(p[0] @ p[1].t() + p[3], act) * (p[0] @ p[2].t() + p[4]) * dy.double()).sum())

        at = [t.double() for t in (x, wg, wu, bg, bu)]
        for i, g in enumerate(grads):
            d = torch.randn(at[i].shape, generator=gen, dtype=torch.float64)
            h = 1e-5
            hi, lo = list(at), list(at)
            hi[i], lo[i] = at[i] + h * d, at[i] - h * d
            slope = (loss(hi) - loss(lo)) / (2 * h)
            # each gradient value is off by a few 2^-20 of its terms at most, so is their sum along d of that size;
            # the difference's own error is h^2 times the third derivative
            size = float((g.cpu().double() * d).abs().sum())
            assert abs(slope - float((g.cpu().double() * d).sum())) < 4e-6 * size + 1e-4, (act, i)


# ---------------------------------------------------------------- where things lie

def guarded(t, rows=256):
    """t on the GPU with `rows` rows of NaN (or of a value that counts) behind its last one."""
    fill = 77 if t.dtype == torch.int8 else math.nan
    room = torch.full((t.shape[0] + rows, t.shape[1]), fill, dtype=t.dtype, device="cuda")
    room[:t.shape[0]] = t.cuda()
    return room[:t.shape[0]]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n", [(50, 72, 40), (193, 4096, 2056), (2100, 4096, 200), (2052, 328, 1932), (321, 4104, 2184)])
def test_what_lies_behind_the_matrices_reaches_no_result(dtype, m, k, n):
    gen = torch.Generator().manual_seed(78)
    t = DTYPES[dtype]
    x, wg, wu, _, _ = gated_case(gen, m, k, n, t, bias=False)
    dy, z, v = (normal(gen, m, n, scale=s, dtype=t) for s in (1.0, 1.5, 1.0))
    c = [a.cuda() for a in (dy, x, wg, wu, z, v)]
    note("guarded gated", dtype, m, k, n)
    got = M.gated_linear_tensors(*[guarded(a) for a in (x, wg, wu)], return_preacts=True)
    within(got, F.gated_linear(c[1], c[2], c[3], None, None, "silu"), ("y", "gate", "up"))
    note("guarded gated backward", dtype, m, k, n)
    got = M.gated_linear_backward_tensors(*[guarded(a) for a in (dy, x, wg, wu, z, v)])
    within(got, F.gated_linear_backward(*c, "silu"), BACK)
    qx, qw = integers(gen, m, k), integers(gen, n, k)
    sx, sw = scales(gen, m).cuda(), scales(gen, n, 0.02 / k ** 0.5).cuda()
    note("guarded 8 bits", dtype, m, k, n)
    y = M.linear_quantized_tensors(guarded(qx), sx, guarded(qw), sw, dtype=t)
    F.assert_within(y, F.linear_quantized(qx.cuda(), sx, qw.cuda(), sw, None, None, "none", t), "8-bit y")


@pytest.mark.parametrize("m,k,n,t", [(33, 80, 50, torch.bfloat16), (300, 256, 260, torch.float16), (70, 30, 45, torch.float32),
                                     (2100, 264, 2056, torch.bfloat16)])
def test_outputs_as_columns_of_wider_matrices(m, k, n, t):
    """Through the C ABI: what lies beside the outputs stays as it is; the weights are halves of one matrix."""
    gen = torch.Generator().manual_seed(79)
    lib, code, e = M.load(), CODES[t], t.itemsize
    x, wg, wu, bg, bu = gated_case(gen, m, k, n, t)
    w = torch.cat([wg, wu]).cuda()
    xg, bgg, bug = x.cuda(), bg.cuda(), bu.cuda()
    wide = n + 7
    room = [torch.full((m, wide), 77.0, dtype=t, device="cuda") for _ in range(3)]
    stream = torch.cuda.current_stream().cuda_stream
    call = M.GATED_LINEAR.pack(xg.data_ptr(), k, w.data_ptr(), k, w.data_ptr() + n * k * e, k, bgg.data_ptr(), bug.data_ptr(),
                               *[a for r in room for a in (r.data_ptr() + 3 * e, wide)], m, k, n, code, M.ACT_GELU)
    note("strided outputs, gated", m, k, n, t)
    space, size = M._workspace(lib.mscl_gated_linear_workspace, call, xg)
    M._check(lib.mscl_gated_linear(call, M._address(space), size, stream), "gated")
    want = F.gated_linear(*[v.cuda() for v in (x, wg, wu, bg, bu)], "gelu")
    for r, e_, name in zip(room, want, ("y", "gate", "up")):
        F.assert_within(r[:, 3:3 + n], e_, name)
        assert bool((r[:, :3] == 77).all()) and bool((r[:, 3 + n:] == 77).all())
    # both weights' gradients as halves of one matrix, dx inside a wider one
    dy, z, v = (normal(gen, m, n, dtype=t).cuda() for _ in range(3))
    dw = torch.full((2 * n + 1, k + 5), 55.0, dtype=t, device="cuda")
    dx = torch.full((m, k + 5), 55.0, dtype=t, device="cuda")
    db = torch.empty(2, n, dtype=t, device="cuda")
    call = M.GATED_LINEAR_BACKWARD.pack(
        dy.data_ptr(), n, xg.data_ptr(), k, w.data_ptr(), k, w.data_ptr() + n * k * e, k, z.data_ptr(), n, v.data_ptr(), n,
        dx.data_ptr() + 2 * e, k + 5, dw.data_ptr() + e, k + 5, dw.data_ptr() + (n * (k + 5) + 1) * e, k + 5, db[0].data_ptr(),
        db[1].data_ptr(), m, k, n, code, M.ACT_GELU)
    note("strided outputs, gated backward", m, k, n, t)
    space, size = M._workspace(lib.mscl_gated_linear_backward_workspace, call, xg)
    M._check(lib.mscl_gated_linear_backward(call, M._address(space), size, stream), "gated backward")
    want = F.gated_linear_backward(dy, xg, wg.cuda(), wu.cuda(), z, v, "gelu")
    within((dx[:, 2:2 + k], dw[:n, 1:1 + k], dw[n:2 * n, 1:1 + k], db[0], db[1]), want, BACK)
    assert bool((dx[:, :2] == 55).all()) and bool((dx[:, 2 + k:] == 55).all())
    assert bool((dw[:, :1] == 55).all()) and bool((dw[:, 1 + k:] == 55).all()) and bool((dw[2 * n] == 55).all())
    # one weight's gradient alone has the same bits
    one = torch.empty(n, k, dtype=t, device="cuda")
    for of_gate in (True, False):
        call = M.GATED_LINEAR_BACKWARD.pack(
            dy.data_ptr(), n, xg.data_ptr(), k, 0, 0, 0, 0, z.data_ptr(), n, v.data_ptr(), n, 0, 0,
            one.data_ptr() if of_gate else 0, k, 0 if of_gate else one.data_ptr(), k, 0, 0, m, k, n, code, M.ACT_GELU)
        space, size = M._workspace(lib.mscl_gated_linear_backward_workspace, call, xg)
        M._check(lib.mscl_gated_linear_backward(call, M._address(space), size, stream), "gated backward")
        assert torch.equal(one, dw[:n, 1:1 + k] if of_gate else dw[n:2 * n, 1:1 + k])
    # 8 bits: integers into a wider matrix, y over the residual
    q = torch.full((m, k + 9), 99, dtype=torch.int8, device="cuda")
    scale = torch.empty(m, device="cuda")
    call = M.QUANTIZE.pack(xg.data_ptr(), k, q.data_ptr() + 3, k + 9, scale.data_ptr(), m, k, code)
    note("strided outputs, 8 bits", m, k, n, t)
    M._check(lib.mscl_quantize(call, stream), "quantize")
    want_q, want_scale = F.quantize(x)
    assert torch.equal(q[:, 3:3 + k].cpu(), want_q) and torch.equal(scale.cpu(), want_scale)
    assert bool((q[:, :3] == 99).all()) and bool((q[:, 3 + k:] == 99).all())
    qw, sw = M.quantize_tensors(wg.cuda())
    r = normal(gen, m, n, dtype=t)
    y = torch.full((m, wide), 77.0, dtype=t, device="cuda")
    y[:, 3:3 + n] = r.cuda()
    at = y.data_ptr() + 3 * e
    call = M.LINEAR_QUANTIZED.pack(q.data_ptr() + 3, k + 9, scale.data_ptr(), qw.data_ptr(), k, sw.data_ptr(), bgg.data_ptr(), at,
                                   wide, at, wide, m, k, n, code, M.ACT_SILU)
    space, size = M._workspace(lib.mscl_linear_quantized_workspace, call, xg)
    M._check(lib.mscl_linear_quantized(call, M._address(space), size, stream), "linear quantized")
    want = F.linear_quantized(q[:, 3:3 + k], scale, qw, sw, bgg, r.cuda(), "silu", t)
    F.assert_within(y[:, 3:3 + n], want, "8-bit y")
    assert bool((y[:, :3] == 77).all()) and bool((y[:, 3 + n:] == 77).all())


def test_offsets_beyond_32_bits():
    """Rows 2^31 elements apart: byte offsets past 2^33 (2^32 for 8 bits)."""
    gen = torch.Generator().manual_seed(80)
    m, k, n, far = 4, 72, 40, 2 ** 31
    room = torch.empty((m - 1) * far + 256, dtype=torch.bfloat16, device="cuda")
    x, wg, wu, bg, bu = gated_case(gen, m, k, n, torch.bfloat16)
    view = torch.as_strided(room, (m, k), (far, 1))
    view.copy_(x)
    note("gated, rows 2^31 elements apart")
    c = [t.cuda() for t in (wg, wu, bg, bu)]
    F.assert_within(M.gated_linear_tensors(view, *c), F.gated_linear(x, wg, wu, bg, bu, "silu")[0], "y")
    note("quantize, rows 2^31 elements apart")
    q, scale = M.quantize_tensors(view)
    assert torch.equal(q.cpu(), F.quantize(x)[0]) and torch.equal(scale.cpu(), F.quantize(x)[1])
    note("gated backward, rows 2^31 elements apart")
    dy, z, v = (normal(gen, m, n, dtype=torch.bfloat16) for _ in range(3))
    view = torch.as_strided(room, (m, n), (far, 1))
    view.copy_(dy)
    got = M.gated_linear_backward_tensors(view, x.cuda(), c[0], c[1], z.cuda(), v.cuda())
    within(got, F.gated_linear_backward(dy, x, wg, wu, z, v, "silu"), BACK)
    note("8 bits, rows 2^31 elements apart")
    bytes_ = room.view(torch.int8)
    xi, wi = integers(gen, 40, k), integers(gen, 5, k)
    view = torch.as_strided(bytes_, (5, k), (far, 1))
    view.copy_(wi)
    sx, sw = scales(gen, 40), scales(gen, 5)
    y = M.linear_quantized_tensors(xi.cuda(), sx.cuda(), view, sw.cuda(), dtype=torch.float32)
    F.assert_within(y, F.linear_quantized(xi, sx, wi, sw, None, None, "none", torch.float32), "8-bit y")


def test_large_products_of_far_rows():
    """Rows far apart, where offsets inside a tile come close to 31 bits, and beyond that, where other kernels run."""
    gen = torch.Generator().manual_seed(81)
    m, k, n = 2304, 520, 2048
    room = torch.empty((m - 1) * (2 ** 22 + 8) + k, dtype=torch.bfloat16, device="cuda")
    x, wg, wu, _, _ = gated_case(gen, m, k, n, torch.bfloat16, bias=False)
    xi, wi = integers(gen, m, 528), integers(gen, 4096, 528)
    c, ci = [t.cuda() for t in (x, wg, wu)], [t.cuda() for t in (xi, wi)]
    sx, sw = scales(gen, m).cuda(), scales(gen, 4096, 0.001).cuda()
    for far in (2 ** 22 - 8, 2 ** 22 + 8):
        note("large gated product of far rows", far)
        view = torch.as_strided(room, (m, k), (far, 1))
        view.copy_(x)
        F.assert_within(M.gated_linear_tensors(view, *c[1:]), F.gated_linear(*c, None, None, "silu")[0], "y")
        note("large 8-bit product of far rows", 2 * far)
        view = torch.as_strided(room.view(torch.int8), (m, 528), (2 * far - 16, 1))
        view.copy_(xi)
        y = M.linear_quantized_tensors(view, sx, ci[1], sw)
        F.assert_within(y, F.linear_quantized(ci[0], sx, ci[1], sw, None, None, "none", torch.bfloat16), "8-bit y")


@pytest.mark.parametrize("stride", [1, 3, 1 << 40])
def test_the_stride_of_a_single_row_is_ignored(stride):
    gen = torch.Generator().manual_seed(82)
    t = torch.bfloat16
    x, wg, wu, _, _ = (v.cuda() if v is not None else None for v in gated_case(gen, 1, 264, 136, t, bias=False))
    dy, z, v = (normal(gen, 1, 136, dtype=t).cuda() for _ in range(3))
    far = lambda a: torch.as_strided(a, tuple(a.shape), (stride, 1))  # noqa: E731
    note("stride of a single row", stride)
    assert torch.equal(M.gated_linear_tensors(far(x), wg, wu), M.gated_linear_tensors(x, wg, wu))
    for a, b in zip(M.gated_linear_backward_tensors(far(dy), far(x), wg, wu, far(z), far(v)),
                    M.gated_linear_backward_tensors(dy, x, wg, wu, z, v)):
        assert torch.equal(a, b)
    (q, s), (qw, sw) = M.quantize_tensors(far(x)), M.quantize_tensors(wg)
    assert torch.equal(q, M.quantize_tensors(x)[0])
    assert torch.equal(M.linear_quantized_tensors(far(q), s, qw, sw), M.linear_quantized_tensors(q, s, qw, sw))


def test_weights_whose_rows_lie_differently():
    """One weight's rows further apart than the other's, and one at odd addresses: each large product, and a small one."""
    gen = torch.Generator().manual_seed(83)
    for m, k, n in ((2304, 520, 2048), (60, 520, 70), (2200, 4096, 264)):
        x, wg, wu, _, _ = gated_case(gen, m, k, n, torch.bfloat16, bias=False)
        dy, z, v = (normal(gen, m, n, dtype=torch.bfloat16) for _ in range(3))
        c = [t.cuda() for t in (dy, x, wg, wu, z, v)]
        for forms in (("plain", "columns"), ("odd", "plain"), ("columns", "odd")):
            note("weights that lie differently", m, k, n, forms)
            a, b = placed(wg, forms[0]), placed(wu, forms[1])
            F.assert_within(M.gated_linear_tensors(c[1], a, b), F.gated_linear(*c[1:4], None, None, "silu")[0], "y")
            got = M.gated_linear_backward_tensors(c[0], c[1], a, b, *c[4:])
            within(got, F.gated_linear_backward(*c, "silu"), BACK)


# ---------------------------------------------------------------- streams, graphs, repeatability

def _inputs(rows, width, inner, t, seed=84):
    gen = torch.Generator().manual_seed(seed)
    x, wg, wu, bg, bu = gated_case(gen, rows, width, inner, t)
    wd = normal(gen, width, inner, scale=inner ** -0.5, dtype=t)
    return [v.cuda() for v in (x, wg, wu, bg, bu, wd, normal(gen, width, dtype=t), normal(gen, rows, width, dtype=t))]


def _run(x, wg, wu, bg, bu, wd, g, dy):
    """A layer's forward and backward pass, and the same forward pass in 8 bits."""
    h, mean, rstd = M.layer_norm_tensors(x, g, return_stats=True)
    a, z, v = M.gated_linear_tensors(h, wg, wu, bg, bu, return_preacts=True)
    y = M.linear_tensors(a, wd, None, x)
    da, dwd, _ = M.linear_backward_tensors(dy, a, wd, need_db=False)
    dh, *dw = M.gated_linear_backward_tensors(da, h, wg, wu, z, v)
    dx, dg, _ = M.layer_norm_backward_tensors(dh, x, mean, rstd, g, need_db=False)
    weights = [M.quantize_tensors(w) for w in (wg, wu, wd)]
    q, s = M.quantize_tensors(h)
    b = M.gated_linear_quantized_tensors(q, s, *weights[0], *weights[1], bg, bu, dtype=x.dtype)
    p, ps = M.quantize_tensors(b)
    served = M.linear_quantized_tensors(p, ps, *weights[2], residual=x, dtype=x.dtype)
    return (a, z, v, y, da, dwd, dh, *dw, dx, dg, q, s, b, p, ps, served)


RUNS = [(3, 256, 520, "bf16"), (200, 384, 1000, "fp16"), (600, 512, 1024, "bf16"), (90, 130, 77, "fp32"), (2100, 4104, 264, "bf16"),
        (2304, 1024, 2056, "fp32")]


@pytest.mark.parametrize("rows,width,inner,dtype", RUNS)
def test_a_layer_run_together(rows, width, inner, dtype):
    """Each result against its formula on what the operators before it gave."""
    t = DTYPES[dtype]
    args = _inputs(rows, width, inner, t)
    x, wg, wu, bg, bu, wd, g, dy = args
    note("layer", rows, width, inner, dtype)
    a, z, v, y, da, dwd, dh, dwg, dwu, dbg, dbu, dx, dg, q, s, b, p, ps, served = _run(*args)
    h, mean, rstd = M.layer_norm_tensors(x, g, return_stats=True)
    within((a, z, v), F.gated_linear(h, wg, wu, bg, bu, "silu"), ("a", "z", "v"))
    F.assert_within(y, O.linear(a, wd, None, x, "none")[0], "y")
    within((dh, dwg, dwu, dbg, dbu), F.gated_linear_backward(da, h, wg, wu, z, v, "silu"), BACK)
    within((da, dwd), O.linear_backward(dy, a, wd, None, "none")[:2], ("da", "dwd"))
    F.assert_within(dx, O.layer_norm_backward(dh, x, mean, rstd, g, t)[0], "dx")
    weights = [F.quantize(w.cpu()) for w in (wg, wu, wd)]
    weights = [(i.cuda(), c.cuda()) for i, c in weights]
    want_q, want_s = F.quantize(h.cpu())
    assert torch.equal(q.cpu(), want_q) and torch.equal(s.cpu(), want_s)
    F.assert_within(b, F.gated_linear_quantized(q, s, *weights[0], *weights[1], bg, bu, "silu", t), "8-bit a")
    want_p, want_ps = F.quantize(b.cpu())
    assert torch.equal(p.cpu(), want_p) and torch.equal(ps.cpu(), want_ps)
    F.assert_within(served, F.linear_quantized(p, ps, *weights[2], None, x, "none", t), "8-bit y")


@pytest.mark.parametrize("rows,width,inner,dtype", RUNS)
def test_the_same_call_gives_the_same_bits(rows, width, inner, dtype):
    """Also on copies of its buffers, and over a workspace that held something else before."""
    args = _inputs(rows, width, inner, DTYPES[dtype])
    note("repeat", rows, width, inner, dtype)
    first = _run(*args)
    for fill in (math.nan, 1.0, -math.inf):
        dirt = [torch.full((1 << 24,), fill, device="cuda") for _ in range(4)]
        del dirt  # memory that the next calls' workspaces and results are made of
        for a, b in zip(first, _run(*[v.clone() for v in args])):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rows,width,inner,dtype", RUNS)
def test_graph_replays(rows, width, inner, dtype):
    args = _inputs(rows, width, inner, DTYPES[dtype])
    note("graph", rows, width, inner, dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _run(*args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(*args)
    gen = torch.Generator().manual_seed(85)
    for replay in range(4):
        args[0].copy_(normal(gen, rows, width, dtype=args[0].dtype))
        args[-1].copy_(normal(gen, rows, width, dtype=args[0].dtype))
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        for a, b in zip(got, _run(*args)):
            assert torch.equal(a, b), f"replay {replay}"


def test_on_another_stream_and_two_at_once():
    args = _inputs(600, 512, 1024, torch.bfloat16)
    x, wg, wu, bg, bu = args[:5]
    want = _run(*args)
    torch.cuda.synchronize()
    note("another stream")
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        y, z, v = M.gated_linear_tensors(x, wg, wu, bg, bu, return_preacts=True, stream=stream)
        back = M.gated_linear_backward_tensors(y, x, wg, wu, z, v, stream=stream)
        q, s = M.quantize_tensors(x, stream=stream)
        w, ws = M.quantize_tensors(wg, stream=stream)
        lin = M.linear_quantized_tensors(q, s, w, ws, bg, stream=stream)
        gat = M.gated_linear_quantized_tensors(q, s, w, ws, w, ws, stream=stream)
        side.synchronize()
        assert torch.equal(y, M.gated_linear_tensors(x, wg, wu, bg, bu)) and torch.equal(q, M.quantize_tensors(x)[0])
        assert torch.equal(lin, M.linear_quantized_tensors(q, s, w, ws, bg))
        assert torch.equal(gat, M.gated_linear_quantized_tensors(q, s, w, ws, w, ws))
        for a, b in zip(back, M.gated_linear_backward_tensors(y, x, wg, wu, z, v)):
            assert torch.equal(a, b)
    results = []
    for stream in (side, other):
        stream.wait_stream(torch.cuda.default_stream())
        with torch.cuda.stream(stream):
            results.append([_run(*args) for _ in range(3)])
    torch.cuda.synchronize()
    for runs in results:
        for got in runs:
            for a, b in zip(got, want):
                assert torch.equal(a, b)


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from allreduce_emulated_peer_amd import mscl as M
x, wg, wu = (torch.randn(s, device="cuda").bfloat16() for s in ((2304, 264), (2048, 264), (2048, 264)))
q = torch.ones(2304, 528, dtype=torch.int8, device="cuda"); s = torch.ones(2304, device="cuda")
f = torch.randn(2304, 1024, device="cuda"); fw = torch.randn(2048, 1024, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, z, v = M.gated_linear_tensors(x, wg, wu, return_preacts=True)
    d = M.gated_linear_backward_tensors(y, x, wg, wu, z, v)
    i = M.linear_quantized_tensors(q, s, q, s)
    p = M.gated_linear_tensors(f, fw, fw)
graph.replay()
torch.cuda.synchronize()
assert torch.equal(y, M.gated_linear_tensors(x, wg, wu)) and torch.equal(i, M.linear_quantized_tensors(q, s, q, s))
assert torch.equal(p, M.gated_linear_tensors(f, fw, fw))
for a, b in zip(d, M.gated_linear_backward_tensors(y, x, wg, wu, z, v)):
    assert torch.equal(a, b)
print("captured first")
"""


def test_the_first_call_of_a_process_can_be_captured():
    note("first call captured")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=110)
    assert out.returncode == 0 and "captured first" in out.stdout, out.stderr[-2000:]


def test_a_gradient_is_not_lost_unseen():
    x = torch.randn(4, 64, device="cuda", requires_grad=True)
    w = torch.randn(32, 64, device="cuda")
    note("autograd")
    y = M.gated_linear_tensors(x, w, w)
    assert y.requires_grad
    with pytest.raises(RuntimeError, match="gated_linear_backward_tensors"):
        y.sum().backward()
    _, scale = M.quantize_tensors(x)
    assert scale.requires_grad
    with pytest.raises(RuntimeError, match="no gradient"):
        scale.sum().backward()
    with torch.no_grad():
        q, scale = M.quantize_tensors(x)
        assert not scale.requires_grad
    qw, sw = M.quantize_tensors(w)
    b = torch.zeros(32, device="cuda", requires_grad=True)
    for y in (M.linear_quantized_tensors(q, scale, qw, sw, b, dtype=torch.float32),
              M.gated_linear_quantized_tensors(q, scale, qw, sw, qw, sw, b, dtype=torch.float32)):
        assert y.requires_grad
        with pytest.raises(RuntimeError, match="no gradient"):
            y.sum().backward()
