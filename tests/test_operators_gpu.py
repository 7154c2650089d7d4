"""The linear layer and layer norm on the GPU against their formulas in 64 bits."""

import math
import sys

import pytest
import torch

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


def placed(t, form):
    """t on the GPU: as it is, as a block of columns of a wider matrix, or off 16-byte alignment."""
    if t is None or form == "plain":
        return None if t is None else t.cuda()
    if t.dim() == 1:
        room = torch.full((t.shape[0] + 3,), math.nan, dtype=t.dtype, device="cuda")
        room[1:-2] = t.cuda()
        return room[1:-2]
    pad = {"columns": (8, 16), "odd": (3, 2)}[form]
    room = torch.full((t.shape[0], t.shape[1] + sum(pad)), math.nan, dtype=t.dtype, device="cuda")
    view = room[:, pad[0]:pad[0] + t.shape[1]]
    view.copy_(t)
    return view


# From one row to several tiles, k from one to many blocks; no size a multiple of what a kernel works in, and some that are.
SIZES = [(1, 1, 1), (1, 256, 128), (2, 40, 3), (5, 1000, 33), (16, 64, 64), (31, 8, 100), (33, 129, 65), (64, 512, 256),
         (65, 72, 136), (100, 2049, 70), (127, 31, 257), (128, 128, 128), (256, 256, 512), (300, 96, 520), (513, 320, 264)]


def linear_case(gen, m, k, n, t, bias=True, residual=True):
    x, w = normal(gen, m, k, dtype=t), normal(gen, n, k, scale=max(k, 1) ** -0.5, dtype=t)
    return x, w, normal(gen, n, scale=0.5, dtype=t) if bias else None, normal(gen, m, n, dtype=t) if residual else None


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", ["plain", "columns", "odd"])
def test_linear(dtype, form):
    gen = torch.Generator().manual_seed(11)
    t = DTYPES[dtype]
    for i, (m, k, n) in enumerate(SIZES):
        act = ACTS[i % len(ACTS)]
        x, w, b, r = linear_case(gen, m, k, n, t, bias=i % 3 != 0, residual=i % 4 != 0)
        note("linear", dtype, form, m, k, n, act)
        y, z = M.linear_tensors(placed(x, form), placed(w, form), placed(b, form), placed(r, form), act,
                                return_preact=True)
        alone = M.linear_tensors(placed(x, form), placed(w, form), placed(b, form), placed(r, form), act)
        want_y, want_z = O.linear(x, w, b, r, act)
        O.assert_within(y, want_y, f"y {m}x{k}x{n} {act}")
        O.assert_within(z, want_z, f"z {m}x{k}x{n} {act}")
        assert torch.equal(alone, y)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ACTS)
def test_activations_over_their_range(dtype, act):
    """One product with the identity: every value of the activation and its slope."""
    t = DTYPES[dtype]
    z = torch.cat([torch.linspace(-14, 14, 4000), torch.linspace(-0.01, 0.01, 96)]).to(t).reshape(64, 64)
    eye = torch.eye(64, dtype=t)
    note("activation", dtype, act)
    y = M.linear_tensors(z.cuda(), eye.cuda(), activation=act)
    O.assert_within(y, O.linear(z, eye, None, None, act)[0], f"{act}")
    ones = torch.ones(64, 64, dtype=t)
    dx, dw, db = M.linear_backward_tensors(ones.cuda(), eye.cuda(), eye.cuda(), z.cuda(), act)
    want = O.linear_backward(ones, eye, eye, z, act)
    for got, w, name in ((dx, want[0], "dx"), (dw, want[1], "dw"), (db, want[2], "db")):
        O.assert_within(got, w, f"{act} {name}")


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("form", ["plain", "columns", "odd"])
def test_linear_backward(dtype, form):
    gen = torch.Generator().manual_seed(12)
    t = DTYPES[dtype]
    for i, (m, k, n) in enumerate(SIZES):
        act = ACTS[(i + 2) % len(ACTS)]
        x, w, _, dy = linear_case(gen, m, k, n, t)
        z = normal(gen, m, n, scale=1.5, dtype=t) if act != "none" else None
        note("linear backward", dtype, form, m, k, n, act)
        args = (placed(dy, form), placed(x, form), placed(w, form), placed(z, form), act)
        got = M.linear_backward_tensors(*args)
        for g, want, name in zip(got, O.linear_backward(dy, x, w, z, act), ("dx", "dw", "db")):
            O.assert_within(g, want, f"{name} {m}x{k}x{n} {act}")
        for only in range(3):
            need = {f"need_{n}": i == only for i, n in enumerate(("dx", "dw", "db"))}
            one = M.linear_backward_tensors(*args, **need)
            assert torch.equal(one[only], got[only]) and sum(g is None for g in one) == 2


# Large products of 16-bit types (256 x 256 tiles): forward, and both gradients, with edges inside a tile, k that ends
# inside a block, odd and even numbers of blocks, and operands that have to be laid out anew.
@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,k,n,form", [(2304, 4096, 4096, "plain"), (2100, 4104, 4000, "plain"),
                                        (2100, 4104, 4000, "columns"), (2300, 4099, 3907, "odd"),
                                        (4097, 320, 2056, "plain"), (2049, 264, 4111, "columns")])
def test_large_products(dtype, m, k, n, form):
    gen = torch.Generator().manual_seed(18)
    t = DTYPES[dtype]
    x, w, b, r = linear_case(gen, m, k, n, t)
    dy, z = normal(gen, m, n, dtype=t), normal(gen, m, n, scale=1.5, dtype=t)
    for act in ("gelu", "none"):
        note("large linear", dtype, m, k, n, form, act)
        xg, wg, bg, rg, dyg, zg = (placed(v, form) for v in (x, w, b, r, dy, z))
        got = M.linear_tensors(xg, wg, bg, rg, act, return_preact=True)
        c = [v.cuda() for v in (x, w, b, r, dy, z)]  # the oracle's 64 bits on the GPU, from contiguous copies
        for g, want, name in zip(got, O.linear(c[0], c[1], c[2], c[3], act), ("y", "z")):
            O.assert_within(g, want, f"{name} {act}")
        note("large linear backward", dtype, m, k, n, form, act)
        back = M.linear_backward_tensors(dyg, xg, wg, zg, act)
        for g, want, name in zip(back, O.linear_backward(c[4], c[0], c[1], c[5], act), ("dx", "dw", "db")):
            O.assert_within(g, want, f"{name} {act}")
        for a, b2 in zip(back, M.linear_backward_tensors(dyg, xg, wg, zg, act)):
            assert torch.equal(a, b2)


def test_large_products_of_far_rows():
    """Rows almost 2^22 elements apart, where offsets inside a tile come close to 31 bits, and k that ends inside a block."""
    gen = torch.Generator().manual_seed(27)
    far, m, k, n = 2 ** 22 - 8, 2304, 520, 4096
    x, w, _, _ = linear_case(gen, m, k, n, torch.bfloat16)
    note("large product of far rows: forward")
    room = torch.empty((m - 1) * far + k, dtype=torch.bfloat16, device="cuda")
    view = torch.as_strided(room, (m, k), (far, 1))
    view.copy_(x)
    c = [v.cuda() for v in (x, w)]
    O.assert_within(M.linear_tensors(view, c[1]), O.linear(c[0], c[1], None, None, "none")[0], "y")
    note("large product of far rows: input gradient")
    dy, wt = normal(gen, m, k, dtype=torch.bfloat16).cuda(), normal(gen, k, n, dtype=torch.bfloat16).cuda()
    del view
    view = torch.as_strided(room, (k, n), (far, 1))
    view.copy_(wt)
    dx, _, _ = M.linear_backward_tensors(dy, torch.empty(m, n, dtype=torch.bfloat16, device="cuda"), view,
                                         need_dw=False, need_db=False)
    O.assert_within(dx, O.linear_backward(dy, torch.zeros(m, n, dtype=torch.bfloat16, device="cuda"), wt, None, "none")[0],
                    "dx")


def test_large_product_keeps_nan_in_its_row_and_column():
    gen = torch.Generator().manual_seed(19)
    m, k, n = 2100, 712, 4100
    x, w, b, _ = linear_case(gen, m, k, n, torch.bfloat16)
    x[2099, 711], w[4099, 700] = math.nan, math.inf
    x[:, 700] = x[:, 700].abs() + 1
    note("large product with NaN")
    y = M.linear_tensors(x.cuda(), w.cuda(), b.cuda()).cpu()
    assert bool(torch.isnan(y[2099]).all()) and bool((y[:2099, 4099] == math.inf).all())
    assert bool(torch.isfinite(y[:2099, :4099]).all())


@pytest.mark.parametrize("m,k,n", [(70, 130, 90), (1001, 300, 1537), (513, 2047, 260)])
def test_binary32_products_over_the_whole_range(m, k, n):
    """Rows and columns of very different size, and sums that leave the range, next to infinities and NaN."""
    gen = torch.Generator().manual_seed(20)
    x, w, b, dy = linear_case(gen, m, k, n, torch.float32)
    x = x * torch.exp2(torch.randint(-60, 60, (m, 1), generator=gen).float())
    w = w * torch.exp2(torch.randint(-60, 60, (n, 1), generator=gen).float())
    note("binary32 range", m, k, n)
    c = [v.cuda() for v in (x, w, dy)]
    O.assert_within(M.linear_tensors(c[0], c[1]), O.linear(c[0], c[1], None, None, "none")[0], "y")
    for g, want, name in zip(M.linear_backward_tensors(c[2], c[0], c[1]), O.linear_backward(c[2], c[0], c[1], None, "none"),
                             ("dx", "dw", "db")):
        O.assert_within(g, want, name)
    top = torch.finfo(torch.float32).max
    x, w = x.sign(), w.sign()
    x[3, :], w[5, :] = 0, 0
    x[3, 0], x[3, 1], w[:, 0], w[:, 1] = top, top, 1, 1  # twice the largest value
    w[5, 0] = 1
    x[7, 2], w[:, 2] = math.inf, 1
    w[9, 4], x[:, 4] = -math.inf, 1
    x[11, 6] = math.nan
    y = M.linear_tensors(x.cuda(), w.cuda()).cpu()
    assert y[3, 5] == math.inf and y[3, 6] == math.inf and y[7, 5] == math.inf and y[5, 9] == -math.inf
    assert bool(torch.isnan(y[11]).all()) and bool(torch.isnan(y[7, 9]))
    rows = [i for i in range(m) if i not in (3, 7, 11)]
    cols = [i for i in range(n) if i != 9]
    assert bool((y[rows][:, 9] == -math.inf).all())
    want = x[rows].double() @ w[cols].double().t()
    assert torch.equal(y[rows][:, cols].double(), want)  # sums of signs are exact


def test_binary32_products_of_the_largest_and_smallest_values():
    top, low = torch.finfo(torch.float32).max, torch.finfo(torch.float32).smallest_normal
    x, w = torch.zeros(80, 70), torch.zeros(100, 70)
    x[3, 0], x[4, 1], x[5, 2] = top, -top, low
    w[:, 0], w[:, 1], w[:, 2] = 1, 1, 1
    note("largest and smallest values")
    y = M.linear_tensors(x.cuda(), w.cuda()).cpu()
    assert bool((y[3] == top).all()) and bool((y[4] == -top).all()) and bool((y[5] == low).all())
    assert not bool(y[[i for i in range(80) if i not in (3, 4, 5)]].any())


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("m,k,n,form", [(1, 8200, 70, "plain"), (3, 4100, 200, "odd"), (9, 12289, 33, "columns"),
                                        (17, 8192, 48, "plain"), (32, 5003, 130, "odd"), (12, 640, 8300, "plain"),
                                        (32, 100, 8200, "columns")])
def test_few_rows(dtype, m, k, n, form):
    """Up to 32 rows: k split over workgroups and waves, ends of k inside a step, one and two tiles of rows."""
    gen = torch.Generator().manual_seed(26)
    x, w, b, r = linear_case(gen, m, k, n, DTYPES[dtype])
    note("few rows", dtype, m, k, n, form)
    args = [placed(v, form) for v in (x, w, b, r)]
    y, z = M.linear_tensors(*args, "gelu_tanh", return_preact=True)
    want = O.linear(x, w, b, r, "gelu_tanh")
    O.assert_within(y, want[0], "y")
    O.assert_within(z, want[1], "z")
    assert torch.equal(y, M.linear_tensors(*args, "gelu_tanh"))


def test_linear_many_leading_dimensions():
    gen = torch.Generator().manual_seed(13)
    x, w, b, _ = linear_case(gen, 30, 24, 40, torch.bfloat16)
    r = normal(gen, 2, 3, 5, 40, dtype=torch.bfloat16)
    note("linear of 2 x 3 x 5 x 24")
    y, z = M.linear_tensors(x.view(2, 3, 5, 24).cuda(), w.cuda(), b.cuda(), r.cuda(), "silu", return_preact=True)
    assert y.shape == z.shape == (2, 3, 5, 40)
    O.assert_within(y.view(30, 40), O.linear(x, w, b, r.view(30, 40), "silu")[0], "y")
    dx, dw, db = M.linear_backward_tensors(r.cuda(), x.view(2, 3, 5, 24).cuda(), w.cuda(), z, "silu")
    assert dx.shape == (2, 3, 5, 24) and dw.shape == (40, 24) and db.shape == (40,)
    one = M.linear_tensors(x[0].cuda(), w.cuda())
    assert one.shape == (40,)
    O.assert_within(one.view(1, 40), O.linear(x[:1], w, None, None, "none")[0], "one row")


@pytest.mark.parametrize("dtype", DTYPES)
def test_linear_empty(dtype):
    t = DTYPES[dtype]
    e = lambda *s: torch.ones(s, dtype=t, device="cuda")  # noqa: E731
    note("empty sizes", dtype)
    assert M.linear_tensors(e(0, 5), e(7, 5)).shape == (0, 7)
    assert M.linear_tensors(e(4, 5), e(0, 5)).shape == (4, 0)
    y = M.linear_tensors(e(4, 0), e(7, 0), e(7), e(4, 7), "relu")  # relu(bias) + residual
    assert torch.equal(y, torch.full_like(y, 2))
    dx, dw, db = M.linear_backward_tensors(e(0, 7), e(0, 5), e(7, 5), e(0, 7), "gelu")
    assert dx.shape == (0, 5) and not dw.any() and not db.any() and dw.shape == (7, 5) and db.shape == (7,)
    dx, dw, db = M.linear_backward_tensors(e(4, 0), e(4, 5), e(0, 5))
    assert dx.shape == (4, 5) and not dx.any() and dw.shape == (0, 5) and db.shape == (0,)
    dx, dw, db = M.linear_backward_tensors(e(4, 7), e(4, 0), e(7, 0))
    assert torch.equal(db, torch.full_like(db, 4))


def test_linear_nan_and_infinity_stay_in_their_rows_and_columns():
    gen = torch.Generator().manual_seed(14)
    for m, k, n in ((40, 70, 50), (300, 320, 512)):
        x, w, b, _ = linear_case(gen, m, k, n, torch.bfloat16)
        x[3, 5], x[7, k - 1], w[11, 0] = math.nan, math.inf, -math.inf
        note("linear with NaN and infinity", m, k, n)
        y = M.linear_tensors(x.cuda(), w.cuda(), b.cuda()).cpu()
        bad = torch.zeros(m, n, dtype=torch.bool)
        bad[3], bad[7], bad[:, 11] = True, True, True
        assert bool(torch.isfinite(y[~bad]).all()) and not bool(torch.isfinite(y[bad]).any())
        assert bool(torch.isnan(y[3]).all())
        inf = y[7].float()
        sign = torch.sign(w[:, k - 1].float())
        rows = torch.arange(n) != 11
        assert torch.equal(inf[rows & (sign != 0)], (sign * math.inf)[rows & (sign != 0)])
    z = torch.tensor([[math.inf, -math.inf, math.nan, 0.0]], dtype=torch.float32)
    for dtype in DTYPES:
        t = DTYPES[dtype]
        for act in ACTS:
            # bias carries the values, so that no product with them is taken
            y = M.linear_tensors(torch.zeros(1, 8, dtype=t, device="cuda"), torch.zeros(4, 8, dtype=t, device="cuda"),
                                 z[0].to(t).cuda(), activation=act).cpu()[0]
            assert y[0] == math.inf and bool(torch.isnan(y[2])) and y[3] == 0
            assert y[1] == (-math.inf if act == "none" else 0)
            db = M.linear_backward_tensors(torch.ones(1, 4, dtype=t, device="cuda"),
                                           torch.zeros(1, 8, dtype=t, device="cuda"),
                                           torch.zeros(4, 8, dtype=t, device="cuda"), z.to(t).cuda(), act)[2].cpu()
            assert db[0] == 1 and db[1] == (1 if act == "none" else 0)


def test_linear_gradients_against_differences():
    gen = torch.Generator().manual_seed(15)
    m, k, n = 70, 90, 130
    for act in ACTS:
        x, w, b, dy = linear_case(gen, m, k, n, torch.float32)
        note("differences", act)
        _, z = M.linear_tensors(x.cuda(), w.cuda(), b.cuda(), activation=act, return_preact=True)
        grads = M.linear_backward_tensors(dy.cuda(), x.cuda(), w.cuda(), z, act)
        if act == "relu":  # away from the corner, which a difference would step over
            keep = z.cpu().abs() > 1e-2
            dy = dy * keep
            grads = M.linear_backward_tensors(dy.cuda(), x.cuda(), w.cuda(), z, act)

        def loss(v):
            return float((O.activate(v[0] @ v[1].t() + v[2], act) * dy.double()).sum())

        at = [x.double(), w.double(), b.double()]
        for i, g in enumerate(grads):
            d = torch.randn(at[i].shape, generator=gen, dtype=torch.float64)
            h = 1e-5
            hi, lo = list(at), list(at)
            hi[i], lo[i] = at[i] + h * d, at[i] - h * d
            slope = (loss(hi) - loss(lo)) / (2 * h)
            # each gradient value is off by 2^-20 of its terms at most, so is their sum along d of that size;
            # the difference's own error is h^2 times the third derivative
            size = float((g.cpu().double() * d).abs().sum())
            assert abs(slope - float((g.cpu().double() * d).sum())) < 2e-6 * size + 1e-4, (act, i)


def test_residual_in_place_and_strided_outputs():
    """Through the C ABI: y over the residual, y and preact as columns of a wider matrix whose other columns stay."""
    gen = torch.Generator().manual_seed(16)
    for m, k, n, t in ((33, 80, 50, torch.bfloat16), (300, 256, 260, torch.float16), (70, 30, 45, torch.float32)):
        x, w, b, r = linear_case(gen, m, k, n, t)
        xg, wg, bg = x.cuda(), w.cuda(), b.cuda()
        room = torch.full((m, n + 7), 77.0, dtype=t, device="cuda")
        room[:, 3:3 + n] = r.cuda()
        keep = torch.full((m, n + 5), 55.0, dtype=t, device="cuda")
        code = {torch.bfloat16: M.BFLOAT16, torch.float16: M.FLOAT16, torch.float32: M.FLOAT32}[t]
        at = room[:, 3:].data_ptr()
        call = M.LINEAR.pack(xg.data_ptr(), k, wg.data_ptr(), k, bg.data_ptr(), at, n + 7, at, n + 7,
                             keep[:, 1:].data_ptr(), n + 5, m, k, n, code, M.ACT_GELU)
        note("residual in place", m, k, n, t)
        space, size = M._workspace(M.load().mscl_linear_workspace, call, xg)
        M._check(M.load().mscl_linear(call, M._address(space), size, torch.cuda.current_stream().cuda_stream), "linear")
        want = O.linear(x, w, b, r, "gelu")
        O.assert_within(room[:, 3:3 + n], want[0], "y")
        O.assert_within(keep[:, 1:1 + n], want[1], "preact")
        assert bool((room[:, :3] == 77).all()) and bool((room[:, 3 + n:] == 77).all())
        assert bool((keep[:, :1] == 55).all()) and bool((keep[:, 1 + n:] == 55).all())


def test_offsets_beyond_32_bits():
    """Rows 2^31 elements apart: byte offsets past 2^33, element offsets past 2^32."""
    gen = torch.Generator().manual_seed(17)
    m, k, n, far = 4, 72, 40, 2 ** 31
    x, w, b, dy = linear_case(gen, m, k, n, torch.bfloat16)
    note("rows 2^31 elements apart")
    room = torch.empty((m - 1) * far + 256, dtype=torch.bfloat16, device="cuda")
    for name in ("linear", "backward", "norm", "norm backward"):
        note(name)
        cols = n if "backward" in name and "norm" not in name else k
        view = torch.as_strided(room, (m, cols), (far, 1))
        if name == "linear":
            view.copy_(x)
            O.assert_within(M.linear_tensors(view, w.cuda(), b.cuda()), O.linear(x, w, b, None, "none")[0], "y")
        elif name == "backward":
            view.copy_(dy)
            got = M.linear_backward_tensors(view, x.cuda(), w.cuda())
            for g, want in zip(got, O.linear_backward(dy, x, w, None, "none")):
                O.assert_within(g, want, name)
        else:
            view.copy_(x)
            y, mean, rstd = M.layer_norm_tensors(view, return_stats=True)
            want = O.layer_norm(x, None, None, 1e-5)
            O.assert_within(y, want[0], name)
            if name == "norm backward":
                g = normal(gen, m, k, dtype=torch.bfloat16)
                got = M.layer_norm_backward_tensors(g.cuda(), view, mean, rstd)
                for a, w2 in zip(got, O.layer_norm_backward(g, x, mean.cpu(), rstd.cpu(), None, torch.bfloat16)):
                    O.assert_within(a, w2, name)


# ---------------------------------------------------------------- layer norm

NORM_SIZES = [(1, 1), (3, 2), (5, 7), (1, 8), (9, 64), (4, 129), (7, 511), (33, 512), (6, 1000), (2, 1025), (17, 2048),
              (3, 2049), (5, 4097), (70, 768), (2, 8192), (3, 8193), (2, 16387), (1, 20001), (2, 33000), (1, 70001),
              (260, 300), (1030, 24), (2051, 40), (1100, 700), (1025, 1500),
              (1100, 3000), (1027, 5000), (2050, 12001)]


def norm_case(gen, rows, width, t, p):
    x = normal(gen, rows, width, scale=2.0) + normal(gen, rows, 1, scale=0.5)
    return x.to(t), (1 + normal(gen, width, scale=0.2)).to(p), normal(gen, width, scale=0.2).to(p)


@pytest.mark.parametrize("dtype,params", [("fp32", "fp32"), ("bf16", "bf16"), ("bf16", "fp32"), ("fp16", "fp16"),
                                          ("fp16", "fp32")])
@pytest.mark.parametrize("form", ["plain", "columns", "odd"])
def test_layer_norm(dtype, params, form):
    gen = torch.Generator().manual_seed(21)
    t, p = DTYPES[dtype], DTYPES[params]
    for i, (rows, width) in enumerate(NORM_SIZES):
        x, w, b = norm_case(gen, rows, width, t, p)
        if i % 5 == 3:
            w = None
        if i % 4 == 2:
            b = None
        note("layer norm", dtype, params, form, rows, width)
        xg, wg, bg = placed(x, form), placed(w, form), placed(b, form)
        y, mean, rstd = M.layer_norm_tensors(xg, wg, bg, return_stats=True)
        want = O.layer_norm(x, w, b, 1e-5)
        for g, e, name in zip((y, mean, rstd), want, ("y", "mean", "rstd")):
            O.assert_within(g, e, f"{name} {rows}x{width}")
        assert torch.equal(M.layer_norm_tensors(xg, wg, bg), y)
        dy = normal(gen, rows, width, dtype=t)
        note("layer norm backward", dtype, params, form, rows, width)
        dyg = placed(dy, form)
        got = M.layer_norm_backward_tensors(dyg, xg, mean, rstd, wg)
        kind = t if w is None else p
        want = O.layer_norm_backward(dy, x, mean.cpu(), rstd.cpu(), w, kind)
        for g, e, name in zip(got, want, ("dx", "dw", "db")):
            O.assert_within(g, e, f"{name} {rows}x{width}")
        assert got[0].dtype == t and got[1].dtype == got[2].dtype == kind
        for only in range(3):
            need = {f"need_{n}": k == only for k, n in enumerate(("dx", "dw", "db"))}
            one = M.layer_norm_backward_tensors(dyg, xg, mean, rstd, wg, **need)
            O.assert_within(one[only], want[only], f"{only} alone {rows}x{width}")


@pytest.mark.parametrize("dtype", DTYPES)
def test_layer_norm_of_no_rows(dtype):
    t = DTYPES[dtype]
    note("layer norm of no rows", dtype)
    for width in (5, 3000):
        x = torch.empty(0, width, dtype=t, device="cuda")
        w = torch.ones(width, dtype=t, device="cuda")
        y, mean, rstd = M.layer_norm_tensors(x, w, w, return_stats=True)
        assert y.shape == (0, width) and mean.shape == rstd.shape == (0,)
        dx, dw, db = M.layer_norm_backward_tensors(x, x, mean, rstd, w)
        assert dx.shape == (0, width) and dw.shape == db.shape == (width,) and not dw.any() and not db.any()


def test_layer_norm_constant_rows_and_far_means():
    for dtype in DTYPES:
        t = DTYPES[dtype]
        note("constant rows", dtype)
        x = torch.full((3, 640), 3.5, dtype=t)
        y, mean, rstd = M.layer_norm_tensors(x.cuda(), eps=1e-5, return_stats=True)
        assert not bool(y.any()) and bool((mean == 3.5).all())
        assert torch.allclose(rstd.cpu(), torch.full((3,), 1e-5).rsqrt(), rtol=1e-6)
        one = M.layer_norm_tensors(torch.full((4, 1), 2.0, dtype=t, device="cuda"))  # one element is its own mean
        assert not bool(one.any())
    gen = torch.Generator().manual_seed(22)
    x = normal(gen, 5, 3000) + 1000.0  # E[x^2] - mean^2 would lose the variance here
    y, mean, rstd = M.layer_norm_tensors(x.cuda(), return_stats=True)
    want = O.layer_norm(x, None, None, 1e-5)
    for g, e, name in zip((y, mean, rstd), want, ("y", "mean", "rstd")):
        O.assert_within(g, e, name)


def test_layer_norm_nan_and_infinity_stay_in_their_row():
    gen = torch.Generator().manual_seed(23)
    for width in (200, 1000, 9000):
        x, w, b = norm_case(gen, 6, width, torch.bfloat16, torch.bfloat16)
        x[1, 3], x[4, width - 1] = math.nan, math.inf
        note("layer norm with NaN", width)
        y = M.layer_norm_tensors(x.cuda(), w.cuda(), b.cuda()).cpu()
        for row in range(6):
            assert bool(torch.isnan(y[row]).all()) == (row in (1, 4))
            assert row in (1, 4) or bool(torch.isfinite(y[row]).all())


def test_layer_norm_gradients_against_differences():
    gen = torch.Generator().manual_seed(24)
    x, w, b = norm_case(gen, 20, 300, torch.float32, torch.float32)
    dy = normal(gen, 20, 300)
    note("layer norm differences")
    _, mean, rstd = M.layer_norm_tensors(x.cuda(), w.cuda(), b.cuda(), return_stats=True)
    grads = M.layer_norm_backward_tensors(dy.cuda(), x.cuda(), mean, rstd, w.cuda())

    def loss(v):
        return float((O.layer_norm(v[0], v[1], v[2], 1e-5)[0][0] * dy.double()).sum())

    at = [x.double(), w.double(), b.double()]
    for i, g in enumerate(grads):
        d = torch.randn(at[i].shape, generator=gen, dtype=torch.float64)
        h = 1e-5
        hi, lo = list(at), list(at)
        hi[i], lo[i] = at[i] + h * d, at[i] - h * d
        size = float((g.cpu().double() * d).abs().sum())
        assert abs((loss(hi) - loss(lo)) / (2 * h) - float((g.cpu().double() * d).sum())) < 2e-6 * size + 1e-4


def test_layer_norm_in_place():
    """Through the C ABI: y over x, dx over dy."""
    gen = torch.Generator().manual_seed(25)
    for rows, width, t, code in ((40, 700, torch.bfloat16, M.BFLOAT16), (300, 5000, torch.float32, M.FLOAT32),
                                 (3, 70000, torch.float16, M.FLOAT16), (700, 300, torch.bfloat16, M.BFLOAT16)):
        x, w, b = norm_case(gen, rows, width, t, t)
        dy = normal(gen, rows, width, dtype=t)
        xg, wg, bg, dg = x.cuda(), w.cuda(), b.cuda(), dy.cuda()
        note("layer norm in place", rows, width)
        stats = torch.empty(2, rows, device="cuda")
        s = torch.cuda.current_stream().cuda_stream
        lib = M.load()
        want = O.layer_norm(x, w, b, 1e-5)
        y = xg.clone()
        M._check(lib.mscl_layer_norm(M.LAYER_NORM.pack(
            y.data_ptr(), width, wg.data_ptr(), bg.data_ptr(), y.data_ptr(), width, stats[0].data_ptr(),
            stats[1].data_ptr(), rows, width, 1e-5, code, code), s), "norm")
        O.assert_within(y, want[0], "y over x")
        dw, db = torch.empty_like(wg), torch.empty_like(wg)
        call = M.LAYER_NORM_BACKWARD.pack(dg.data_ptr(), width, xg.data_ptr(), width, stats[0].data_ptr(),
                                          stats[1].data_ptr(), wg.data_ptr(), dg.data_ptr(), width, dw.data_ptr(),
                                          db.data_ptr(), rows, width, code, code)
        space, size = M._workspace(lib.mscl_layer_norm_backward_workspace, call, xg)
        M._check(lib.mscl_layer_norm_backward(call, M._address(space), size, s), "norm backward")
        want = O.layer_norm_backward(dy, x, stats[0].cpu(), stats[1].cpu(), w, t)
        for g, e, name in zip((dg, dw, db), want, ("dx over dy", "dw", "db")):
            O.assert_within(g, e, name)


# ---------------------------------------------------------------- streams, graphs, repeatability

def _layer(x, w1, b1, w2, g, b, dy):
    """Forward and backward of linear -> gelu -> linear + residual -> layer norm."""
    h, z = M.linear_tensors(x, w1, b1, None, "gelu", return_preact=True)
    s = M.linear_tensors(h, w2, None, x)
    y, mean, rstd = M.layer_norm_tensors(s, g, b, return_stats=True)
    ds, dg, db = M.layer_norm_backward_tensors(dy, s, mean, rstd, g)
    dh, dw2, _ = M.linear_backward_tensors(ds, h, w2, need_db=False)
    dx, dw1, db1 = M.linear_backward_tensors(dh, x, w1, z, "gelu")
    return y, ds, dg, db, dh, dw2, dx, dw1, db1


def _layer_inputs(rows, width, inner, t, seed=31):
    gen = torch.Generator().manual_seed(seed)
    return [v.cuda() for v in (normal(gen, rows, width, dtype=t), normal(gen, inner, width, scale=width ** -0.5, dtype=t),
                               normal(gen, inner, dtype=t), normal(gen, width, inner, scale=inner ** -0.5, dtype=t),
                               normal(gen, width, dtype=t), normal(gen, width, dtype=t), normal(gen, rows, width, dtype=t))]


@pytest.mark.parametrize("rows,width,inner,dtype", [(3, 256, 520, "bf16"), (200, 384, 1000, "fp16"),
                                                    (600, 512, 1024, "bf16"), (90, 130, 77, "fp32")])
def test_the_same_call_gives_the_same_bits(rows, width, inner, dtype):
    args = _layer_inputs(rows, width, inner, DTYPES[dtype])
    note("repeat", rows, width, inner, dtype)
    first = _layer(*args)
    for _ in range(3):
        for a, b in zip(first, _layer(*args)):
            assert torch.equal(a, b)


@pytest.mark.parametrize("rows,width,inner,dtype", [(3, 256, 520, "bf16"), (600, 512, 1024, "bf16"),
                                                    (90, 130, 77, "fp32")])
def test_graph_replays(rows, width, inner, dtype):
    args = _layer_inputs(rows, width, inner, DTYPES[dtype])
    note("graph", rows, width, inner, dtype)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        _layer(*args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _layer(*args)
    gen = torch.Generator().manual_seed(32)
    for replay in range(4):
        args[0].copy_(normal(gen, rows, width, dtype=args[0].dtype))
        args[-1].copy_(normal(gen, rows, width, dtype=args[0].dtype))
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        for a, b in zip(got, _layer(*args)):
            assert torch.equal(a, b), f"replay {replay}"


def test_on_another_stream():
    args = _layer_inputs(300, 512, 768, torch.bfloat16)
    want = _layer(*args)
    torch.cuda.synchronize()
    note("another stream")
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream):
        y, mean, rstd = M.layer_norm_tensors(args[0], args[4], args[5], return_stats=True, stream=stream)
        h, z = M.linear_tensors(args[0], args[1], args[2], None, "gelu", return_preact=True, stream=stream)
        got = M.linear_backward_tensors(h, args[0], args[1], z, "gelu", stream=stream)
        back = M.layer_norm_backward_tensors(args[6], args[0], mean, rstd, args[4], stream=stream)
        side.synchronize()
        assert torch.equal(y, M.layer_norm_tensors(args[0], args[4], args[5]))
        for a, b in zip(got, M.linear_backward_tensors(h, args[0], args[1], z, "gelu")):
            assert torch.equal(a, b)
        for a, b in zip(back, M.layer_norm_backward_tensors(args[6], args[0], mean, rstd, args[4])):
            assert torch.equal(a, b)
    with torch.cuda.stream(side):
        side.wait_stream(torch.cuda.default_stream())
        got = _layer(*args)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
