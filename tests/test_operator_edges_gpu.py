"""The operators on the GPU at the edges of their kernels' ranges, against their formulas in 64 bits."""

import math
import os
import subprocess
import sys

import pytest
import torch

import operator_oracle as O
from allreduce_emulated_peer_amd import mscl as M

pytestmark = pytest.mark.gpu
DTYPES = O.DTYPES


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


def note(*what):
    print("[gpu-case]", *what, file=sys.stderr, flush=True)


def normal(gen, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(shape, generator=gen) * scale).to(dtype)


def guarded(t, rows=256):
    """t on the GPU with `rows` rows of NaN behind its last one."""
    room = torch.full((t.shape[0] + rows, t.shape[1]), math.nan, dtype=t.dtype, device="cuda")
    room[:t.shape[0]] = t.cuda()
    return room[:t.shape[0]]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("rows", [193, 320, 321, 337, 351, 352])
def test_large_weight_gradient_whose_last_block_has_few_rows(dtype, rows):
    """256 x 256 tiles, 64 rows at a time: rows of the last block that do not exist count as 0, whatever lies there."""
    gen = torch.Generator().manual_seed(50)
    t, k, n = DTYPES[dtype], 4096, 2056
    dy, x = normal(gen, rows, n, dtype=t), normal(gen, rows, k, dtype=t)
    w, z = normal(gen, n, k, scale=k ** -0.5, dtype=t), normal(gen, rows, n, scale=1.5, dtype=t)
    for act in ("none", "silu"):
        note("large weight gradient", dtype, rows, act)
        got = M.linear_backward_tensors(guarded(dy), guarded(x), guarded(w), guarded(z), act)
        want = O.linear_backward(dy.cuda(), x.cuda(), w.cuda(), z.cuda(), act)
        for g, e, name in zip(got, want, ("dx", "dw", "db")):
            O.assert_within(g, e, f"{name} {act}")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,k,n", [(2049, 256, 4097), (2052, 328, 3848)])
def test_large_product_whose_last_tiles_have_few_rows(dtype, m, k, n):
    """Tile rows that do not exist are not read: what lies there is NaN, and reaches no result."""
    gen = torch.Generator().manual_seed(51)
    t = DTYPES[dtype]
    x, w = normal(gen, m, k, dtype=t), normal(gen, n, k, scale=k ** -0.5, dtype=t)
    note("large product, few rows in its last tiles", dtype, m, k, n)
    O.assert_within(M.linear_tensors(guarded(x), guarded(w)), O.linear(x.cuda(), w.cuda(), None, None, "none")[0], "y")


# x 2^low times random mantissas, w 2^high: ordinary results of operands at the bottom of binary32's range, where a
# value's smaller parts leave bfloat16's range; and at its top, where the scaled parts do.
@pytest.mark.parametrize("m,k,n", [(1, 300, 70), (32, 130, 90), (33, 130, 90), (300, 1030, 200)])
@pytest.mark.parametrize("low,high", [(-111, 100), (-115, 100), (-120, 100), (-126, 100), (-135, 100), (-115, 0), (-126, 20),
                                      (105, -100), (125, -120)])
def test_binary32_products_at_the_ends_of_the_range(m, k, n, low, high):
    gen = torch.Generator().manual_seed(52)

    def values(size, *shape):
        sign = torch.randint(0, 2, shape, generator=gen) * 2.0 - 1
        return ((1 + torch.rand(shape, generator=gen, dtype=torch.float64)) * sign * 2.0 ** size).float()

    x, w, dy = values(low, m, k), values(high, n, k), values(low, m, n)
    note("binary32 ends", m, k, n, low, high)
    c = [v.cuda() for v in (x, w, dy)]
    O.assert_within(M.linear_tensors(c[0], c[1]), O.linear(c[0], c[1], None, None, "none")[0], "y")
    dx, _, _ = M.linear_backward_tensors(c[2], c[0], c[1], need_dw=False, need_db=False)
    O.assert_within(dx, O.linear_backward(c[2], c[0], c[1], None, "none")[0], "dx")
    xw = values(high, m, k).cuda()  # dw of tiny dy and large x
    _, dw, _ = M.linear_backward_tensors(c[2], xw, c[1], need_dx=False, need_db=False)
    O.assert_within(dw, O.linear_backward(c[2], xw, c[1], None, "none")[1], "dw")
    assert bool((dw != 0).all())


def test_binary32_products_of_the_largest_smaller_parts():
    """One product each, of values whose bfloat16 parts leave out most: the stated bound, and the sums' and the result's roundings."""
    v = torch.tensor([1 + 2.0 ** -8 - 2.0 ** -17 + i * 2.0 ** -23 for i in range(-40, 41)])
    note("binary32 products of single values")
    y = M.linear_tensors(v.view(-1, 1).cuda(), v.view(-1, 1).cuda()).cpu().double()
    exact = v.double().view(-1, 1) @ v.double().view(1, -1)
    assert float(((y - exact) / exact).abs().max()) <= 2.0 ** -24 + 2.0 ** -34 + 2 * O.U * (1 + 2.0 ** -6)


# A vocabulary's outputs, more than 128 tiles of 256 columns: from one token to more rows than a tile has.
@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("m", [1, 16, 17, 32, 33, 200, 513, 800])
@pytest.mark.parametrize("n,offset", [(32776, 0), (32771, 3), (65536, 0), (65400, 3)])
def test_many_outputs_of_few_rows(dtype, m, n, offset):
    gen = torch.Generator().manual_seed(53)
    t, k = DTYPES[dtype], 264
    x, w = normal(gen, m, k, dtype=t), normal(gen, n, k, scale=k ** -0.5, dtype=t)
    b, r = normal(gen, n, dtype=t), normal(gen, m, n, dtype=t)
    room = torch.full((n, k + offset + 1), math.nan, dtype=t, device="cuda")
    view = room[:, offset:offset + k] if offset else w.cuda()
    view.copy_(w)
    note("many outputs", dtype, m, n, offset)
    y = M.linear_tensors(x.cuda(), view, b.cuda(), r.cuda(), "silu")
    O.assert_within(y, O.linear(x.cuda(), w.cuda(), b.cuda(), r.cuda(), "silu")[0], "y")
    # the mirrored product: many rows, few outputs
    z = M.linear_tensors(view, x.cuda())
    O.assert_within(z, O.linear(w.cuda(), x.cuda(), None, None, "none")[0], "many rows")


@pytest.mark.parametrize("stride", [1, 3, 1 << 40])
def test_the_stride_of_a_single_row_is_ignored(stride):
    gen = torch.Generator().manual_seed(54)
    t = torch.bfloat16
    note("stride of a single row", stride)
    dy, w, x = normal(gen, 1, 264, dtype=t).cuda(), normal(gen, 264, 32776, dtype=t).cuda(), normal(gen, 1, 32776, dtype=t).cuda()
    got = M.linear_backward_tensors(torch.as_strided(dy, (1, 264), (stride, 1)), torch.as_strided(x, (1, 32776), (stride, 1)), w)
    for g, e, name in zip(got, O.linear_backward(dy, x, w, None, "none"), ("dx", "dw", "db")):
        O.assert_within(g, e, name)
    many, one = normal(gen, 66000, 264, dtype=t).cuda(), normal(gen, 1, 264, dtype=t).cuda()
    y = M.linear_tensors(many, torch.as_strided(one, (1, 264), (stride, 1)))
    O.assert_within(y, O.linear(many, one, None, None, "none")[0], "y")


def in_64_bits(z, act):
    """An activation and its slope; gelu_tanh by (1 + tanh u) / 2 = sigmoid(2 u), which does not cancel in the tail."""
    if act != "gelu_tanh":
        return O.activate(z, act), O.slope(z, act)
    a = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)
    da = 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    return z * torch.sigmoid(a), torch.sigmoid(a) + z * torch.sigmoid(a) * torch.sigmoid(-a) * da


def relative_error(z, act, fast):
    """Of an activation (and of its slope's terms): some ten operations, exp's argument, and the fast forms' tail."""
    if act == "gelu_tanh":
        return (10 + 6 * (2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)).abs()) * O.U
    if act == "silu":
        return (10 + 2 * z.abs()) * O.U
    return (10 + 2 * z * z) * O.U + (1.2e-5 if fast else 0.0)


def slope_terms(z, act):
    """The sizes of what the slope is a sum of, and what 1 - (a value near 1) is off by in it."""
    if act == "gelu":
        return 0.5 * torch.special.erfc(-z * math.sqrt(0.5)) + z.abs() * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi), 0.0
    if act == "silu":
        s = torch.sigmoid(z)
        return s + (z * s * (1 - s)).abs(), 2 * O.U * z.abs() * s
    du = math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z * z)
    s = torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
    return s + (2 * z * s * (1 - s) * du).abs(), 4 * O.U * (z * s * du).abs()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu"])
def test_activations_keep_their_relative_accuracy(dtype, act):
    """Down the negative tail, where results are small, as elsewhere: to the rounding of the result and of exp's argument."""
    t = DTYPES[dtype]
    z = torch.cat([torch.linspace(-12, -4, 2048), torch.linspace(-4, 4, 1024), torch.linspace(4, 12, 512),
                   torch.linspace(-0.01, 0.01, 512)]).to(t).reshape(64, 64)
    eye, ones = torch.eye(64, dtype=t).cuda(), torch.ones(64, 64, dtype=t).cuda()
    note("relative accuracy", dtype, act)
    y, kept = M.linear_tensors(z.cuda(), eye, activation=act, return_preact=True)
    assert torch.equal(kept.cpu(), z)  # the product with the identity is exact
    v = z.double()
    rel = relative_error(v, act, dtype != "fp32")
    least = torch.finfo(torch.float32).smallest_normal  # a sigmoid or tail below it may be 0
    floor = 16 * least  # times z
    want, steep = in_64_bits(v, act)
    O.assert_within(y, (want, O.rounded(want, rel * want.abs() + floor, t)), f"{act}")
    dx, _, _ = M.linear_backward_tensors(ones, eye, eye, z.cuda(), act)
    terms, near = slope_terms(v, act)
    if act == "gelu_tanh":  # the slope has 2 z u' times the sigmoid
        floor = least * (1 + 2 * math.sqrt(2 / math.pi) * v.abs() * (1 + 3 * 0.044715 * v * v))
    O.assert_within(dx, (steep, O.rounded(steep, rel * terms + near + floor, t)), f"slope of {act}")


CODES = {"bf16": M.BFLOAT16, "fp16": M.FLOAT16, "fp32": M.FLOAT32}


@pytest.mark.parametrize("dtype,m,k,n", [("bf16", 20, 72, 90), ("fp32", 70, 130, 45), ("fp16", 300, 256, 264),
                                         ("bf16", 2100, 264, 4100)])
def test_outputs_as_column_blocks_of_one_matrix(dtype, m, k, n):
    """Through the C ABI: residual, y and preact side by side; dy, x and dx side by side; a norm's y beside its x."""
    gen = torch.Generator().manual_seed(55)
    t, lib, stream = DTYPES[dtype], M.load(), torch.cuda.current_stream().cuda_stream
    x, w = normal(gen, m, k, dtype=t).cuda(), normal(gen, n, k, scale=k ** -0.5, dtype=t).cuda()
    r, b = normal(gen, m, n, dtype=t).cuda(), normal(gen, n, dtype=t).cuda()
    note("column blocks", dtype, m, k, n)

    def run(query, entry, call):
        space, size = M._workspace(query, call, x)
        M._check(entry(call, M._address(space), size, stream), "column blocks")
        torch.cuda.synchronize()

    wide = 3 * n + 5
    room = torch.full((m, wide), 77.0, dtype=t, device="cuda")
    room[:, 1:1 + n] = r
    y, z = room[:, 2 + n:2 + 2 * n], room[:, 3 + 2 * n:3 + 3 * n]
    run(lib.mscl_linear_workspace, lib.mscl_linear,
        M.LINEAR.pack(x.data_ptr(), k, w.data_ptr(), k, b.data_ptr(), room[:, 1:].data_ptr(), wide, y.data_ptr(), wide,
                      z.data_ptr(), wide, m, k, n, CODES[dtype], M.ACT_SILU))
    want = O.linear(x, w, b, r, "silu")
    O.assert_within(y, want[0], "y")
    O.assert_within(z, want[1], "preact")
    assert torch.equal(room[:, 1:1 + n], r)
    for column in (0, 1 + n, 2 + 2 * n, 3 + 3 * n, 4 + 3 * n):
        assert bool((room[:, column] == 77).all())

    wide = n + 2 * k + 4
    room = torch.full((m, wide), 55.0, dtype=t, device="cuda")
    dy = room[:, 1:1 + n].copy_(r)
    xs = room[:, 2 + n:2 + n + k].copy_(x)
    dx = room[:, 3 + n + k:3 + n + 2 * k]
    dw, db = torch.empty(n, k, dtype=t, device="cuda"), torch.empty(n, dtype=t, device="cuda")
    run(lib.mscl_linear_backward_workspace, lib.mscl_linear_backward,
        M.LINEAR_BACKWARD.pack(dy.data_ptr(), wide, xs.data_ptr(), wide, w.data_ptr(), k, 0, 0, dx.data_ptr(), wide,
                               dw.data_ptr(), k, db.data_ptr(), m, k, n, CODES[dtype], M.ACT_NONE))
    for g, e, name in zip((dx, dw, db), O.linear_backward(r, x, w, None, "none"), ("dx", "dw", "db")):
        O.assert_within(g, e, name)
    assert torch.equal(dy, r) and torch.equal(xs, x)
    for column in (0, 1 + n, 2 + n + k, 3 + n + 2 * k):
        assert bool((room[:, column] == 55).all())

    wide = 2 * k + 3
    room = torch.full((m, wide), 33.0, dtype=t, device="cuda")
    xs, y = room[:, 1:1 + k].copy_(x), room[:, 2 + k:2 + 2 * k]
    M._check(lib.mscl_layer_norm(M.LAYER_NORM.pack(xs.data_ptr(), wide, 0, 0, y.data_ptr(), wide, 0, 0, m, k, 1e-5,
                                                   CODES[dtype], CODES[dtype]), stream), "norm")
    O.assert_within(y, O.layer_norm(x, None, None, 1e-5)[0], "norm")
    assert torch.equal(xs, x)
    for column in (0, 1 + k, 2 + 2 * k):
        assert bool((room[:, column] == 33).all())


def test_a_gradient_is_not_lost_unseen():
    """Autograd does not reach through the operators: a backward pass that would need it raises."""
    gen = torch.Generator().manual_seed(56)
    x, w, b = normal(gen, 6, 40).cuda(), normal(gen, 24, 40).cuda(), normal(gen, 24).cuda()
    g, head = normal(gen, 24).cuda(), normal(gen, 24).cuda().requires_grad_()
    note("autograd")
    y, z = M.linear_tensors(x, w, b, None, "gelu", return_preact=True)
    n, mean, rstd = M.layer_norm_tensors(y, g, return_stats=True)
    assert not any(t.requires_grad for t in (y, z, n, mean, rstd))
    side = torch.cuda.Stream()
    for stream in (None, side):
        for which in range(4):
            args = [t.clone().requires_grad_(i == which) for i, t in enumerate((x, w, b, y))]
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            got = M.linear_tensors(*args, "gelu", return_preact=True, stream=stream)
            with torch.no_grad():
                want = M.linear_tensors(*args, "gelu", return_preact=True)
            torch.cuda.synchronize()
            for a, e in zip(got, want):
                assert torch.equal(a, e) and a.requires_grad and not e.requires_grad
            for loss in ((got[0] * head).sum(), (got[1] * head).sum()):
                with pytest.raises(RuntimeError, match="linear_backward_tensors"):
                    loss.backward()
        for which in range(3):
            args = [t.clone().requires_grad_(i == which) for i, t in enumerate((y, g, b))]
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            got = M.layer_norm_tensors(*args, return_stats=True, stream=stream)
            with torch.no_grad():
                want = M.layer_norm_tensors(*args, return_stats=True)
            torch.cuda.synchronize()
            for a, e in zip(got, want):
                assert torch.equal(a, e) and a.requires_grad and not e.requires_grad
            with pytest.raises(RuntimeError, match="layer_norm_backward_tensors"):
                (got[0] * head).sum().backward()
    # what only a head on top needs goes through, as does a result that is changed in place
    h = M.linear_tensors(x.clone().requires_grad_(), w)
    h.mul_(2)
    head.grad = None  # the passes that raised had reached it
    (h.detach() * head).sum().backward()
    assert torch.allclose(head.grad, h.detach().sum(0))
    # the gradients' functions run by hand on parameters, outside of any graph
    p = w.clone().requires_grad_()
    for t in M.linear_backward_tensors(torch.ones_like(y), x, p, z, "gelu"):
        assert not t.requires_grad


@pytest.mark.parametrize("dtype", DTYPES)
def test_copies_that_lie_equally_give_the_same_bits(dtype):
    """The order of sums may go by the pointers' place between 16-byte boundaries, and by nothing else of an address."""
    gen = torch.Generator().manual_seed(57)
    t, rows, width, out = DTYPES[dtype], 40, 1003, 130
    x, w, dy = normal(gen, rows, width, dtype=t), normal(gen, out, width, dtype=t), normal(gen, rows, out, dtype=t)
    step = 16 // x.element_size()
    note("equally placed copies", dtype)
    for shift in range(0, step, 3):
        seen = None
        for far in (0, 5, 64):  # 16-byte steps
            def at(v):
                room = torch.full((shift + step * far + v.numel() + step,), math.nan, dtype=t, device="cuda")
                view = room[shift + step * far:shift + step * far + v.numel()].view(v.shape)
                return view.copy_(v)

            a = [at(v) for v in (x, w, dy)]
            y, mean, rstd = M.layer_norm_tensors(a[0], return_stats=True)
            got = [y, mean, rstd, M.linear_tensors(a[0], a[1]), *M.linear_backward_tensors(a[2], a[0], a[1]),
                   *M.layer_norm_backward_tensors(a[0], a[0], mean, rstd)]
            seen = seen or got
            for g, e in zip(got, seen):
                assert torch.equal(g, e)
        for g, e, name in zip(got, O.layer_norm(x, None, None, 1e-5), ("y", "mean", "rstd")):
            O.assert_within(g, e, name)


def large_layer(x, w, b, r, dy, z):
    y, kept = M.linear_tensors(x, w, b, r, "gelu", return_preact=True)
    return (y, kept) + M.linear_backward_tensors(dy, x, w, z, "silu")


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("m,k,n,odd", [(2304, 4096, 4096, False), (2300, 4099, 3907, True)])
def test_graph_replays_of_large_products(dtype, m, k, n, odd):
    """256 x 256 tiles, and operands laid out anew, captured; eager work and synchronizations between the replays."""
    gen = torch.Generator().manual_seed(58)
    t = DTYPES[dtype]
    note("graph of large products", dtype, m, k, n, odd)
    args = [v.cuda() for v in (normal(gen, m, k, dtype=t), normal(gen, n, k, scale=k ** -0.5, dtype=t), normal(gen, n, dtype=t),
                               normal(gen, m, n, dtype=t), normal(gen, m, n, dtype=t), normal(gen, m, n, dtype=t))]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        large_layer(*args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = large_layer(*args)
    for replay in range(4):
        for i in (0, 4):
            args[i].copy_(normal(gen, *args[i].shape, dtype=t))
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        for a, b in zip(got, large_layer(*args)):
            assert torch.equal(a, b), f"replay {replay}"


FIRST_CALL = """
import torch
from allreduce_emulated_peer_amd import mscl as M
x, w = torch.randn(2304, 520, device="cuda").bfloat16(), torch.randn(4099, 520, device="cuda").bfloat16()
dy = torch.randn(2304, 4099, device="cuda").bfloat16()
f = torch.randn(200, 300, device="cuda")
def layer():
    return (M.linear_tensors(x, w), *M.linear_backward_tensors(dy, x, w), M.linear_tensors(f, f),
            *M.linear_backward_tensors(f[:, :200].contiguous(), f, f), *M.layer_norm_tensors(x, return_stats=True))
M.load()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    out = layer()
for _ in range(3):
    x.copy_(torch.randn(2304, 520, device="cuda"))
    graph.replay()
    got = [o.clone() for o in out]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, layer()))
print("replays equal")
"""


def test_the_first_call_of_a_process_can_be_captured():
    """Whatever is looked up or set once for a device is no work on a stream."""
    note("first call captured, in a child process")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    done = subprocess.run([sys.executable, "-c", FIRST_CALL], capture_output=True, text=True, timeout=110, cwd=root)
    assert done.returncode == 0 and done.stdout.strip().endswith("replays equal"), done.stdout + done.stderr


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows,width", [(5, 40), (21, 600), (300, 9000), (2100, 96)])
def test_an_infinite_input_counts_once_in_the_weight_gradient(dtype, rows, width):
    """With finite statistics, as the formula has it: infinite in its column and nowhere else."""
    gen = torch.Generator().manual_seed(59)
    t = DTYPES[dtype]
    x, dy = normal(gen, rows, width, dtype=t), normal(gen, rows, width, dtype=t)
    x[rows - 1, 7], x[rows // 2, 30] = math.inf, -math.inf
    dy[rows - 1, 7], dy[rows // 2, 30] = 2, 3
    mean, rstd = torch.zeros(rows, device="cuda"), torch.ones(rows, device="cuda")
    note("infinite input", dtype, rows, width)
    for need_dx in (True, False):
        _, dw, db = M.layer_norm_backward_tensors(dy.cuda(), x.cuda(), mean, rstd, need_dx=need_dx)
        assert dw[7] == math.inf and dw[30] == -math.inf
        keep = [i for i in range(width) if i not in (7, 30)]
        clean = x.clone()
        clean[rows - 1, 7] = clean[rows // 2, 30] = 0
        _, want_dw, want_db = O.layer_norm_backward(dy, clean, mean.cpu(), rstd.cpu(), None, t)
        O.assert_within(dw.cpu()[keep], (want_dw[0][keep], want_dw[1][keep]), "dw")
        O.assert_within(db, want_db, "db")
