"""The gated feed-forward block's and the 8-bit products' checks of arguments, on the CPU: nothing here reaches a GPU call."""

import ctypes

import pytest
import torch

import feedforward_oracle as F
import operator_oracle as O
from allreduce_emulated_peer_amd import mscl as M

A = 0x100000  # fake addresses: never dereferenced (validation fails, or there is nothing to do)
STEP = 0x1000000

GATED = ("x", "x_stride", "gate_w", "gate_w_stride", "up_w", "up_w_stride", "gate_bias", "up_bias", "y", "y_stride",
         "gate", "gate_stride", "up", "up_stride", "rows", "in_features", "out_features", "dtype", "activation")
GATED_BACKWARD = ("dy", "dy_stride", "x", "x_stride", "gate_w", "gate_w_stride", "up_w", "up_w_stride", "gate", "gate_stride",
                  "up", "up_stride", "dx", "dx_stride", "dgate_w", "dgate_w_stride", "dup_w", "dup_w_stride", "dgate_bias",
                  "dup_bias", "rows", "in_features", "out_features", "dtype", "activation")
QUANTIZE = ("x", "x_stride", "q", "q_stride", "scale", "rows", "width", "dtype")
INT8 = ("x", "x_stride", "x_scale", "w", "w_stride", "w_scale", "bias", "residual", "residual_stride", "y", "y_stride",
        "rows", "in_features", "out_features", "dtype", "activation")
GATED_INT8 = ("x", "x_stride", "x_scale", "gate_w", "gate_w_stride", "gate_scale", "up_w", "up_w_stride", "up_scale",
              "gate_bias", "up_bias", "y", "y_stride", "rows", "in_features", "out_features", "dtype", "activation")

SIZES = dict(rows=8, in_features=16, out_features=24, activation=M.ACT_SILU)
INNER, OUTER = ("x", "gate_w", "up_w", "w", "dx", "dgate_w", "dup_w"), ("y", "gate", "up", "dy", "residual")
STRIDES = {**{n + "_stride": 16 for n in INNER}, **{n + "_stride": 24 for n in OUTER}}
FORMS = {
    "gated_linear": (M.GATED_LINEAR, GATED, SIZES),
    "gated_linear_backward": (M.GATED_LINEAR_BACKWARD, GATED_BACKWARD, SIZES),
    "quantize": (M.QUANTIZE, QUANTIZE, dict(rows=8, width=16, q_stride=16)),
    "linear_quantized": (M.LINEAR_QUANTIZED, INT8, SIZES),
    "gated_linear_quantized": (M.GATED_LINEAR_QUANTIZED, GATED_INT8, SIZES),
}
PRODUCTS = [op for op in FORMS if op != "quantize"]
NOT_POINTERS = {"rows", "in_features", "out_features", "width", "dtype", "activation"}
BYTES = {("quantize", "q"): 1, **{(op, n): 1 for op in ("linear_quantized", "gated_linear_quantized") for n in ("x", "w", "gate_w", "up_w")}}


def is_pointer(name):
    return name not in NOT_POINTERS and not name.endswith("_stride")


def record(op, **change):
    form, names, values = FORMS[op]
    values = {**STRIDES, **{n: A + i * STEP for i, n in enumerate(names) if is_pointer(n)}, "dtype": M.BFLOAT16, **values, **change}
    return form.pack(*[values[name] for name in names])


def call(op, space=0, size=0, **change):
    """(status, text) of an entry point on a valid call of fake addresses with `change` made to it."""
    lib = M.load()
    if op == "quantize":
        status = lib.mscl_quantize(record(op, **change), None)
    else:
        status = getattr(lib, "mscl_" + op)(record(op, **change), space or None, size, None)
    return status, M.last_error_string()


def workspace(op, **change):
    need = ctypes.c_size_t()
    status = getattr(M.load(), f"mscl_{op}_workspace")(record(op, **change), ctypes.byref(need))
    return status, need.value


@pytest.mark.parametrize("op", FORMS)
def test_null_record(op):
    lib = M.load()
    if op == "quantize":
        assert lib.mscl_quantize(None, None) == M.ERR_INVALID_ARGUMENT
        return
    assert getattr(lib, "mscl_" + op)(None, None, 0, None) == M.ERR_INVALID_ARGUMENT
    size = ctypes.c_size_t()
    query = getattr(lib, f"mscl_{op}_workspace")
    assert query(None, ctypes.byref(size)) == M.ERR_INVALID_ARGUMENT
    assert query(record(op), None) == M.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("op,names", [
    ("gated_linear", ("x", "gate_w", "up_w", "y")), ("gated_linear_backward", ("dy", "x", "gate_w", "up_w", "gate", "up")),
    ("quantize", ("x", "q", "scale")), ("linear_quantized", ("x", "x_scale", "w", "w_scale", "y")),
    ("gated_linear_quantized", ("x", "x_scale", "gate_w", "gate_scale", "up_w", "up_scale", "y"))])
def test_null_pointers(op, names):
    for name in names:
        status, text = call(op, **{name: 0})
        assert status == M.ERR_INVALID_ARGUMENT and name in text and "null" in text


@pytest.mark.parametrize("op", FORMS)
def test_unknown_types(op):
    for dtype in (-1, 3):
        assert call(op, dtype=dtype) == (M.ERR_INVALID_ARGUMENT, "unknown dtype")
    if op != "quantize":
        for act in (-1, 5):
            assert call(op, activation=act) == (M.ERR_INVALID_ARGUMENT, "unknown activation")


@pytest.mark.parametrize("op", FORMS)
def test_short_strides_and_misaligned_pointers(op):
    for i, name in enumerate(FORMS[op][1]):
        if name.endswith("_stride"):
            status, text = call(op, **{name: 15})
            assert status == M.ERR_INVALID_ARGUMENT and "stride" in text and name[:-7] in text, name
        elif is_pointer(name) and BYTES.get((op, name), 2) > 1:
            status, text = call(op, **{name: A + i * STEP + 1})
            assert status == M.ERR_MISALIGNED and name in text


@pytest.mark.parametrize("op", FORMS)
@pytest.mark.parametrize("size", [2 ** 31, 2 ** 61, 2 ** 64 - 1])
def test_sizes_that_are_too_large(op, size):
    big = {n: 2 ** 61 for n in FORMS[op][1] if n.endswith("_stride")}
    for name in ("rows", "in_features", "out_features", "width"):
        if name in FORMS[op][1] and not (name == "width" and size == 2 ** 31):
            assert call(op, **{name: size}, **big)[0] == M.ERR_INVALID_ARGUMENT


def test_integer_sums_that_could_overflow_are_refused():
    for op in ("linear_quantized", "gated_linear_quantized"):
        strides = {n: 1 << 18 for n in FORMS[op][1] if n.endswith("_stride") and n[:-7] in INNER}
        status, text = call(op, in_features=131072, **strides)
        assert status == M.ERR_INVALID_ARGUMENT and "131071" in text
        assert workspace(op, in_features=131071, **strides)[0] == M.SUCCESS


@pytest.mark.parametrize("op,out,other", [
    ("gated_linear", "y", "x"), ("gated_linear", "y", "up_w"), ("gated_linear", "gate", "up"), ("gated_linear", "up", "y"),
    ("gated_linear", "gate", "gate_bias"), ("gated_linear_backward", "dx", "dy"), ("gated_linear_backward", "dx", "x"),
    ("gated_linear_backward", "dgate_w", "gate_w"), ("gated_linear_backward", "dup_w", "dgate_w"),
    ("gated_linear_backward", "dup_bias", "dgate_bias"), ("gated_linear_backward", "dx", "up"), ("quantize", "q", "x"),
    ("quantize", "scale", "x"), ("quantize", "scale", "q"), ("linear_quantized", "y", "x"), ("linear_quantized", "y", "w_scale"),
    ("gated_linear_quantized", "y", "up_w"), ("gated_linear_quantized", "y", "x_scale")])
def test_overlaps(op, out, other):
    at = A + FORMS[op][1].index(other) * STEP
    status, text = call(op, **{out: at})
    assert status == M.ERR_INVALID_ARGUMENT and "overlap" in text and out in text and other in text


def test_in_place_needs_the_same_matrix():
    at = A + INT8.index("residual") * STEP
    for change in ({"y": at + 32}, {"y": at, "y_stride": 40}):
        status, text = call("linear_quantized", **change)
        assert status == M.ERR_INVALID_ARGUMENT and "overlap" in text
    assert workspace("linear_quantized", y=at)[0] == M.SUCCESS


def test_both_halves_of_one_weight_are_taken():
    at = A + GATED.index("gate_w") * STEP
    assert workspace("gated_linear", up_w=at + 24 * 16 * 2)[0] == M.SUCCESS
    assert workspace("gated_linear", up_w=at)[0] == M.SUCCESS  # read only: even the same
    # the gradients may be halves of one matrix too, and interleave
    at = A + GATED_BACKWARD.index("dgate_w") * STEP
    assert workspace("gated_linear_backward", dup_w=at + 24 * 16 * 2)[0] == M.SUCCESS
    assert workspace("gated_linear_backward", dgate_w_stride=32, dup_w_stride=32, dup_w=at + 32)[0] == M.SUCCESS


@pytest.mark.parametrize("op", ["gated_linear_backward", "linear_quantized"])
def test_a_workspace_that_is_too_small_or_in_the_way_is_refused(op):
    # 32 rows of a long k: split over workgroups
    change = {} if op == "gated_linear_backward" else dict(rows=32, in_features=65536, x_stride=65536, w_stride=65536)
    status, need = workspace(op, **change)
    assert status == M.SUCCESS and need > 0
    status, text = call(op, A * 4096, need - 1, **change)
    assert status == M.ERR_INVALID_ARGUMENT and str(need) in text
    assert call(op, 0, need, **change)[0] == M.ERR_INVALID_ARGUMENT
    assert call(op, A * 4096 + 8, need, **change)[0] == M.ERR_MISALIGNED
    out = "dx" if op == "gated_linear_backward" else "y"
    status, text = call(op, A + FORMS[op][1].index(out) * STEP, need, **change)
    assert status == M.ERR_INVALID_ARGUMENT and "workspace" in text and "overlap" in text


def test_nothing_to_do():
    for op in ("gated_linear", "linear_quantized", "gated_linear_quantized"):
        assert call(op, rows=0)[0] == M.SUCCESS
        assert call(op, out_features=0)[0] == M.SUCCESS
    none = dict(dgate_w=0, dup_w=0, dgate_bias=0, dup_bias=0)
    assert call("gated_linear_backward", A << 20, 1 << 30, dx=0, **none)[0] == M.SUCCESS
    assert call("gated_linear_backward", A << 20, 1 << 30, rows=0, **none)[0] == M.SUCCESS
    assert call("quantize", rows=0)[0] == M.SUCCESS
    assert call("quantize", width=0)[0] == M.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("m", [1, 16, 32, 33, 200, 700])
def test_no_copy_of_weights_that_few_rows_use(m):
    k, n = 8192, 16384
    strides = {s: k + 3 for s in ("gate_w_stride", "up_w_stride", "w_stride")}
    far = {name: A + i * (1 << 38) for i, name in enumerate(GATED) if is_pointer(name)}
    sizes = dict(rows=m, in_features=k, out_features=n, x_stride=k, y_stride=n, gate_stride=n, up_stride=n)
    status, need = workspace("gated_linear", **{**far, **sizes, **strides})
    assert status == M.SUCCESS and need < n * k * 2 // 2
    far = {name: A + i * (1 << 38) for i, name in enumerate(INT8) if is_pointer(name)}
    sizes = dict(rows=m, in_features=k, out_features=n, x_stride=k, y_stride=n, residual_stride=n)
    status, need = workspace("linear_quantized", **{**far, **sizes, **strides})
    assert status == M.SUCCESS and need < n * k // 4


@pytest.mark.parametrize("stride", [0, 1, 3, 1 << 40, (1 << 64) - 1])
def test_the_stride_of_a_single_row_changes_nothing(stride):
    one = dict(rows=1, in_features=4096, out_features=512, gate_w_stride=4096, up_w_stride=4096, w_stride=4096, dgate_w_stride=4096,
               dup_w_stride=4096)
    rows = {n + "_stride": stride for n in ("x", "y", "gate", "up", "dy", "dx", "residual")}
    usual = {**{n + "_stride": 512 for n in OUTER}, "x_stride": 4096, "dx_stride": 4096}
    for op in PRODUCTS:
        assert workspace(op, **{**one, **rows}) == workspace(op, **{**one, **usual})


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_tensor_forms_refuse_before_any_gpu_call():
    x, w, b = _t(4, 8), _t(6, 8), _t(6)
    for args, kwargs, match in [
        ((x.int(), w, w), {}, "unsupported dtype"),
        ((x, w.half(), w), {}, "gate_weight must be of"),
        ((x, w, w.half()), {}, "up_weight must be of"),
        ((x, w[0], w), {}, "must be matrices"),
        ((x, w, w[:5]), {}, "same shape"),
        ((x, w, w, b.half()), {}, "gate_bias must be of"),
        ((x, w, w, None, b[:5]), {}, "vector of 6"),
        ((x, w, w), {"activation": "swish"}, "unknown activation"),
        ((x, w, w), {}, "on a GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            M.gated_linear_tensors(*args, **kwargs)
    dy = _t(4, 6)
    for args, match in [((dy, x.half(), w, w, dy, dy), "x must be of"), ((dy, x, w, w, dy.half(), dy), "gate must be of"),
                        ((dy, x, w, w, dy, dy), "on a GPU")]:
        with pytest.raises(ValueError, match=match):
            M.gated_linear_backward_tensors(*args)
    for t, match in [(x.int(), "unsupported dtype"), (_t(4, 0), "at least 1"), (_t(), "at least 1"), (x, "on a GPU")]:
        with pytest.raises(ValueError, match=match):
            M.quantize_tensors(t)
    q, p, s, c = _t(4, 8, dtype=torch.int8), _t(6, 8, dtype=torch.int8), _t(4), _t(6)
    for args, kwargs, match in [
        ((x, s, p, c), {}, "x must be of torch.int8"),
        ((q, s, w, c), {}, "weight must be of torch.int8"),
        ((q, s[:3], p, c), {}, "x's scales"),
        ((q, s, p, c.double()), {}, "weight's scales"),
        ((q, s, p, c), {"dtype": torch.int8}, "unsupported dtype"),
        ((q, s, p, c, b), {}, "bias must be of torch.bfloat16"),
        ((q, s, p, c), {"residual": _t(4, 6), "dtype": torch.float16}, "residual must be of torch.float16"),
        ((q, s, p, c), {"activation": "swish"}, "unknown activation"),
        ((q, s, p, c), {}, "on a GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            M.linear_quantized_tensors(*args, **kwargs)
    for args, kwargs, match in [
        ((q, s, p, c, p[:5], c[:5]), {}, "same shape"),
        ((q, s, p, c, p, c[:5]), {}, "up_weight's scales"),
        ((q, s, p, c, w, c), {}, "up_weight must be of torch.int8"),
        ((q, s, p, c, p, c, b), {}, "gate_bias must be of"),
        ((q, s, p, c, p, c), {}, "on a GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            M.gated_linear_quantized_tensors(*args, **kwargs)


# ---------------------------------------------------------------- the oracle itself

@pytest.mark.parametrize("act", sorted(M.ACTIVATION_CODES))
def test_oracle_gradients_against_differences(act):
    torch.manual_seed(5)
    x, wg, wu = torch.randn(5, 7).double(), torch.randn(6, 7).double(), torch.randn(6, 7).double()
    bg, bu, dy = torch.randn(6).double(), torch.randn(6).double(), torch.randn(5, 6).double()

    def loss(x, wg, wu, bg, bu):
        return float((O.activate(x @ wg.t() + bg, act) * (x @ wu.t() + bu) * dy).sum())

    grads = F.gated_linear_backward(dy, x, wg, wu, x @ wg.t() + bg, x @ wu.t() + bu, act)
    h = 1e-6
    for (grad, _), at in zip(grads, range(5)):
        v = [x, wg, wu, bg, bu]
        d = torch.randn_like(v[at])
        lo, hi = list(v), list(v)
        lo[at], hi[at] = v[at] - h * d, v[at] + h * d
        assert abs((loss(*hi) - loss(*lo)) / (2 * h) - float((grad * d).sum())) < 1e-5


def test_oracle_of_quantize():
    x = torch.tensor([[0.0, 0.0, 0.0], [127.0, -3.5, 2.5], [2.0 ** -101, 0.0, -2.0 ** -104], [1.0, -2.0, 0.5]])
    q, scale = F.quantize(x)
    assert q.tolist() == [[0, 0, 0], [127, -4, 2], [64, 0, -8], [64, -127, 32]]  # 63.5 and -7.9..: ties to even
    assert torch.equal(scale, torch.tensor([2.0 ** -100, 127.0, 2.0 ** -100, 2.0]) / 127)
    big = torch.randn(64, 300) * 10
    q, scale = F.quantize(big)
    assert float((q * scale[:, None] - big).abs().max() / scale.max()) <= 0.5001 and int(q.abs().max()) == 127
