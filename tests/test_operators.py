"""The operators' checks of arguments, on the CPU: nothing here reaches a GPU call."""

import ctypes
import math

import pytest
import torch

import operator_oracle as O
from allreduce_emulated_peer_amd import mscl as M

A = 0x100000  # fake addresses: never dereferenced (validation fails, or there is nothing to do)
STEP = 0x1000000

LINEAR = ("x", "x_stride", "w", "w_stride", "bias", "residual", "residual_stride", "y", "y_stride", "preact",
          "preact_stride", "rows", "in_features", "out_features", "dtype", "activation")
LINEAR_BACKWARD = ("dy", "dy_stride", "x", "x_stride", "w", "w_stride", "preact", "preact_stride", "dx", "dx_stride",
                   "dw", "dw_stride", "dbias", "rows", "in_features", "out_features", "dtype", "activation")
NORM = ("x", "x_stride", "weight", "bias", "y", "y_stride", "mean", "rstd", "rows", "width", "eps", "dtype",
        "param_dtype")
NORM_BACKWARD = ("dy", "dy_stride", "x", "x_stride", "mean", "rstd", "weight", "dx", "dx_stride", "dweight", "dbias",
                 "rows", "width", "dtype", "param_dtype")

FORMS = {
    "linear": (M.LINEAR, LINEAR, dict(rows=8, in_features=16, out_features=24, x_stride=16, w_stride=16,
                                      residual_stride=24, y_stride=24, preact_stride=24, activation=M.ACT_GELU)),
    "linear_backward": (M.LINEAR_BACKWARD, LINEAR_BACKWARD,
                        dict(rows=8, in_features=16, out_features=24, dy_stride=24, x_stride=16, w_stride=16,
                             preact_stride=24, dx_stride=16, dw_stride=16, activation=M.ACT_GELU)),
    "layer_norm": (M.LAYER_NORM, NORM, dict(rows=8, width=16, x_stride=16, y_stride=16, eps=1e-5)),
    "layer_norm_backward": (M.LAYER_NORM_BACKWARD, NORM_BACKWARD,
                            dict(rows=8, width=16, dy_stride=16, x_stride=16, dx_stride=16)),
}
NOT_POINTERS = {"rows", "in_features", "out_features", "width", "eps", "dtype", "param_dtype", "activation"}


def call(op, space=0, size=0, **change):
    """(status, text) of an entry point on a valid call of fake addresses with `change` made to it."""
    form, names, values = FORMS[op]
    values = dict(values)
    for i, name in enumerate(names):
        if name not in NOT_POINTERS and not name.endswith("_stride"):
            values[name] = A + i * STEP
    values.setdefault("dtype", M.BFLOAT16)
    values.setdefault("param_dtype", M.BFLOAT16)
    values.update(change)
    record = form.pack(*[values[name] for name in names])
    lib = M.load()
    if op == "layer_norm":
        status = lib.mscl_layer_norm(record, None)
    else:
        status = getattr(lib, "mscl_" + op)(record, space or None, size, None)
    return status, M.last_error_string()


@pytest.mark.parametrize("op", FORMS)
def test_null_record(op):
    lib = M.load()
    if op == "layer_norm":
        assert lib.mscl_layer_norm(None, None) == M.ERR_INVALID_ARGUMENT
        return
    assert getattr(lib, "mscl_" + op)(None, None, 0, None) == M.ERR_INVALID_ARGUMENT
    size = ctypes.c_size_t()
    query = getattr(lib, f"mscl_{op}_workspace")
    assert query(None, ctypes.byref(size)) == M.ERR_INVALID_ARGUMENT
    assert query(FORMS[op][0].pack(*[0] * len(FORMS[op][1])), None) == M.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("op,names", [("linear", ("x", "w", "y")), ("linear_backward", ("dy", "x", "w", "preact")),
                                      ("layer_norm", ("x", "y")), ("layer_norm_backward", ("dy", "x", "mean", "rstd"))])
def test_null_pointers(op, names):
    for name in names:
        status, text = call(op, **{name: 0})
        assert status == M.ERR_INVALID_ARGUMENT and name in text and "null" in text


@pytest.mark.parametrize("op", FORMS)
@pytest.mark.parametrize("dtype", [-1, 3])
def test_unknown_types(op, dtype):
    assert call(op, dtype=dtype)[0] == M.ERR_INVALID_ARGUMENT
    if "norm" in op:
        assert call(op, param_dtype=dtype)[0] == M.ERR_INVALID_ARGUMENT
        assert call(op, param_dtype=M.FLOAT16)[0] == M.ERR_INVALID_ARGUMENT  # neither the rows' type nor float32
    else:
        for act in (-1, 5):
            assert call(op, activation=act)[0] == M.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("op", FORMS)
def test_short_strides_and_misaligned_pointers(op):
    for name in FORMS[op][1]:
        if name.endswith("_stride"):
            status, text = call(op, **{name: 15})
            assert status == M.ERR_INVALID_ARGUMENT and "stride" in text, name
    for i, name in enumerate(FORMS[op][1]):
        if name not in NOT_POINTERS and not name.endswith("_stride"):
            status, text = call(op, **{name: A + i * STEP + 1})
            assert status == M.ERR_MISALIGNED and name in text


@pytest.mark.parametrize("op", FORMS)
def test_sizes_that_overflow(op):
    rows = [n for n in ("rows", "in_features", "out_features", "width") if n in FORMS[op][1]]
    for name in rows:
        # with strides that follow, so that nothing but the size is wrong
        big = {n: 2 ** 61 for n in FORMS[op][1] if n.endswith("_stride")}
        assert call(op, **{name: 2 ** 61}, **big)[0] == M.ERR_INVALID_ARGUMENT
        assert call(op, **{name: 2 ** 64 - 1}, **big)[0] == M.ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("op,out,other", [
    ("linear", "y", "x"), ("linear", "y", "w"), ("linear", "y", "bias"), ("linear", "preact", "residual"),
    ("linear", "preact", "y"), ("linear_backward", "dx", "dy"), ("linear_backward", "dw", "w"),
    ("linear_backward", "dbias", "dx"), ("linear_backward", "dx", "preact"), ("layer_norm", "y", "weight"),
    ("layer_norm", "mean", "x"), ("layer_norm", "rstd", "mean"), ("layer_norm_backward", "dx", "x"),
    ("layer_norm_backward", "dweight", "dbias"), ("layer_norm_backward", "dbias", "weight")])
def test_overlaps(op, out, other):
    at = A + FORMS[op][1].index(other) * STEP
    status, text = call(op, **{out: at})
    assert status == M.ERR_INVALID_ARGUMENT and "overlap" in text and out in text and other in text


@pytest.mark.parametrize("op,out,other", [("linear", "y", "residual"), ("layer_norm", "y", "x"),
                                          ("layer_norm_backward", "dx", "dy")])
def test_in_place_needs_the_same_matrix(op, out, other):
    at = A + FORMS[op][1].index(other) * STEP
    status, text = call(op, **{out: at + 32})
    assert status == M.ERR_INVALID_ARGUMENT and "overlap" in text
    assert call(op, **{out: at, out + "_stride": 40})[0] == M.ERR_INVALID_ARGUMENT


def test_a_workspace_that_is_too_small_is_refused():
    lib = M.load()
    form, names, values = FORMS["linear_backward"]
    values = {**{n: A + i * STEP for i, n in enumerate(names) if n not in NOT_POINTERS and not n.endswith("_stride")},
              **values, "dtype": M.BFLOAT16}
    record = form.pack(*[values[n] for n in names])
    need = ctypes.c_size_t()
    assert lib.mscl_linear_backward_workspace(record, ctypes.byref(need)) == M.SUCCESS and need.value > 0
    status, text = call("linear_backward", A * 4096, need.value - 1)
    assert status == M.ERR_INVALID_ARGUMENT and str(need.value) in text
    assert call("linear_backward", 0, need.value)[0] == M.ERR_INVALID_ARGUMENT
    assert call("linear_backward", A * 4096 + 8, need.value)[0] == M.ERR_MISALIGNED


def test_a_workspace_over_an_output_is_refused():
    status, text = call("linear_backward", A + LINEAR_BACKWARD.index("dx") * STEP, 1 << 20)
    assert status == M.ERR_INVALID_ARGUMENT and "workspace" in text and "overlap" in text


def test_nothing_to_do():
    assert call("linear", rows=0)[0] == M.SUCCESS
    assert call("linear", out_features=0)[0] == M.SUCCESS
    assert call("layer_norm", rows=0)[0] == M.SUCCESS
    assert call("linear_backward", dx=0, dw=0, dbias=0)[0] == M.SUCCESS
    assert call("linear_backward", rows=0, dw=0, dbias=0)[0] == M.SUCCESS
    assert call("layer_norm_backward", rows=0, dweight=0, dbias=0)[0] == M.SUCCESS
    assert call("layer_norm_backward", dx=0, dweight=0, dbias=0)[0] == M.SUCCESS


def test_norm_values():
    assert call("layer_norm", width=0)[0] == M.ERR_INVALID_ARGUMENT
    assert call("layer_norm_backward", width=0)[0] == M.ERR_INVALID_ARGUMENT
    assert call("layer_norm", eps=-1e-9)[0] == M.ERR_INVALID_ARGUMENT
    assert call("layer_norm", eps=math.nan)[0] == M.ERR_INVALID_ARGUMENT


def _t(*shape, dtype=torch.float32):
    return torch.zeros(shape, dtype=dtype)


def test_tensor_forms_refuse_before_any_gpu_call():
    x, w = _t(4, 8), _t(6, 8)
    for args, kwargs, match in [
        ((x.int(), w), {}, "unsupported dtype"),
        ((x, w.half()), {}, "weight must be of"),
        ((x, w[0]), {}, "must be a matrix"),
        ((x, w), {"activation": "swish"}, "unknown activation"),
        ((x, w), {}, "on a GPU"),
    ]:
        with pytest.raises(ValueError, match=match):
            M.linear_tensors(*args, **kwargs)
    with pytest.raises(ValueError, match="needs preact"):
        M.linear_backward_tensors(_t(4, 6), x, w, activation="gelu")
    with pytest.raises(ValueError, match="on a GPU"):
        M.linear_backward_tensors(_t(4, 6), x, w)
    for args, match in [((x.int(),), "unsupported dtype"), ((_t(4, 0),), "at least 1"), ((x, _t(7)), "vector of 8"),
                        ((x, _t(8), _t(8, dtype=torch.float16)), "parameters"), ((x,), "on a GPU")]:
        with pytest.raises(ValueError, match=match):
            M.layer_norm_tensors(*args)
    with pytest.raises(ValueError, match="eps"):
        M.layer_norm_tensors(x, eps=-1.0)
    with pytest.raises(ValueError, match="same shape"):
        M.layer_norm_backward_tensors(x, _t(4, 9), _t(4), _t(4))
    with pytest.raises(ValueError, match="on a GPU"):
        M.layer_norm_backward_tensors(x, x, _t(4), _t(4))


def test_matrix_forms():
    """What counts as a matrix of contiguous rows."""
    assert M._matrix("x", _t(3, 4, 5), 5).shape == (12, 5)
    assert M._matrix("x", _t(5), 5).shape == (1, 5)
    assert M._matrix("x", _t(4, 9)[:, 2:7], 5).stride() == (9, 1)
    for t, match in [(_t(5, 4).t(), "contiguous"), (_t(1, 5).expand(4, 5), "overlap"), (_t(4, 6), "5 columns"),
                     (_t(4, 10)[:, ::2], "contiguous")]:
        with pytest.raises(ValueError, match=match):
            M._matrix("x", t, 5)


# ---------------------------------------------------------------- the oracle itself

@pytest.mark.parametrize("act", sorted(M.ACTIVATION_CODES))
def test_oracle_gradients_against_differences(act):
    torch.manual_seed(5)
    x, w, b = torch.randn(5, 7).double(), torch.randn(6, 7).double(), torch.randn(6).double()
    dy = torch.randn(5, 6).double()

    def loss(x, w, b):
        return float((O.activate(x @ w.t() + b, act) * dy).sum())

    z = x @ w.t() + b
    (dx, _), (dw, _), (db, _) = O.linear_backward(dy, x, w, z, act)
    h = 1e-6
    for grad, at in ((dx, 0), (dw, 1), (db, 2)):
        v = [x, w, b]
        d = torch.randn_like(v[at])
        lo, hi = list(v), list(v)
        lo[at], hi[at] = v[at] - h * d, v[at] + h * d
        assert abs((loss(*hi) - loss(*lo)) / (2 * h) - float((grad * d).sum())) < 1e-6


def test_oracle_norm_gradients_against_differences():
    torch.manual_seed(6)
    x, w, b = torch.randn(4, 9).double(), torch.randn(9).double(), torch.randn(9).double()
    dy = torch.randn(4, 9).double()

    def loss(x, w, b):
        return float((O.layer_norm(x, w, b, 1e-3)[0][0] * dy).sum())

    _, (mean, _), (rstd, _) = O.layer_norm(x, w, b, 1e-3)
    (dx, _), (dw, _), (db, _) = O.layer_norm_backward(dy, x, mean, rstd, w, torch.float64)
    h = 1e-6
    for grad, at in ((dx, 0), (dw, 1), (db, 2)):
        v = [x, w, b]
        d = torch.randn_like(v[at])
        lo, hi = list(v), list(v)
        lo[at], hi[at] = v[at] - h * d, v[at] + h * d
        assert abs((loss(*hi) - loss(*lo)) / (2 * h) - float((grad * d).sum())) < 1e-6


def test_oracle_against_torch():
    torch.manual_seed(7)
    F = torch.nn.functional
    z = torch.randn(50).double() * 4
    for act, f in (("relu", F.relu), ("gelu", F.gelu), ("silu", F.silu),
                   ("gelu_tanh", lambda t: F.gelu(t, approximate="tanh"))):
        assert torch.allclose(O.activate(z, act), f(z), rtol=1e-12, atol=1e-14)
    x, w, b = torch.randn(6, 33).double(), torch.randn(33).double(), torch.randn(33).double()
    assert torch.allclose(O.layer_norm(x, w, b, 1e-5)[0][0], F.layer_norm(x, (33,), w, b, 1e-5), rtol=1e-12)
