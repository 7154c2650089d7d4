"""Sizes whose tiles no launch can hold are refused by the workspace query and by the call, before any GPU call (CPU)."""

import pytest

import test_feedforward as T
from allreduce_emulated_peer_amd import mscl as M

NAMES = {"gated_linear": T.GATED, "gated_linear_backward": T.GATED_BACKWARD, "linear_quantized": T.INT8,
         "gated_linear_quantized": T.GATED_INT8}
BIASES = dict(dx=0, dgate_w=0, dup_w=0)


def sized(op, m, k, n, **change):
    """A call's fields at these sizes, its buffers 2^42 bytes apart."""
    at = {name: (i + 1) << 42 for i, name in enumerate(NAMES[op]) if T.is_pointer(name)}
    strides = {s + "_stride": k for s in T.INNER} | {s + "_stride": n for s in T.OUTER}
    return {**at, **strides, "rows": m, "in_features": k, "out_features": n, **change}


# A launch has fewer than 2^32 threads: few rows take 512 for 16 outputs, tiles 256 for up to 128 x 128, the last sums of
# the biases' gradients 256 for 32.
@pytest.mark.parametrize("op,m,k,n,change", [
    ("linear_quantized", 1, 16, 2 ** 27, {}), ("linear_quantized", 8, 64, 2 ** 30, {}),
    ("gated_linear_quantized", 32, 16, 2 ** 27, {}), ("gated_linear", 1, 16, 2 ** 27, {}),
    ("gated_linear", 3, 8, 2 ** 28, dict(dtype=M.FLOAT32)), ("linear_quantized", 2 ** 31 - 1, 16, 256, {}),
    ("gated_linear", 2 ** 31 - 1, 8, 200, {}), ("gated_linear_backward", 1, 8, 2 ** 29, BIASES),
    ("gated_linear_backward", 2 ** 30, 1024, 8, {})])
def test_too_many_tiles_for_a_launch(op, m, k, n, change):
    fields = sized(op, m, k, n, **change)
    assert T.workspace(op, **fields)[0] == M.ERR_INVALID_ARGUMENT
    status, text = T.call(op, 1 << 62, 1 << 61, **fields)
    assert status == M.ERR_INVALID_ARGUMENT and "launch" in text


@pytest.mark.parametrize("op,m,k,n,change", [
    ("linear_quantized", 1, 16, 2 ** 27 - 16, {}), ("linear_quantized", 17, 16, 2 ** 28 - 32, {}),
    ("gated_linear_quantized", 32, 16, 2 ** 27 - 16, {}), ("gated_linear", 1, 16, 2 ** 27 - 16, {}),
    ("linear_quantized", 33, 16, 2 ** 29, {}), ("gated_linear", 2 ** 28, 8, 100, {}),
    ("gated_linear_backward", 1, 8, 2 ** 29 - 32, BIASES)])
def test_the_largest_that_fit(op, m, k, n, change):
    assert T.workspace(op, **sized(op, m, k, n, **change))[0] == M.SUCCESS
