"""The sizes that the GPU tests of binary32 parts run at are sizes at which the library takes them (CPU: workspace queries)."""

import pytest

import binary32_parts as P
import test_feedforward as T
from allreduce_emulated_peer_amd import mscl as M

SLACK = 64 * 1024  # roundings of each piece to 256 bytes
GRADIENTS = ("dx", "dgate_w", "dup_w", "dgate_bias", "dup_bias")


def asked(op, names, m, k, n, **change):
    far = {name: T.A + i * (1 << 38) for i, name in enumerate(names) if T.is_pointer(name)}
    strides = {s + "_stride": k for s in T.INNER} | {s + "_stride": n for s in T.OUTER}
    status, need = T.workspace(op, **{**far, **strides, "rows": m, "in_features": k, "out_features": n, "dtype": M.FLOAT32,
                                      **change})
    assert status == M.SUCCESS
    return need


@pytest.mark.parametrize("m,k,n,forward,dx,dw", P.SIZES)
def test_sizes_are_taken_into_parts(m, k, n, forward, dx, dw):
    want = P.forward_bytes(m, k, n, forward)
    assert want <= asked("gated_linear", T.GATED, m, k, n) <= want + SLACK
    for names, of_dx, of_dw in ((("dx",), dx, None), (("dgate_w", "dup_w"), None, dw)):
        shares = of_dx if of_dw is None else of_dw
        if shares == 0:
            continue
        want = P.gradient_bytes(m, k, n, of_dx, of_dw)
        got = asked("gated_linear_backward", T.GATED_BACKWARD, m, k, n, **{g: 0 for g in GRADIENTS if g not in names})
        assert want <= got <= want + SLACK, names


def test_both_gradients_and_shares_are_covered():
    for at, least in ((3, {1, 2}), (4, {0, 1, 2, 4}), (5, {0, 1, 2})):
        assert least <= {size[at] for size in P.SIZES}


IN_SHARES = [(*size[:3], M.FLOAT32) for size in P.SIZES if size[5] > 1]
IN_SHARES += [(m, k, n, dtype) for m, k, n in ((2048, 260, 130), (4000, 100, 70)) for dtype in (M.FLOAT32, M.BFLOAT16)]


@pytest.mark.parametrize("m,k,n,dtype", IN_SHARES)
def test_a_weight_gradient_that_is_not_wanted_takes_no_share_of_the_workspace(m, k, n, dtype):
    def need(*names):
        return asked("gated_linear_backward", T.GATED_BACKWARD, m, k, n, dtype=dtype,
                     **{g: 0 for g in GRADIENTS if g not in names})

    both, gate, up = need("dgate_w", "dup_w"), need("dgate_w"), need("dup_w")
    assert gate == up and both - gate >= P._shares(2, n, k) // 2  # a share of one of them at the least
