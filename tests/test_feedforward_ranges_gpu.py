"""The ends of binary16's range in the gated block's backward pass, as the header states them."""

import math

import pytest
import torch

import feedforward_oracle as F
from allreduce_emulated_peer_amd import mscl as M
from test_feedforward_gpu import gated_case, note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


def constant(m, n, value):
    return torch.full((m, n), value, dtype=torch.float16, device="cuda")


def test_products_gradients_at_the_ends_of_binary16():
    m, k, n = 64, 72, 40
    gen = torch.Generator().manual_seed(131)
    x, wg, wu = (a.cuda() for a in gated_case(gen, m, k, n, torch.float16, bias=False)[:3])
    z = constant(m, n, 0.0)  # dv is 0
    note("small binary16 gradients")
    # dz = dy v: 2^-26 is nothing to the products, and counts in the bias's gradient
    dx, dg, du, dbg, _ = M.gated_linear_backward_tensors(constant(m, n, 2.0 ** -13), x, wg, wu, z, constant(m, n, 2.0 ** -13), "none")
    assert not bool(dx.any()) and not bool(dg.any()) and not bool(du.any())
    assert torch.equal(dbg, torch.full_like(dbg, m * 2.0 ** -26))
    # 2^-24, binary16's smallest, is there
    dx, dg, _, _, _ = M.gated_linear_backward_tensors(constant(m, n, 2.0 ** -12), x, wg, wu, z, constant(m, n, 2.0 ** -12), "none")
    want = F.gated_linear_backward(constant(m, n, 2.0 ** -12), x, wg, wu, z, constant(m, n, 2.0 ** -12), "none")
    F.assert_within(dx, want[0], "dx")
    F.assert_within(dg, want[1], "dwg")
    assert bool(dx.any()) and bool(dg.any())
    note("large binary16 gradients")
    one = torch.ones(n, k, dtype=torch.float16, device="cuda")
    for v, finite in ((255.75, True), (256.0, False)):  # times 256: 65472 and 65536
        dx, _, _, dbg, _ = M.gated_linear_backward_tensors(constant(1, n, 256.0), x[:1], one / 128, one, z[:1], constant(1, n, v), "none")
        assert bool(torch.isfinite(dx).all()) == finite and bool((dx == math.inf).all()) != finite
        assert bool(torch.isfinite(dbg).all()) == finite  # a single row's sum is past the range too
