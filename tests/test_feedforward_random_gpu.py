"""Seeded random calls of the gated feed-forward block and of the 8-bit products against their formulas in 64 bits."""

import math
import random

import pytest
import torch

import feedforward_oracle as F
from allreduce_emulated_peer_amd import mscl as M
from test_feedforward_gpu import ACTS, DTYPES, note, placed

pytestmark = pytest.mark.gpu
FORMS = ("plain", "plain", "columns", "odd")
BACK = ("dx", "dwg", "dwu", "dbg", "dbu")


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


def size(rng, most):
    n = int(round(math.exp(rng.uniform(0, math.log(most)))))
    return n // 64 * 64 if n >= 128 and rng.random() < 0.4 else n


@pytest.mark.parametrize("seed", range(48))
def test_random_calls(seed):
    rng = random.Random(1000 + seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    for _ in range(4):
        m, k, n = size(rng, 5000), size(rng, 5000), size(rng, 5000)
        while m * k * n > 2e9:
            m = max(1, m // 2)
        dtype, act, form = rng.choice(sorted(DTYPES)), rng.choice(ACTS), [rng.choice(FORMS) for _ in range(8)]
        t = DTYPES[dtype]
        bias, residual = rng.random() < 0.5, rng.random() < 0.5

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=gen, device="cuda") * scale).to(t)

        def integers(*shape):
            return torch.randint(-128, 128, shape, generator=gen, device="cuda", dtype=torch.int8)

        x, wg, wu = normal(m, k), normal(n, k, scale=k ** -0.5), normal(n, k, scale=k ** -0.5)
        bg, bu = (normal(n), normal(n)) if bias else (None, None)
        note("random", seed, m, k, n, dtype, act, form, bias, residual)
        there = [placed(a, f) for a, f in zip((x, wg, wu, bg, bu), form)]
        got = M.gated_linear_tensors(*there, act, return_preacts=True)
        for g, want, name in zip(got, F.gated_linear(x, wg, wu, bg, bu, act), ("y", "gate", "up")):
            F.assert_within(g, want, name)
        dy, z, v = normal(m, n), normal(m, n, scale=1.5), normal(m, n)
        there = [placed(a, f) for a, f in zip((dy, x, wg, wu, z, v), form)]
        got = M.gated_linear_backward_tensors(*there, act)
        for g, want, name in zip(got, F.gated_linear_backward(dy, x, wg, wu, z, v, act), BACK):
            F.assert_within(g, want, name)
        q, s = M.quantize_tensors(placed(x, form[6]))
        want_q, want_s = F.quantize(x.cpu())
        assert torch.equal(q.cpu(), want_q) and torch.equal(s.cpu(), want_s)
        w, u, r = integers(n, k), integers(n, k), normal(m, n) if residual else None
        sw, su = (torch.rand(n, generator=gen, device="cuda") * 0.02 / k ** 0.5 + 1e-5 for _ in range(2))
        y = M.linear_quantized_tensors(placed(q, form[0]), s, placed(w, form[1]), sw, bg, placed(r, form[2]), act, dtype=t)
        F.assert_within(y, F.linear_quantized(q, s, w, sw, bg, r, act, t), "8-bit y")
        y = M.gated_linear_quantized_tensors(placed(q, form[3]), s, placed(w, form[4]), sw, placed(u, form[5]), su, bg, bu, act,
                                             dtype=t)
        F.assert_within(y, F.gated_linear_quantized(q, s, w, sw, u, su, bg, bu, act, t), "gated 8-bit y")
