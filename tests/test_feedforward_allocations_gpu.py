"""Who watches torch's allocations sees those of the gated block and the 8-bit products."""

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

from allreduce_emulated_peer_amd import mscl as M
from test_feedforward_gpu import normal, note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


class Watch(TorchDispatchMode):
    def __init__(self):
        super().__init__()
        self.made = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if isinstance(out, torch.Tensor) and "empty" in str(func):
            self.made.add(out.data_ptr())
        return out


class Listen(torch.overrides.TorchFunctionMode):
    def __init__(self):
        super().__init__()
        self.names = []

    def __torch_function__(self, func, types, args=(), kwargs=None):
        self.names.append(getattr(func, "__name__", ""))
        return func(*args, **(kwargs or {}))


def _calls():
    """Each form, and how many tensors it allocates besides a workspace."""
    gen = torch.Generator().manual_seed(121)
    m, k, n = 40, 96, 48
    dy, z, v = (normal(gen, m, n).cuda() for _ in range(3))
    x, wg, wu = normal(gen, m, k).cuda(), normal(gen, n, k).cuda(), normal(gen, n, k).cuda()
    (q, s), (qg, sg), (qu, su) = (M.quantize_tensors(t) for t in (x, wg, wu))
    return [(lambda: M.gated_linear_tensors(x, wg, wu, return_preacts=True), 3),
            (lambda: M.gated_linear_backward_tensors(dy, x, wg, wu, z, v), 5),
            (lambda: M.quantize_tensors(x), 2),
            (lambda: (M.linear_quantized_tensors(q, s, qg, sg),), 1),
            (lambda: (M.gated_linear_quantized_tensors(q, s, qg, sg, qu, su),), 1)]


def test_modes_see_the_allocations():
    for call, count in _calls():
        note("watched allocations", count)
        want = call()
        with Watch() as watch:
            got = call()
        assert {t.data_ptr() for t in got} <= watch.made and len(watch.made) >= count
        with Listen() as listen:
            again = call()
        assert sum("empty" in name for name in listen.names) >= count
        assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, got, again))


def test_fresh_memory_is_filled_where_torch_fills_it(monkeypatch):
    """In torch's deterministic mode new tensors are filled; the results are the same, as they are written whole."""
    made = []
    empty_strided = torch.empty_strided

    def counted(*args, **kwargs):
        t = empty_strided(*args, **kwargs)
        made.append(t.numel() == 0 or t.dtype == torch.uint8 or bool(torch.isnan(t).all()) or not t.is_floating_point())
        return t

    calls = _calls()
    want = [call() for call, _ in calls]
    monkeypatch.setattr(torch, "empty_strided", counted)
    torch.use_deterministic_algorithms(True)
    try:
        for (call, count), w in zip(calls, want):
            note("filled allocations", count)
            del made[:]
            assert all(torch.equal(a, b) for a, b in zip(call(), w))
            assert len(made) >= count and all(made)
    finally:
        torch.use_deterministic_algorithms(False)
