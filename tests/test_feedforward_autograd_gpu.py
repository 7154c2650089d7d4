"""What autograd may lose at the gated block and the 8-bit products is refused."""

import pytest
import torch

from allreduce_emulated_peer_amd import mscl as M
from test_feedforward_gpu import normal, note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


def tensors(seed=111, m=6, k=40, n=24):
    gen = torch.Generator().manual_seed(seed)
    dy, z, v = (normal(gen, m, n).cuda() for _ in range(3))
    return dy, normal(gen, m, k).cuda(), normal(gen, n, k).cuda(), normal(gen, n, k).cuda(), z, v


def test_a_second_derivative_is_not_lost_unseen():
    args = tensors()
    note("second derivative")
    want = M.gated_linear_backward_tensors(*args)
    assert not any(g.requires_grad for g in want)
    side = torch.cuda.Stream()
    for stream in (None, side):
        for which in range(6):
            some = [t.clone().requires_grad_(i == which) for i, t in enumerate(args)]
            if stream is not None:
                stream.wait_stream(torch.cuda.current_stream())
            got = M.gated_linear_backward_tensors(*some, stream=stream)
            torch.cuda.synchronize()
            for a, b in zip(got, want):
                assert a.requires_grad and torch.equal(a, b)
                with pytest.raises(RuntimeError, match="gated_linear_backward_tensors has no gradient"):
                    a.sum().backward()
            with torch.no_grad():
                assert not any(g.requires_grad for g in M.gated_linear_backward_tensors(*some))
            dx, dg, du, dbg, dbu = M.gated_linear_backward_tensors(*some, need_dx=False, need_db=False)
            assert dx is dbg is dbu is None and dg.requires_grad and du.requires_grad
            assert M.gated_linear_backward_tensors(*some, need_dx=False, need_dw=False, need_db=False) == (None,) * 5


class Gated(torch.autograd.Function):
    """A user's own function around the block."""

    @staticmethod
    def forward(ctx, x, wg, wu):
        y, gate, up = M.gated_linear_tensors(x, wg, wu, return_preacts=True)
        ctx.save_for_backward(x, wg, wu, gate, up)
        return y

    @staticmethod
    def backward(ctx, dy):
        x, wg, wu, gate, up = ctx.saved_tensors
        return M.gated_linear_backward_tensors(dy.contiguous(), x, wg, wu, gate, up, need_db=False)[:3]


def test_a_function_of_ones_own_has_a_first_derivative_and_no_second():
    _, x, wg, wu, _, _ = tensors()
    x.requires_grad_()
    note("a function of one's own")
    exact = x.detach().double().requires_grad_()
    y = torch.nn.functional.silu(exact @ wg.double().t()) * (exact @ wu.double().t())
    want, = torch.autograd.grad(y.square().sum(), exact)
    dx, = torch.autograd.grad(Gated.apply(x, wg, wu).square().sum(), x)
    assert float((dx.double() - want).norm()) <= 1e-5 * float(want.norm())
    dx, = torch.autograd.grad(Gated.apply(x, wg, wu).square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="no gradient"):
        dx.square().sum().backward()


def _calls():
    """name -> (call, its inputs), each with all optional inputs."""
    dy, x, wg, wu, z, v = tensors()
    b, r = dy[0].clone(), dy.clone()
    q, s = M.quantize_tensors(x)
    (qg, sg), (qu, su) = M.quantize_tensors(wg), M.quantize_tensors(wu)
    g = x[0].clone()
    y, mean, rstd = M.layer_norm_tensors(x, g, return_stats=True)
    t = torch.float32
    return {
        "gated_linear": (lambda x, wg, wu, bg, bu, **k: M.gated_linear_tensors(x, wg, wu, bg, bu, **k), (x, wg, wu, b, b)),
        "gated_linear_backward": (lambda *a, **k: M.gated_linear_backward_tensors(*a, **k)[0], (dy, x, wg, wu, z, v)),
        "quantize": (lambda x, **k: M.quantize_tensors(x, **k)[1], (x,)),
        "linear_quantized": (lambda s, sw, b, r, **k: M.linear_quantized_tensors(q, s, qg, sw, b, r, dtype=t, **k), (s, sg, b, r)),
        "gated_linear_quantized": (lambda s, sg, su, bg, bu, **k: M.gated_linear_quantized_tensors(
            q, s, qg, sg, qu, su, bg, bu, dtype=t, **k), (s, sg, su, b, b)),
        "linear": (lambda *a, **k: M.linear_tensors(*a, **k), (x, wg, b, r)),
        "linear_backward": (lambda dy, x, w, z, **k: M.linear_backward_tensors(dy, x, w, z, "gelu", **k)[0], (dy, x, wg, z)),
        "layer_norm": (lambda *a, **k: M.layer_norm_tensors(*a, **k), (x, g, g)),
        "layer_norm_backward": (lambda *a, **k: M.layer_norm_backward_tensors(*a, **k)[0], (x, y, mean, rstd, g)),
    }


@pytest.mark.parametrize("name", ["gated_linear", "gated_linear_backward", "quantize", "linear_quantized",
                                  "gated_linear_quantized", "linear", "linear_backward", "layer_norm", "layer_norm_backward"])
def test_a_forward_mode_tangent_is_not_lost_unseen(name):
    call, args = _calls()[name]
    note("forward-mode tangent", name)
    want = call(*args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.autograd.forward_ad.dual_level():
        for which in range(len(args)):
            some = list(args)
            some[which] = torch.autograd.forward_ad.make_dual(args[which], torch.ones_like(args[which]))
            for more in ({}, {"stream": side}):
                with pytest.raises(RuntimeError, match=f"^{name}_tensors has no forward-mode derivative"):
                    call(*some, **more)
            with torch.no_grad(), pytest.raises(RuntimeError, match="forward-mode"):
                call(*some)
        # tensors without a tangent go through inside of a dual level too
        assert torch.equal(call(*args), want)
    assert torch.equal(call(*args), want)
    if name != "quantize":
        with pytest.raises(RuntimeError):
            torch.func.jvp(lambda a: call(a, *args[1:]), (args[0],), (torch.ones_like(args[0]),))
