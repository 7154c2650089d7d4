"""The gated feed-forward block of examples/ against the whole block in 64 bits."""

import importlib.util
import os

import pytest
import torch

import feedforward_oracle as F
from allreduce_emulated_peer_amd import mscl as M

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "gated_feedforward.py")


def example():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    spec = importlib.util.spec_from_file_location("gated_feedforward", PATH)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def d(t):
    return t.detach().cpu().double()


@pytest.mark.parametrize("ranks,tokens,width,inner", [(4, 24, 256, 512), (8, 65, 320, 1024), (2, 1, 128, 96)])
def test_block_against_64_bits(ranks, tokens, width, inner):
    block = example().Block(ranks, width, inner)
    gen = torch.Generator().manual_seed(60)
    x, dy = (torch.randn(tokens, width, generator=gen).bfloat16() for _ in range(2))
    print(f"[gpu-case] gated block R={ranks} {tokens} x {width} -> {inner}", flush=True)
    y, saved = block.forward(x.cuda())
    dx, dgain, dshift, grads = block.backward(dy.cuda(), saved)
    torch.cuda.synchronize()

    wg, wu, wd = (d(torch.cat(v, k)) for v, k in ((block.wg, 0), (block.wu, 0), (block.wd, 1)))
    leaves = [d(x), d(block.gain), d(block.shift), wg, wu, wd]
    for t in leaves:
        t.requires_grad_()
    h = torch.nn.functional.layer_norm(leaves[0], (width,), leaves[1], leaves[2], 1e-5)
    want = (torch.nn.functional.silu(h @ leaves[3].t()) * (h @ leaves[4].t())) @ leaves[5].t() + leaves[0]
    (want * d(dy)).sum().backward()
    got = [y, dx, dgain, dshift, torch.cat([g[0] for g in grads]), torch.cat([g[1] for g in grads]),
           torch.cat([g[2] for g in grads], 1)]
    exact = [want.detach()] + [t.grad for t in leaves]
    # In the 2-norm: every value on the way is rounded to bf16 (at most half a step, 2^-8), and none passes more than
    # ten such roundings (h, z, v, a, s_r, the sum; then da, dz or dv, dh_r, the sum, the gradient; the first half's
    # reach the second through z and v).
    bound = 11 * 2.0 ** -8 / 3 ** 0.5
    for g, e, name in zip(got, exact, ("y", "dx", "dgain", "dshift", "dwg", "dwu", "dwd")):
        off = float((d(g) - e).norm() / e.norm())
        assert off < bound, f"{name}: {off:.3g} of its size off"


@pytest.mark.parametrize("ranks,tokens,width,inner", [(4, 24, 256, 512), (8, 300, 320, 1024), (2, 1, 128, 96)])
def test_serving_in_8_bits(ranks, tokens, width, inner):
    """Rank by rank against the formulas of the same integers, and the whole against what 8 bits leave out."""
    block = example().Block(ranks, width, inner)
    weights = block.quantize()
    for r, of_rank in enumerate(weights):
        for (q, scale), w in zip(of_rank, (block.wg[r], block.wu[r], block.wd[r])):
            want_q, want_scale = F.quantize(w.cpu())
            assert torch.equal(q.cpu(), want_q) and torch.equal(scale.cpu(), want_scale)
    gen = torch.Generator().manual_seed(61)
    x = torch.randn(tokens, width, generator=gen).bfloat16().cuda()
    print(f"[gpu-case] gated block in 8 bits R={ranks} {tokens} x {width} -> {inner}", flush=True)
    y = block.serve(x, weights)
    torch.cuda.synchronize()

    h = M.layer_norm_tensors(x, block.gain, block.shift).cpu()
    q, scale = F.quantize(h)
    total = torch.zeros(tokens, width, dtype=torch.float64)
    slack, size = torch.zeros_like(total), torch.zeros_like(total)
    for r, of_rank in enumerate(weights):
        (wg, sg), (wu, su), (wd, sd) = [(a.cpu(), b.cpu()) for a, b in of_rank]
        there = [t.cuda() for t in (q, scale, wg, sg, wu, su)]
        a = M.gated_linear_quantized_tensors(*there, dtype=torch.bfloat16).cpu()
        F.assert_within(a, F.gated_linear_quantized(q, scale, wg, sg, wu, su, None, None, "silu", torch.bfloat16), f"a of {r}")
        p, p_scale = F.quantize(a)
        exact, bound = F.linear_quantized(p, p_scale, wd, sd, None, x.cpu() if r == 0 else None, "none", torch.bfloat16)
        total, slack, size = total + exact, slack + bound, size + exact.abs() + bound
    # the ranks' parts add up in binary32 and are rounded once more
    F.assert_within(y, (total, slack + 2.0 ** -8 * (total.abs() + slack) + ranks * 2.0 ** -23 * size), "y")


def test_the_program_runs(capsys, monkeypatch):
    module = example()
    monkeypatch.setattr("sys.argv", ["gated_feedforward.py", "--ranks", "2", "--tokens", "8", "--width", "128", "--inner", "256"])
    module.main()
    assert "8-bit forward" in capsys.readouterr().out
