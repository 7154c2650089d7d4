"""The tensor-parallel block of examples/ against the whole block in 64 bits."""

import importlib.util
import os

import pytest
import torch

import operator_oracle as O
from allreduce_emulated_peer_amd import mscl as M

pytestmark = pytest.mark.gpu
PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "tensor_parallel_layer.py")


@pytest.mark.parametrize("ranks,tokens,width,inner", [(4, 24, 256, 512), (8, 65, 320, 1024), (2, 1, 128, 96)])
def test_block_against_64_bits(ranks, tokens, width, inner):
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    spec = importlib.util.spec_from_file_location("tensor_parallel_layer", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    block = example.Block(ranks, width, inner)
    gen = torch.Generator().manual_seed(40)
    x = torch.randn(tokens, width, generator=gen).bfloat16()
    dy = torch.randn(tokens, width, generator=gen).bfloat16()
    print(f"[gpu-case] block R={ranks} {tokens} x {width} -> {inner}", flush=True)
    y, saved = block.forward(x.cuda())
    dx, dgain, dshift, grads = block.backward(dy.cuda(), saved)
    torch.cuda.synchronize()

    d = lambda t: t.detach().cpu().double()  # noqa: E731
    w1, b1, w2 = (d(torch.cat(v, k)) for v, k in ((block.w1, 0), (block.b1, 0), (block.w2, 1)))
    leaves = [d(x), d(block.gain), d(block.shift), w1, b1, w2]
    for t in leaves:
        t.requires_grad_()
    h = torch.nn.functional.layer_norm(leaves[0], (width,), leaves[1], leaves[2], 1e-5)
    want = O.activate(h @ leaves[3].t() + leaves[4], "gelu") @ leaves[5].t() + leaves[0]
    (want * d(dy)).sum().backward()
    got = [y, dx, dgain, dshift, torch.cat([g[0] for g in grads]), torch.cat([g[1] for g in grads]),
           torch.cat([g[2] for g in grads], 1)]
    exact = [want.detach()] + [t.grad for t in leaves]
    # In the 2-norm: every value on the way is rounded to bf16 (2^-9 rms at most half a step, 2^-8), and no value
    # passes more than eight such roundings (h, a, s_r, the sum; then da, dz, dh_r, the sum, the gradient).
    bound = 9 * 2.0 ** -8 / 3 ** 0.5
    for g, e, name in zip(got, exact, ("y", "dx", "dgain", "dshift", "dw1", "db1", "dw2")):
        off = float((d(g) - e).norm() / e.norm())
        assert off < bound, f"{name}: {off:.3g} of the gradient's size off"
