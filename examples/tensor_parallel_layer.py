"""A tensor-parallel MLP block over R emulated ranks of one GPU, forward and backward.

    h   = layer_norm(x)                                   (every rank the same)
    a_r = gelu(h w1_r^T + b1_r)                           column-parallel: rank r has a slice of w1's rows
    s_r = a_r w2_r^T  (+ x on rank 0: the residual)       row-parallel: rank r has a slice of w2's columns
    y   = allreduce(s_r)

The backward pass runs the same layers in the other direction; its AllReduce
adds the ranks' gradients of h.  Run it on an MI355X after the library is
built:

    python examples/tensor_parallel_layer.py [--ranks 8] [--tokens 512] [--width 8192] [--inner 32768]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from allreduce_emulated_peer_amd import mscl  # noqa: E402


class Block:
    """The block's parameters, sliced over the ranks, and its two passes."""

    def __init__(self, ranks, width, inner, dtype=torch.bfloat16, device="cuda", seed=0):
        if inner % ranks:
            raise ValueError("inner must be a multiple of ranks")
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=g) * scale).to(dtype).to(device)

        self.ranks = ranks
        self.gain, self.shift = 1 + normal(width, scale=0.1), normal(width, scale=0.1)
        self.w1 = list(normal(inner, width, scale=width ** -0.5).chunk(ranks, 0))
        self.b1 = list(normal(inner, scale=0.1).chunk(ranks))
        # w2's columns: each rank's slice as it lies, rows `inner` elements apart
        self.w2 = list(normal(width, inner, scale=inner ** -0.5).chunk(ranks, 1))
        mscl.channel_create(ranks, torch.device(device).index or 0)

    def _sum(self, parts):
        """AllReduce, in place; every rank ends up with the same rows."""
        mscl.allreduce_tensors(parts, parts)
        return parts[0]

    def forward(self, x):
        """y and what backward needs."""
        h, mean, rstd = mscl.layer_norm_tensors(x, self.gain, self.shift, return_stats=True)
        kept, parts = [], []
        for r in range(self.ranks):
            a, z = mscl.linear_tensors(h, self.w1[r], self.b1[r], activation="gelu", return_preact=True)
            parts.append(mscl.linear_tensors(a, self.w2[r], residual=x if r == 0 else None))
            kept.append((a, z))
        return self._sum(parts), (x, h, mean, rstd, kept)

    def backward(self, dy, saved):
        """Gradients of x, of the norm's gain and shift, and of each rank's (w1, b1, w2)."""
        x, h, mean, rstd, kept = saved
        parts, grads = [], []
        for r, (a, z) in enumerate(kept):
            da, dw2, _ = mscl.linear_backward_tensors(dy, a, self.w2[r], need_db=False)
            dh, dw1, db1 = mscl.linear_backward_tensors(da, h, self.w1[r], z, "gelu")
            parts.append(dh)
            grads.append((dw1, db1, dw2))
        dx, dgain, dshift = mscl.layer_norm_backward_tensors(self._sum(parts), x, mean, rstd, self.gain)
        return dx + dy, dgain, dshift, grads


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=8)
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--width", type=int, default=8192)
    p.add_argument("--inner", type=int, default=32768)
    a = p.parse_args()
    block = Block(a.ranks, a.width, a.inner)
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    dy = torch.randn_like(x)
    times = []
    for _ in range(5):
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(3)]
        marks[0].record()
        y, saved = block.forward(x)
        marks[1].record()
        grads = block.backward(dy, saved)
        marks[2].record()
        torch.cuda.synchronize()
        times.append((marks[0].elapsed_time(marks[1]), marks[1].elapsed_time(marks[2])))
    fwd, bwd = (sorted(t)[len(t) // 2] for t in zip(*times))
    flops = 4 * a.tokens * a.width * a.inner
    print(f"{a.ranks} ranks, {a.tokens} x {a.width} -> {a.inner}, bf16: forward {fwd:.3f} ms "
          f"({flops / fwd / 1e9:.0f} TFLOP/s), backward {bwd:.3f} ms ({2 * flops / bwd / 1e9:.0f} TFLOP/s)")
    print(f"|y| {y.float().norm():.4g}, |dx| {grads[0].float().norm():.4g}")


if __name__ == "__main__":
    main()
