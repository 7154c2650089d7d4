"""A tensor-parallel gated feed-forward block over R emulated ranks of one GPU: training in bfloat16, serving in 8 bits.

    h   = layer_norm(x)                                          (every rank the same)
    a_r = silu(h wg_r^T) * (h wu_r^T)                            column-parallel: rank r has a slice of both weights' rows
    s_r = a_r wd_r^T  (+ x on rank 0: the residual)              row-parallel: rank r has a slice of wd's columns
    y   = allreduce(s_r)

The backward pass runs the same layers in the other direction; its AllReduce
adds the ranks' gradients of h.  For serving, each rank's weights become 8-bit
integers with a scale for each output, once, and every step turns its rows to 8
bits with a scale for each token in front of either product.  Run it on an
MI355X after the library is built:

    python examples/gated_feedforward.py [--ranks 8] [--tokens 512] [--width 8192] [--inner 32768]
"""

import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from allreduce_emulated_peer_amd import mscl  # noqa: E402


class Block:
    """The block's parameters, sliced over the ranks, and its passes."""

    def __init__(self, ranks, width, inner, dtype=torch.bfloat16, device="cuda", seed=0):
        if inner % ranks:
            raise ValueError("inner must be a multiple of ranks")
        g = torch.Generator().manual_seed(seed)

        def normal(*shape, scale=1.0):
            return (torch.randn(shape, generator=g) * scale).to(dtype).to(device)

        self.ranks = ranks
        self.gain, self.shift = 1 + normal(width, scale=0.1), normal(width, scale=0.1)
        self.wg = list(normal(inner, width, scale=width ** -0.5).chunk(ranks, 0))
        self.wu = list(normal(inner, width, scale=width ** -0.5).chunk(ranks, 0))
        # wd's columns: each rank's slice as it lies, rows `inner` elements apart
        self.wd = list(normal(width, inner, scale=inner ** -0.5).chunk(ranks, 1))
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
            a, z, v = mscl.gated_linear_tensors(h, self.wg[r], self.wu[r], return_preacts=True)
            parts.append(mscl.linear_tensors(a, self.wd[r], residual=x if r == 0 else None))
            kept.append((a, z, v))
        return self._sum(parts), (x, h, mean, rstd, kept)

    def backward(self, dy, saved):
        """Gradients of x, of the norm's gain and shift, and of each rank's (wg, wu, wd)."""
        x, h, mean, rstd, kept = saved
        parts, grads = [], []
        for r, (a, z, v) in enumerate(kept):
            da, dwd, _ = mscl.linear_backward_tensors(dy, a, self.wd[r], need_db=False)
            dh, dwg, dwu, _, _ = mscl.gated_linear_backward_tensors(da, h, self.wg[r], self.wu[r], z, v, need_db=False)
            parts.append(dh)
            grads.append((dwg, dwu, dwd))
        dx, dgain, dshift = mscl.layer_norm_backward_tensors(self._sum(parts), x, mean, rstd, self.gain)
        return dx + dy, dgain, dshift, grads

    def quantize(self):
        """The ranks' weights in 8 bits, for serve()."""
        return [tuple(mscl.quantize_tensors(w[r]) for w in (self.wg, self.wu, self.wd)) for r in range(self.ranks)]

    def serve(self, x, weights):
        """y from 8-bit weights and rows."""
        h = mscl.layer_norm_tensors(x, self.gain, self.shift)
        q, scale = mscl.quantize_tensors(h)
        parts = []
        for r, ((wg, sg), (wu, su), (wd, sd)) in enumerate(weights):
            a = mscl.gated_linear_quantized_tensors(q, scale, wg, sg, wu, su, dtype=x.dtype)
            p, p_scale = mscl.quantize_tensors(a)
            parts.append(mscl.linear_quantized_tensors(p, p_scale, wd, sd, residual=x if r == 0 else None, dtype=x.dtype))
        return self._sum(parts)


def main():
    p = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    p.add_argument("--ranks", type=int, default=8)
    p.add_argument("--tokens", type=int, default=512)
    p.add_argument("--width", type=int, default=8192)
    p.add_argument("--inner", type=int, default=32768)
    a = p.parse_args()
    block = Block(a.ranks, a.width, a.inner)
    weights = block.quantize()
    x = torch.randn(a.tokens, a.width, device="cuda").bfloat16()
    dy = torch.randn_like(x)
    times = []
    for _ in range(5):
        marks = [torch.cuda.Event(enable_timing=True) for _ in range(4)]
        marks[0].record()
        y, saved = block.forward(x)
        marks[1].record()
        grads = block.backward(dy, saved)
        marks[2].record()
        served = block.serve(x, weights)
        marks[3].record()
        torch.cuda.synchronize()
        times.append([marks[i].elapsed_time(marks[i + 1]) for i in range(3)])
    fwd, bwd, srv = (sorted(t)[len(t) // 2] for t in zip(*times))
    flops = 6 * a.tokens * a.width * a.inner
    print(f"{a.ranks} ranks, {a.tokens} x {a.width} -> {a.inner}: bf16 forward {fwd:.3f} ms ({flops / fwd / 1e9:.0f} TFLOP/s), "
          f"backward {bwd:.3f} ms ({2 * flops / bwd / 1e9:.0f} TFLOP/s), 8-bit forward {srv:.3f} ms")
    off = float((served.float() - y.float()).norm() / y.float().norm())
    print(f"|y| {y.float().norm():.4g}, |dx| {grads[0].float().norm():.4g}, 8 bits against bf16 {off:.2g}")


if __name__ == "__main__":
    main()
