"""The gated block's small gradients where their last tile of columns lies over the one before it: one bit pattern each."""

import math

import pytest
import torch

import feedforward_oracle as F
from allreduce_emulated_peer_amd import mscl as M
from test_feedforward_gpu import DTYPES, gated_case, normal, note

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


def bits(t):
    return t.view(torch.int32 if t.dtype == torch.float32 else torch.int16)


# k 64 and more and no multiple of 64: the last tile of 64 columns starts at k - 64.  Tiles of 64 and of 128 rows, with k
# of the products in one run and in shares.
@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("m,k,n", [(40, 100, 50), (70, 330, 45), (33, 94, 700), (700, 65, 40), (515, 1025, 770)])
@pytest.mark.parametrize("far", [2.0 ** 106, math.inf, math.nan])
def test_columns_of_two_tiles_have_one_value(dtype, m, k, n, far):
    """A column that makes a binary32 wave sum its columns again changes no bit of the columns that other tiles store."""
    gen = torch.Generator().manual_seed(91)
    t = DTYPES[dtype]
    x, wg, wu, _, _ = (a if a is None else a.cuda() for a in gated_case(gen, m, k, n, t, bias=False))
    dy, z, v = (normal(gen, m, n, scale=s, dtype=t).cuda() for s in (1.0, 1.5, 1.0))
    last = (k - 1) // 64 * 64  # the last tile's own first column; it lies over those from k - 64 on

    def run(x, wg):
        return M.gated_linear_backward_tensors(dy, x, wg, wu, z, v, "silu")

    plain = run(x, wg)
    for hot in sorted({last, min(last + 1, k - 1), k - 1, last - 1, k - 64}):
        xh, wh = x.clone(), wg.clone()
        xh[:, hot], wh[:, hot] = far, far
        note("columns of two tiles", dtype, m, k, n, far, hot)
        first = run(xh, wh)
        for _ in range(4):
            for a, b in zip(first, run(xh.clone(), wh.clone())):
                assert torch.equal(bits(a), bits(b))
        # 32 columns at most are summed together with this one, in the tile that has it
        near = torch.zeros(k, dtype=torch.bool, device="cuda")
        begin = k - 64 if hot >= last else hot // 64 * 64
        block = begin + (hot - begin) // 32 * 32
        near[max(block, last if hot >= last else 0):min(block + 32, k if hot >= last else last)] = True
        if hot < last:  # the moved tile's own columns beside it may be summed again as well
            near[last:] = True
        for a, b in zip(first[:3], plain[:3]):
            assert torch.equal(bits(a)[:, ~near], bits(b)[:, ~near]), hot
        rest = [c for c in range(k) if c != hot]
        want = F.gated_linear_backward(dy, x[:, rest], wg[:, rest], wu[:, rest], z, v, "silu")
        for a, w, name in zip(first[:3], want, ("dx", "dwg", "dwu")):
            F.assert_within(a[:, rest], w, name)
