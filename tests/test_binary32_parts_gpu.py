"""The gated block's large binary32 products, whose operands are taken into bfloat16 parts once, against 64 bits."""

import math
import os
import subprocess
import sys

import pytest
import torch

import binary32_parts as P
import feedforward_oracle as F
from allreduce_emulated_peer_amd import mscl as M
from test_feedforward_edges_gpu import BACK, guarded, within
from test_feedforward_gpu import ACTS, gated_case, normal, note, placed

pytestmark = pytest.mark.gpu
SIZES = [size[:3] for size in P.SIZES]


@pytest.fixture(scope="module", autouse=True)
def gpu():
    assert torch.cuda.is_available(), "GPU tests need a visible GPU"
    M.load()
    yield


def bits(t):
    return t.view(torch.int32)


def same(a, b):
    return all(torch.equal(bits(x), bits(y)) for x, y in zip(a, b))


def assert_in_range(got, want, name):
    """assert_within, but a value past binary32's range is not finite: its terms (2^108 times 2^40, say) already are
    infinities, of both signs, whose sum is an infinity or a NaN."""
    exact, bound = want
    past = exact.abs() > torch.finfo(torch.float32).max * (1 + 2.0 ** -20)
    assert not bool(torch.isfinite(got[past]).any()), name
    F.assert_within(got.masked_fill(past, 0), (exact.masked_fill(past, 0), bound), name)


def inputs(seed, m, k, n, bias=False):
    gen = torch.Generator().manual_seed(seed)
    x, wg, wu, bg, bu = gated_case(gen, m, k, n, torch.float32, bias=bias)
    return (x, wg, wu, bg, bu), [normal(gen, m, n, scale=s) for s in (1.0, 1.5, 1.0)]


@pytest.mark.parametrize("m,k,n", SIZES)
@pytest.mark.parametrize("form", ["plain", "columns", "odd"])
def test_forward_and_gradients(m, k, n, form):
    act = ACTS[(m + len(form)) % len(ACTS)]
    args, (dy, z, v) = inputs(101, m, k, n, bias=True)
    c = [a.cuda() for a in args]
    note("binary32 parts", m, k, n, form, act)
    there = [placed(a, form) for a in args]
    got = M.gated_linear_tensors(*there, act, return_preacts=True)
    within(got, F.gated_linear(*c, act), ("y", "gate", "up"))
    assert same([M.gated_linear_tensors(*there, act)], got)
    note("binary32 parts, gradients", m, k, n, form, act)
    there = [placed(dy, form), *there[:3], placed(z, form), placed(v, form), act]
    got = M.gated_linear_backward_tensors(*there)
    within(got, F.gated_linear_backward(dy.cuda(), *c[:3], z.cuda(), v.cuda(), act), BACK)
    for only, at in (("dx", (0,)), ("dw", (1, 2))):
        one = M.gated_linear_backward_tensors(*there, **{f"need_{o}": o == only for o in ("dx", "dw", "db")})
        assert same([one[i] for i in at], [got[i] for i in at])


@pytest.mark.parametrize("m,k,n", SIZES[:5])
def test_infinities_nan_and_far_values(m, k, n):
    """What the parts of a value cannot hold: waves with such sums add them again in binary32, each share for itself."""
    (x, wg, wu, _, _), (dy, z, v) = inputs(102, m, k, n)
    x[5, 3], x[7, k - 1], wu[11, 40] = math.inf, math.nan, -math.inf
    x[9] *= 2.0 ** 108  # no parts
    x[13] *= 2.0 ** 60  # parts, but with the row below sums from 2^80 on
    wg[17] *= 2.0 ** 40
    x[300:, 40] = x[300:, 40].abs() + 1
    x[:300, 40] = -x[:300, 40].abs() - 1
    note("binary32 parts with infinities", m, k, n)
    c = [a.cuda() for a in (x, wg, wu)]
    y, gate, up = M.gated_linear_tensors(*c, activation="none", return_preacts=True)
    assert same(M.gated_linear_tensors(*c, activation="none", return_preacts=True), (y, gate, up))
    bad = torch.zeros(m, n, dtype=torch.bool)
    bad[[5, 7]] = True
    assert not bool(torch.isfinite(gate.cpu()[bad]).any()) and bool(torch.isnan(gate[7]).all())
    assert torch.equal(up[300:, 11].cpu(), torch.full((m - 300,), -math.inf))
    ok = [i for i in range(m) if i not in (5, 7)]
    cols = [i for i in range(n) if i != 11]
    _, want_gate, want_up = F.gated_linear(c[0][ok], c[1][cols], c[2][cols], None, None, "none")
    assert_in_range(gate[ok][:, cols], want_gate, "gate")
    assert_in_range(up[ok][:, cols], want_up, "up")

    note("binary32 parts with infinities, gradients", m, k, n)
    (x, wg, wu, _, _), _ = inputs(103, m, k, n)
    dy[5, 3], dy[7, 12] = math.inf, math.nan
    dy[9] *= 2.0 ** 108
    dy[m - 1] *= 2.0 ** 58
    wg[:, k - 2] *= 2.0 ** 40
    c = [a.cuda() for a in (dy, x, wg, wu, z, v)]
    got = M.gated_linear_backward_tensors(*c, "none")
    assert same(M.gated_linear_backward_tensors(*c, "none"), got)
    assert not bool(torch.isfinite(got[0][[5, 7]]).any()) and not bool(torch.isfinite(got[1][[3, 12]]).any())
    rows = [c[0][ok], c[1][ok], c[2], c[3], c[4][ok], c[5][ok]]
    assert_in_range(got[0][ok], F.gated_linear_backward(*rows, "none")[0], "dx")
    cols = [i for i in range(n) if i not in (3, 12)]
    some = [c[0][:, cols], c[1], c[2][cols], c[3][cols], c[4][:, cols], c[5][:, cols]]
    want = F.gated_linear_backward(*some, "none")
    for g, w, name in zip(got[1:], want[1:], BACK[1:]):
        assert_in_range(g[cols], w, name)


@pytest.mark.parametrize("m,k,n", SIZES[:2] + SIZES[3:4])
def test_what_lies_around_the_matrices(m, k, n):
    """NaN behind the inputs reaches no result; through the C ABI, what lies beside the outputs stays as it is."""
    (x, wg, wu, bg, bu), (dy, z, v) = inputs(104, m, k, n, bias=True)
    x, wg, wu, dy, z, v = (guarded(a) for a in (x, wg, wu, dy, z, v))
    bg, bu = bg.cuda(), bu.cuda()
    lib = M.load()
    stream = torch.cuda.current_stream().cuda_stream
    wide = n + 7
    room = [torch.full((m + 1, wide), 77.0, device="cuda") for _ in range(3)]
    call = M.GATED_LINEAR.pack(x.data_ptr(), k, wg.data_ptr(), k, wu.data_ptr(), k, bg.data_ptr(), bu.data_ptr(),
                               *[a for r in room for a in (r.data_ptr() + 12, wide)], m, k, n, M.FLOAT32, M.ACT_GELU)
    note("binary32 parts, strided outputs", m, k, n)
    space, size = M._workspace(lib.mscl_gated_linear_workspace, call, x)
    M._check(lib.mscl_gated_linear(call, M._address(space), size, stream), "gated")
    for r, e, name in zip(room, F.gated_linear(x, wg, wu, bg, bu, "gelu"), ("y", "gate", "up")):
        F.assert_within(r[:m, 3:3 + n], e, name)
        assert bool((r[:, :3] == 77).all()) and bool((r[:, 3 + n:] == 77).all()) and bool((r[m] == 77).all())

    dw = torch.full((2 * n + 1, k + 5), 55.0, device="cuda")
    dx = torch.full((m + 1, k + 5), 55.0, device="cuda")
    db = torch.empty(2, n, device="cuda")

    def backward(dx_at, dg_at, du_at, db_at, pitch):
        call = M.GATED_LINEAR_BACKWARD.pack(
            dy.data_ptr(), n, x.data_ptr(), k, wg.data_ptr(), k, wu.data_ptr(), k, z.data_ptr(), n, v.data_ptr(), n,
            dx_at, pitch, dg_at, pitch, du_at, pitch, *db_at, m, k, n, M.FLOAT32, M.ACT_GELU)
        space, size = M._workspace(lib.mscl_gated_linear_backward_workspace, call, x)
        M._check(lib.mscl_gated_linear_backward(call, M._address(space), size, stream), "gated backward")
        return size

    note("binary32 parts, strided gradients", m, k, n)
    both = backward(dx.data_ptr() + 8, dw.data_ptr() + 4, dw.data_ptr() + (n * (k + 5) + 1) * 4,
                    (db[0].data_ptr(), db[1].data_ptr()), k + 5)
    want = F.gated_linear_backward(dy, x, wg, wu, z, v, "gelu")
    within((dx[:m, 2:2 + k], dw[:n, 1:1 + k], dw[n:2 * n, 1:1 + k], db[0], db[1]), want, BACK)
    assert bool((dx[:, :2] == 55).all()) and bool((dx[:, 2 + k:] == 55).all()) and bool((dx[m] == 55).all())
    assert bool((dw[:, :1] == 55).all()) and bool((dw[:, 1 + k:] == 55).all()) and bool((dw[2 * n] == 55).all())
    # one weight's gradient alone has the same bits
    one = torch.empty(n, k, device="cuda")
    for gate in (True, False):
        one.fill_(99)
        note("binary32 parts, one weight's gradient", m, k, n, gate)
        assert backward(0, one.data_ptr() if gate else 0, 0 if gate else one.data_ptr(), (0, 0), k) <= both
        assert torch.equal(one, dw[:n, 1:1 + k] if gate else dw[n:2 * n, 1:1 + k])


def _run(x, wg, wu, bg, bu, dy):
    y, z, v = M.gated_linear_tensors(x, wg, wu, bg, bu, return_preacts=True)
    return (y, z, v, *M.gated_linear_backward_tensors(dy, x, wg, wu, z, v))


@pytest.mark.parametrize("m,k,n", SIZES[:4])
def test_repeated_calls_and_graph_replays(m, k, n):
    """Over workspaces that held something else before, and in a captured graph among eager work."""
    args, (dy, _, _) = inputs(105, m, k, n, bias=True)
    args = [a.cuda() for a in (*args, dy)]
    note("binary32 parts, repeated", m, k, n)
    first = _run(*args)
    for fill in (math.nan, -math.inf):
        dirt = [torch.full((1 << 25,), fill, device="cuda") for _ in range(6)]
        del dirt
        assert same(first, _run(*[a.clone() for a in args]))
    note("binary32 parts, graph", m, k, n)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = _run(*args)
    gen = torch.Generator().manual_seed(106)
    for _ in range(3):
        args[0].copy_(normal(gen, m, k))
        args[5].copy_(normal(gen, m, n))
        graph.replay()
        got = [o.clone() for o in out]
        torch.cuda.synchronize()
        assert same(got, _run(*args))


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from allreduce_emulated_peer_amd import mscl as M
x, wg, wu = (torch.randn(2048, 2048, device="cuda") for _ in range(3))
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, z, v = M.gated_linear_tensors(x, wg, wu, return_preacts=True)
    d = M.gated_linear_backward_tensors(y, x, wg, wu, z, v)
for _ in range(3):
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, M.gated_linear_tensors(x, wg, wu))
    for a, b in zip(d, M.gated_linear_backward_tensors(y, x, wg, wu, z, v)):
        assert torch.equal(a, b)
print("captured first")
"""


def test_the_first_call_of_a_process_can_be_captured():
    assert (2048, 2048, 2048) in SIZES
    note("binary32 parts, first call captured")
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    out = subprocess.run([sys.executable, "-c", FIRST.format(root=root)], capture_output=True, text=True, timeout=110)
    assert out.returncode == 0 and "captured first" in out.stdout, out.stderr[-2000:]
