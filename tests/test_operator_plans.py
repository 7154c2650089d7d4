"""What a call asks for as workspace, on the CPU: which kernels it would run shows there."""

import ctypes

import pytest

from allreduce_emulated_peer_amd import mscl as M

A = 1 << 40  # fake addresses: nothing here reaches a GPU call
FAR = 1 << 38


def linear_need(m, k, n, dtype=M.BFLOAT16, w_at=0, w_stride=None, x_stride=None):
    """Workspace of x (m, k) and w (n, k); `w_at`: bytes that w starts behind a 16-byte boundary."""
    call = M.LINEAR.pack(A, k if x_stride is None else x_stride, A + FAR + w_at, k if w_stride is None else w_stride, 0, 0, 0,
                         A + 2 * FAR, n, 0, 0, m, k, n, dtype, M.ACT_NONE)
    need = ctypes.c_size_t()
    M._check(M.load().mscl_linear_workspace(call, ctypes.byref(need)), "mscl_linear_workspace")
    return need.value


@pytest.mark.parametrize("m", [1, 16, 17, 32, 33, 128, 200, 257, 512, 700, 768])
@pytest.mark.parametrize("k,n", [(8192, 32768), (4096, 65536), (1000, 150001)])
def test_no_copy_of_a_weight_that_few_rows_use(m, k, n):
    for how in (dict(w_at=2), dict(w_stride=k + 3), dict(w_at=6, w_stride=k + 1)):
        assert linear_need(m, k, n, **how) < n * k * 2 // 4


def test_no_copy_of_rows_that_few_outputs_use():
    for n in (1, 40, 200, 700):
        assert linear_need(65536, 4096, n, x_stride=4099) < 65536 * 4096 * 2 // 4


def backward_need(m, k, n, dy_stride, x_stride, w_stride, dtype=M.BFLOAT16):
    call = M.LINEAR_BACKWARD.pack(A, dy_stride, A + FAR, x_stride, A + 2 * FAR, w_stride, 0, 0, A + 3 * FAR, k, A + 4 * FAR, k,
                                  A + 5 * FAR, m, k, n, dtype, M.ACT_NONE)
    need = ctypes.c_size_t()
    M._check(M.load().mscl_linear_backward_workspace(call, ctypes.byref(need)), "mscl_linear_backward_workspace")
    return need.value


@pytest.mark.parametrize("stride", [0, 1, 3, 1 << 40, (1 << 64) - 1])
def test_the_stride_of_a_single_row_changes_nothing(stride):
    """It is ignored, so a call is planned as with any other value there."""
    for m, k, n in ((1, 32768, 8192), (1, 4096, 4096), (1, 72, 40)):
        assert backward_need(m, k, n, stride, stride, k) == backward_need(m, k, n, n, k, k)
        assert linear_need(m, k, n, x_stride=stride) == linear_need(m, k, n)
    for m, k in ((300, 2048), (66000, 8192)):
        assert linear_need(m, k, 1, w_stride=stride) == linear_need(m, k, 1)
        assert backward_need(m, k, 1, 1, k, stride) == backward_need(m, k, 1, 1, k, k)
