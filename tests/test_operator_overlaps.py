"""Which outputs may lie between each other's rows, on the CPU: validation alone, nothing reaches a GPU call."""

import ctypes
import random

from allreduce_emulated_peer_amd import mscl as M

A, FAR = 1 << 40, 1 << 36


def status(y, y_stride, z, z_stride, rows, cols):
    """Of a linear call whose y and preact are at elements `y` and `z` of one float32 buffer."""
    call = M.LINEAR.pack(A + FAR, 4, A + 2 * FAR, 4, 0, 0, 0, A + 4 * y, y_stride, A + 4 * z, z_stride, rows, 4, cols, M.FLOAT32,
                         M.ACT_GELU)
    need = ctypes.c_size_t()
    return M.load().mscl_linear_workspace(call, ctypes.byref(need))


def test_column_blocks_of_one_matrix_do_not_overlap():
    rows, cols, stride = 50, 24, 60
    assert status(0, stride, 24, stride, rows, cols) == M.SUCCESS
    assert status(36, stride, 0, stride, rows, cols) == M.SUCCESS
    assert status(40, stride, 4, stride, rows, cols) == M.SUCCESS
    assert status(0, stride, 23, stride, rows, cols) == M.ERR_INVALID_ARGUMENT  # one column in both
    assert "overlap" in M.last_error_string()
    assert status(0, stride, 37, stride, rows, cols) == M.ERR_INVALID_ARGUMENT  # into the next row's first column
    assert status(0, stride, 24, stride + 1, rows, cols) == M.ERR_INVALID_ARGUMENT  # rows that drift into each other


def test_against_the_elements_themselves():
    rng = random.Random(70)
    seen = set()
    for _ in range(4000):
        rows, cols = rng.choice([1, 1, 2, 3, 5]), rng.randint(1, 9)
        stride = rng.randint(cols, 2 * cols + 3)
        y, z = rng.randint(0, 40), rng.randint(0, 40)
        at = [{s + i * stride + j for i in range(rows) for j in range(cols)} for s in (y, z)]
        shared = bool(at[0] & at[1])
        seen.add((rows > 1, shared))
        assert (status(y, stride, z, stride, rows, cols) != M.SUCCESS) == shared, (rows, cols, stride, y, z)
    assert len(seen) == 4


def test_a_vector_between_the_rows_of_a_matrix():
    """bias and dbias have one row, whose length may exceed the other's stride."""
    rng = random.Random(71)
    lib, need, seen = M.load(), ctypes.c_size_t(), set()
    for _ in range(4000):
        rows, k, n = rng.randint(1, 4), rng.randint(1, 6), rng.randint(1, 12)
        stride, dx, db = rng.randint(k, k + 14), rng.randint(0, 40), rng.randint(0, 40)
        call = M.LINEAR_BACKWARD.pack(A + FAR, n, A + 2 * FAR, k, A + 3 * FAR, k, 0, 0, A + 4 * dx, stride, 0, 0, A + 4 * db,
                                      rows, k, n, M.FLOAT32, M.ACT_NONE)
        shared = bool({dx + i * stride + j for i in range(rows) for j in range(k)} & set(range(db, db + n)))
        seen.add((db < dx, shared))
        assert (lib.mscl_linear_backward_workspace(call, ctypes.byref(need)) != M.SUCCESS) == shared
    assert len(seen) == 4


def test_matrices_of_different_strides_must_lie_apart():
    assert status(0, 10, 40, 12, 4, 5) == M.SUCCESS
    assert status(0, 10, 34, 12, 4, 5) == M.ERR_INVALID_ARGUMENT
    assert status(0, 10, 5, 12, 4, 5) == M.ERR_INVALID_ARGUMENT
