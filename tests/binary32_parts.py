"""Sizes at which the gated block's binary32 products take their operands into bfloat16 parts once, in the workspace.

Each is (rows, in_features, out_features, shares of k forward, of the input
gradient, of the weights' gradients), where 0 shares mean that small tiles run
that product.  The library chooses by an estimate of time; what it asks for as
workspace shows the choice, and test_binary32_parts.py holds these sizes to it.
"""

SIZES = [
    (2041, 2043, 2045, 2, 4, 2),
    (4089, 1019, 4090, 1, 4, 2),
    (3100, 2045, 2040, 1, 0, 2),
    (8190, 2040, 505, 2, 1, 0),
    (2046, 3838, 3838, 1, 2, 1),
    (2048, 2048, 2048, 2, 4, 2),
]


def _up(v, to):
    return -(-v // to) * to


def _parts(rows, cols):
    """Bytes of a matrix in three parts, rows at 128-byte boundaries."""
    return 3 * _up(rows * _up(cols, 64) * 2, 256)


def _shares(shares, rows, cols):
    """Bytes of the shares' sums; the last row's padding may be left out."""
    return 4 * shares * rows * _up(cols, 8) if shares > 1 else 0


def forward_bytes(rows, k, n, shares):
    return _parts(rows, k) + 2 * _parts(n, k) + 2 * _shares(shares, rows, n) if shares else 0


def gradient_bytes(rows, k, n, dx, dw):
    """dz and dv side by side and in parts, and what the products of `dx` and `dw` shares take (None: not wanted)."""
    both = 2 * _up(n, 128)
    need = 4 * rows * both
    if dx or dw:
        need += _parts(rows, both)
    if dx:
        need += 2 * _parts(n, k) + _shares(dx, rows, k)
    if dw:
        need += _parts(rows, k) + 2 * _shares(dw, n, k)
    return need
