"""What the operators' contract says about their arithmetic, in 64 bits on the CPU."""

import os

import torch


def parts(v):
    """A binary32 value as the products take it: multiplied by 2^24, then three bfloat16 parts (here scaled back)."""
    rest, out = v * 2.0 ** 24, []
    for _ in range(3):
        near = rest.bfloat16().float()
        out.append(near.double() * 2.0 ** -24)
        rest = rest - near
    return out


def left_out(x, w):
    """What the six products of the larger parts leave out of x w, relative to it."""
    a, b = parts(x), parts(w)
    kept = sum(a[i] * b[j] for i in range(3) for j in range(3 - i))
    exact = x.double() * w.double()
    return ((exact - kept) / exact).abs()


def values(gen, n, low, high):
    size = torch.randint(low, high, (n,), generator=gen).double()
    return ((1 + torch.rand(n, generator=gen, dtype=torch.float64)) * 2.0 ** size).float()


def test_three_parts_hold_every_binary32_value():
    gen = torch.Generator().manual_seed(60)
    v = torch.cat([values(gen, 200000, -149, 103), torch.tensor([2.0 ** -149, 3 * 2.0 ** -149, 2.0 ** -126])])
    assert torch.equal(sum(parts(v)), v.double())


def test_products_of_parts_stay_within_the_stated_bound():
    gen = torch.Generator().manual_seed(61)
    bound = 2.0 ** -24 + 2.0 ** -34
    x, w = values(gen, 1 << 20, -40, 40), values(gen, 1 << 20, -40, 40)
    assert float(left_out(x, w).max()) <= bound
    # the largest smaller parts: 1 + 2^-8 - 2^-17 is split into 1, 2^-8 and -2^-17
    worst = torch.tensor([1 + 2.0 ** -8 - 2.0 ** -17, 1 + 2.0 ** -8 - 2.0 ** -17 + 2.0 ** -23])
    assert float(left_out(worst, worst).max()) <= bound
    assert float(left_out(worst, worst).max()) > 0.98 * 2.0 ** -24


def header():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with open(os.path.join(root, "include", "mscl.h")) as f:
        return " ".join(f.read().replace("*", " ").split())


def test_the_header_states_that_bound():
    assert "to within 2^-24 + 2^-34 of each product" in header()


def test_the_header_names_what_fixes_the_order_of_sums():
    assert "order fixed by the sizes, the strides and the pointers' alignment" in header()
