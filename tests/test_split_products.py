"""The arithmetic of fp32 products on bf16 tensor cores, emulated on the host: an operand as
three bf16 parts, and the six products of parts that are kept."""
import numpy as np
import pytest
import torch


def bf16(x):
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).float().numpy()


def parts(x):
    """x0 = bf16(x), x1 = bf16(x - x0), x2 = bf16(x - x0 - x1), differences in fp32."""
    x0 = bf16(x)
    r = x - x0
    x1 = bf16(r)
    return x0, x1, bf16(r - x1)


def values(n, seed, narrow):
    """fp32 values of either sign over many binades; narrow: mantissas just above a power of two,
    where a part's rounding is largest against the value."""
    rs = np.random.RandomState(seed)
    low = rs.randint(0, 1 << (16 if narrow else 23), n).astype(np.uint32)
    bits = (rs.randint(127 - 60, 127 + 60, n).astype(np.uint32) << 23) | low | (rs.randint(0, 2, n).astype(np.uint32) << 31)
    return bits.view(np.float32)


@pytest.mark.parametrize("narrow", [False, True])
def test_three_parts_hold_the_value(narrow):
    # 8 significant bits each: |x - x0| <= 2^-8 and |x - x0 - x1| <= 2^-17 of x's power of two, and
    # what is left is a multiple of x's last bit, 2^-23, so at most 64 of them: seven bits
    x = values(1 << 20, 1, narrow)
    x0, x1, x2 = (p.astype(np.float64) for p in parts(x))
    assert np.array_equal(x0 + x1 + x2, x.astype(np.float64))
    two = 2.0 ** np.floor(np.log2(np.abs(x.astype(np.float64))))
    assert np.all(np.abs(x1) <= 2.0 ** -8 * two) and np.all(np.abs(x2) <= 2.0 ** -17 * two)


@pytest.mark.parametrize("narrow", [False, True])
def test_kept_products_are_within_half_a_step_of_fp32(narrow):
    # left out: x1 y2 + x2 y1 + x2 y2, at most 2 * 2^-8 * 2^-17 + 2^-34 of both powers of two, and so
    # of the product: 2^-24 (1 + 2^-10)
    worst = 0.0
    for seed in range(8):
        x, y = values(1 << 20, 2 * seed + 2, narrow), values(1 << 20, 2 * seed + 3, narrow)
        x0, x1, x2 = (p.astype(np.float64) for p in parts(x))
        y0, y1, y2 = (p.astype(np.float64) for p in parts(y))
        exact = x.astype(np.float64) * y.astype(np.float64)
        left_out = x1 * y2 + x2 * y1 + x2 * y2
        kept = exact - left_out  # (the products of parts, and these few sums, are exact to 2^-52)
        assert np.allclose(x0 * y0 + (x0 * y1 + x1 * y0) + (x1 * y1 + x0 * y2 + x2 * y0), kept, rtol=2.0 ** -50, atol=0)
        worst = max(worst, np.abs(left_out / exact).max())
    assert worst <= 2.0 ** -24 * (1 + 2.0 ** -10)
    if narrow:
        assert worst > 2.0 ** -25  # a bound of 2^-25 would be too small
