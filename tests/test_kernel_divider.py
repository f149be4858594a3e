"""The grouped WGrad decodes its tiles with multiplications in place of divisions
(csrc/fp8q_gemm.cu, Divider): for a divisor d, with 2^s the first power of two from d on,
n / d = (umulhi(m, n) + n) >> s, m = floor(2^32 (2^s - d) / d) + 1. The same arithmetic here,
against integer division."""
import numpy as np
import pytest


def divider(d):
    s = 0
    while (1 << s) < d:
        s += 1
    m = (((1 << s) - d) << 32) // d + 1
    assert m < 1 << 32
    return m, s


def quotient(n, m, s):
    total = ((np.uint64(m) * n) >> np.uint64(32)) + n
    assert total.max() < 1 << 32        # the device adds in 32 bits
    return total >> np.uint64(s)


@pytest.mark.parametrize("divisors", [range(1, 4097), [2**k + j for k in range(12, 31) for j in (-1, 0, 1)],
                                      [2**31 - 1, 2**31 - 2, 3**19, 10**9 + 7, 641 * 6700417 // 7]])
def test_divider(divisors):
    rng = np.random.RandomState(11)
    top = 2**31 - 1
    fixed = np.array([0, 1, 2, 127, 128, top - 1, top], np.uint64)
    for d in divisors:
        if d > top:
            continue
        near = (np.array([1, 2, 3, 1000, top // d], np.uint64) * np.uint64(d))
        near = np.concatenate([near - np.uint64(1), near, near + np.uint64(d - 1)])
        n = np.concatenate([fixed, near[near <= top], rng.randint(0, top, 400).astype(np.uint64)])
        assert np.array_equal(quotient(n, *divider(d)), n // np.uint64(d)), d
