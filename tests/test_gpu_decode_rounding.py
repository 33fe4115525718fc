"""Verification by the formula's own roundings: remainders of a row that are exactly
0 as products and differences in float64, and not where a product is kept unrounded."""
import numpy as np
import pytest

from oracle import decode_oracle as D
from tests.test_gpu_decode import _ivc, _verify_check


def _rows():
    """(p, q) where, once token 0 is rejected, r / z is q / w for each of the m tokens
    left: r = a / den, q = d / den each, all exact in fp32. The three children's
    tokens are 0, 0 again (which leaves a remainder of exactly 0) and 1."""
    for den in (16, 32, 64):
        for a in range(1, den):
            for d in range(1, den):
                for m in (2, 3, 5, 6, 7):
                    if m * d >= den or m * (a + d) >= den:
                        continue
                    z, w = m * a / den, m * d / den
                    if (a / den) * (1 / z) - (d / den) * (1 / w) != 0.0:
                        continue             # not 0 in separately rounded float64
                    rest = np.full(m, 1.0)
                    p = np.concatenate([[1 - m * (a + d) / den], rest * (a + d) / den])
                    q = np.concatenate([[1 - m * d / den], rest * d / den])
                    if p[0] < q[0]:
                        yield p, q


def test_formula_leaves_nothing_there():
    """The oracle: no third child, and the next token from the node's own row."""
    count = 0
    for p, q in _rows():
        p, q = (np.repeat(x[None], 4, 0) for x in (p, q))
        path, token = D.verify(p, q, [0, 0, 0, 1], [-1, 0, 0, 0], [0, 0.99, 0.99, 0.99], p[0, 0] / 2)
        assert path == [0] and token == 0
        count += 1
    assert count > 400


@pytest.mark.gpu
@pytest.mark.parametrize("V", [8, 5000])
def test_verification_rounds_as_the_formula_does(V):
    rows = list(_rows())
    if V > 8:
        rows = rows[::7]
    B = len(rows)
    p, q = np.zeros((4 * B, V), np.float32), np.zeros((4 * B, V), np.float32)
    at = np.linspace(0, V - 1, 8).astype(int)  # the tokens, over the whole vocabulary
    for b, (x, y) in enumerate(rows):
        p[4 * b:4 * b + 4, at[:len(x)]] = x
        q[4 * b:4 * b + 4, at[:len(x)]] = y
    tok = np.tile([0, at[0], at[0], at[1]], B).astype(np.int32)
    u = np.tile([0, 0.99, 0.99, 0.99], B).astype(np.float32)
    un = np.array([x[0] / 2 for x, _ in rows], np.float32)
    off = 4 * np.arange(B + 1, dtype=np.int32)
    _verify_check(_ivc(), p, q, tok, [[-1, 0, 0, 0]] * B, off, u, un, width=4)
