"""The case of weight_pieces tells weights of three bf16 pieces from weights of two (CPU)."""
import pytest
import torch

from weight_pieces import BOUND, bf16, heads, pieces, result, weight


@pytest.mark.parametrize("d", [64, 128])
def test_two_pieces_fail_and_three_pass(d):
    b = heads(d)
    assert len(b) >= 8
    p = weight(b, d)
    exact = result(p)
    for n, x in enumerate(pieces(p), 1):
        # the sum of the weights takes p itself, the product with V its pieces
        err = ((3 * x / (1 + 3 * p)) - exact).abs() / exact
        assert (err <= BOUND / 4).all() if n == 3 else (err > 3 * BOUND).all()
    assert torch.equal(b, bf16(b))
