"""The limits that fp32 gradients are held to: the six partial products of a product
stay far below them, and any five of them go beyond."""
import pytest

from oracle.split import PRODUCTS, SPLIT_CASES, SPLIT_REL, SPLIT_RMS, split_exact, split_inputs


@pytest.mark.parametrize("n,vocab,width", SPLIT_CASES)
def test_a_partial_product_left_out_shows(n, vocab, width):
    x = split_inputs(n, vocab, width)
    want = split_exact(*x)

    def off(products):
        logp, dh, dw = split_exact(*x, products)
        return ((logp - want[0]).norm() / len(logp) ** 0.5 / SPLIT_RMS, (dh - want[1]).norm() / want[1].norm() / SPLIT_REL,
                (dw - want[2]).norm() / want[2].norm() / SPLIT_REL)

    assert max(off(PRODUCTS)) < 0.1
    for left_out in PRODUCTS:
        assert min(off([p for p in PRODUCTS if p != left_out])) > 3, left_out
