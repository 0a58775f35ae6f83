"""The bound that the layer for a few tokens is held to tells an h of one number from one of two, on the inputs that
the GPU tests take (the mistake is planted in the 64-bit form)."""
import pytest
import torch

import few_ref as few

CASES = [(s, t, False) for s in few.SMALL for t in (0, 1)] + [(s, t, True) for s in few.LARGE for t in (0, 1)] + \
    [(s, 1, True) for s in few.LONG]


@pytest.mark.parametrize("shape,x_dtype,large", CASES, ids=str)
def test_one_number_breaks_the_bound(shape, x_dtype, large):
    t = few.inputs(shape, x_dtype)
    want, bound = few.layer(*t, torch.float32, large)
    held = torch.float16 if large else few.DT[x_dtype]
    one, _ = few.layer(*t, torch.float32, large, lambda h: h.to(held).double())
    assert not bool(((one - want).abs() <= bound).all())

    def two(h):
        first = h.to(held)
        return first.double() + (h - first.double()).to(held).double()
    both, _ = few.layer(*t, torch.float32, large, two)
    assert bool(((both - want).abs() <= bound).all())
