"""The bounds of kv_bounds.py can fail: for every e4m3 case they refuse zeros and
outputs 2 % too small, in every element's place and in the norm, and take the exact
outputs rounded to bf16."""
import numpy as np
import pytest
import torch

from kv_bounds import E4M3_CASES, exact, faults


@pytest.mark.parametrize("name", list(E4M3_CASES))
def test_bounds_refuse_wrong_outputs(name):
    c = E4M3_CASES[name]()
    reference = exact(c)
    want, lse = reference[0], reference[1]
    rounded = torch.tensor(want).bfloat16().double().numpy()
    assert faults(c, rounded, lse, reference) == []
    assert faults(c, np.zeros_like(want), lse, reference)
    assert faults(c, want * 0.98, lse, reference)
    assert faults(c, want * 1.02, lse, reference)
    assert faults(c, want, lse + 0.1, reference)
    if sum(c.chunks) > 1:  # a row in another's place
        assert faults(c, np.roll(want, 1, 0), lse, reference)
