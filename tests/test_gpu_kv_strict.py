"""Attention over e4m3 caches against bounds that a wrong output does not pass
(tests/test_kv_bounds.py shows that they can fail)."""
import pytest

import test_gpu_kv as kv
from kv_bounds import E4M3_CASES, exact, faults
from speculative_decoding_verification_03_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", list(E4M3_CASES))
def test_attention_e4m3(name):
    c = E4M3_CASES[name]()
    out, lse, ws = kv.run_attention(c)
    assert binding.status(ws) == (0, 0)
    assert faults(c, out.cpu().double().numpy(), lse.cpu().double().numpy(), exact(c)) == []
