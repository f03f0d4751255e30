"""Arguments of the cache operators that are refused before a launch."""
import pytest
import torch

import kv_reference as ref
import test_gpu_kv as kv
from speculative_decoding_verification_03_gb300 import binding

pytestmark = pytest.mark.gpu


def test_attention_workspace_refusals():
    c = ref.Case([5], [2], 4, 2, 64, 16, False, seed=17)
    args = (c.q.cuda(), kv.gpu_cache(c), c.q_start.cuda(), c.kv_len.cuda(), c.table.cuda())
    n = binding.lib().sv_attention_workspace_bytes()
    with pytest.raises(ValueError):
        binding.paged_attention(*args, workspace=torch.zeros(n, dtype=torch.uint8))  # on the host
    with pytest.raises(ValueError):
        binding.paged_attention(*args, workspace=torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2])
    with pytest.raises(TypeError):
        binding.paged_attention(*args, workspace=torch.zeros(n, dtype=torch.int32, device="cuda"))
    ws = torch.zeros(n + 256, dtype=torch.uint8, device="cuda")
    with pytest.raises(binding.SVError):
        binding.paged_attention(*args, workspace=ws[16:])
    out, lse = binding.paged_attention(*args, workspace=ws)
    kv.check_attention(c, out, lse)
