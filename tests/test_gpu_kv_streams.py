"""The cache operators on a stream other than the current one, with outputs and
workspace of their own making."""
import pytest
import torch

import kv_reference as ref
import test_gpu_kv as kv
from speculative_decoding_verification_03_gb300 import binding

pytestmark = pytest.mark.gpu


def test_memory_of_calls_on_another_stream():
    """While the calls wait behind other work on their stream, the current stream takes
    and fills as much memory as they made: neither disturbs the other."""
    c = ref.Case([3000, 700], [3, 40], 8, 2, 128, 16, False, seed=41)
    cache = kv.gpu_cache(c)
    i32 = dict(dtype=torch.int32, device="cuda")
    q, q_start, kv_len, table = (x.cuda() for x in (c.q, c.q_start, c.kv_len, c.table))
    positions = torch.arange(c.T, **i32)
    plan = binding.RopePlan.make(128)
    kv_start = torch.tensor([0, 3000, 3700], **i32)
    own = binding.KVCache.empty(8, 16, 2, 128)
    k = torch.randn(c.T, 2, 128, device="cuda").bfloat16()
    rows = torch.arange(6, **i32).view(2, 3)
    zero = torch.zeros(2, **i32)

    def calls(**kw):
        return [*binding.paged_attention(q, cache, q_start, kv_len, table, **kw), binding.rope(q, positions, plan, **kw),
                binding.kv_append(own, k, k, q_start, zero, rows, q=q, plan=plan, **kw),
                *binding.kv_read(cache, kv_start, table, 3700, **kw)]

    want = calls()
    sizes = [binding.lib().sv_attention_workspace_bytes()] + [x.numel() * x.element_size() for x in want]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(2):  # (the second time from memory that either stream has had before)
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)
        got = calls(stream=side)
        mine = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in sizes for _ in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
        for x in mine:
            assert (x == 255).all()
        del got, mine
    kv.check_attention(c, *want[:2])
