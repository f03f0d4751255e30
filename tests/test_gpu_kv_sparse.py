"""Batches most of whose sequences have no new tokens, or that mix prompts with
many single tokens: the same results, and no time for what has no tokens."""
import pytest
import torch

import kv_reference as ref
import test_gpu_kv as kv
from kv_bounds import exact, faults
from speculative_decoding_verification_03_gb300 import binding

pytestmark = pytest.mark.gpu

BATCHES = {
    "empty between": ([130] * 400, [3 if b in (0, 1, 33, 200, 201, 399) else 0 for b in range(400)]),
    "empty first": ([70] * 300, [0] * 299 + [2]),
    "empty last": ([70] * 300, [0, 2] + [0] * 298),
    "one prompt among tokens": ([90] * 200, [1] * 77 + [300] + [1] * 122),
    "prompts among empty": ([90] * 150, [140 if b in (0, 64, 65, 149) else (2 if b % 40 == 3 else 0) for b in range(150)]),
}


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name", list(BATCHES))
def test_sparse_batches(name, fp8):
    lens, chunks = BATCHES[name]
    c = ref.Case(lens, chunks, 8, 2, 64, 16, fp8, seed=51)
    out, lse, ws = kv.run_attention(c)
    assert binding.status(ws) == (0, 0)
    assert faults(c, out.cpu().double().numpy(), lse.cpu().double().numpy(), exact(c)) == []


@pytest.mark.parametrize("place", [0, 10000, 19999])
def test_empty_sequences_take_no_time(place):
    """One token among 20,000 sequences without: reading their lengths takes some tens of
    microseconds, a walk over them one by one takes 2800."""
    B = 20000
    i32 = dict(dtype=torch.int32, device="cuda")
    cache = binding.KVCache.empty(16, 16, 2, 64)
    q = torch.randn(1, 8, 64, device="cuda").bfloat16()
    q_start = torch.zeros(B + 1, **i32)
    q_start[place + 1:] = 1
    args = (q, cache, q_start, torch.full((B,), 100, **i32), torch.arange(16, **i32).repeat(B, 1))
    ws = binding.attention_workspace()
    binding.paged_attention(*args, workspace=ws)
    times = []
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(5):
            binding.paged_attention(*args, workspace=ws)
        b.record()
        torch.cuda.synchronize()
        times.append(a.elapsed_time(b) / 5)
    assert min(times) < 0.4, times
