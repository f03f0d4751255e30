"""Queries with a large channel beside many small ones, over e4m3 caches."""
import numpy as np
import pytest
import torch

import kv_reference as ref
import test_gpu_kv as kv
from speculative_decoding_verification_03_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("small", [0.0107421875, 0.0034, 0.3])
@pytest.mark.parametrize("tokens", [6, 25, 50])  # 24, 100, 200 rows of a key head: narrow, wide, pair
def test_query_outliers(tokens, small):
    """Scores come from the small channels (the large one meets zeros).  A query's
    value may be off by 2^-21 of its row's largest: scores by that times the sum of
    |k|, beside the roundings of D fp32 sums; a score's error changes its weight by
    that factor; the weight is rounded to 8 bits and the output to bf16."""
    D, G, Hkv = 128, 4, 2
    c = ref.Case([700, 90], [tokens, tokens], G * Hkv, Hkv, D, 16, True, seed=tokens)
    rng = np.random.default_rng(tokens)
    sign = np.where(rng.random(D) < 0.5, -1.0, 1.0)
    q = small * sign * (1 + (np.arange(c.T * G * Hkv).reshape(c.T, -1, 1) % 5) / 16)
    q[..., 0] = 256.0
    c.q = torch.tensor(q).bfloat16()
    count = c.cache["k"].shape[0]
    k = (0.3 / small) * sign * rng.standard_normal((count, 16, Hkv, 1)) * (1 + 0.2 * rng.standard_normal((count, 16, Hkv, D)))
    k[..., 0] = 0.0
    code, byte = ref.quantise(k)
    c.cache["k"] = torch.tensor(code).float().to(torch.float8_e4m3fn)
    c.cache["k_exp"] = torch.tensor(byte).to(torch.uint8).transpose(1, 2).contiguous()
    c.values[0] = code * np.exp2(byte - 127.0)[..., None]
    out, lse, ws = kv.run_attention(c)
    assert binding.status(ws) == (0, 0)
    want, wl, mag, noise = c.attention()
    reach = np.zeros_like(wl)  # |scale| max |q| sum |k|, the largest of a key head's slots
    for b in range(c.B):
        s = slice(int(c.q_start[b]), int(c.q_start[b + 1]))
        keys = np.repeat(np.abs(c.rows(0, b)).sum(-1).max(0), G)
        reach[s] = D ** -0.5 * np.abs(c.q[s].double().numpy()).max(-1) * keys
    ds = (D + 4) * 2.0 ** -24 * noise + 2.0 ** -21 + 2.0 ** -21 * reach
    tol = (2.0 ** -8 + 2 * ds + 2.0 ** -18)[..., None] * mag + 2.0 ** -8 * np.abs(want)
    got, gl = out.cpu().double().numpy(), lse.cpu().double().numpy()
    assert np.isfinite(got).all()
    assert (np.abs(gl - wl) <= ds + np.abs(wl) * 2.0 ** -22).all(), (np.abs(gl - wl) / ds).max()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()
