"""Values of far larger scale than the others', over e4m3 caches: in a slot of
little weight, or one that a row does not see, they leave the others' weights alone."""
import numpy as np
import pytest
import torch

import kv_bounds
import kv_reference as ref
import test_gpu_kv as kv
from speculative_decoding_verification_03_gb300 import binding

pytestmark = pytest.mark.gpu


def scaled(c, slots, bits):
    """The values of sequence 0's `slots` times 2^bits."""
    for j in slots:
        p, s = int(c.table[0, j // c.page]), j % c.page
        c.cache["v_exp"][p, :, s] += bits
        c.values[1][p, s] *= 2.0 ** bits


def floor(c):
    """What the outputs may be off by beside 2^-8 of each weight: a weight loses at most
    all of itself, and at most 2^-25 of its row's largest times the largest power of two
    among the 128 slots that it lies with, over its own value's."""
    n, G = c.T, c.Hq // c.Hkv
    out = np.zeros((n, c.Hq, c.D))
    k, v = c.rows(0, 0), np.abs(c.rows(1, 0))
    own = np.ceil(np.log2(v.max(-1) / 448.0))  # (a row's largest code is in (224, 448])
    most = own.copy()
    for i in range(0, len(v), 128):
        most[i:i + 128] = own[i:i + 128].max(0)
    see, q = ref.visible(n, c.lens[0]), c.q.double().numpy()
    for h in range(c.Hq):
        s = np.where(see, c.D ** -0.5 * (q[:, h] @ k[:, h // G].T), -np.inf)
        p = np.exp(s - s.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
        off = np.minimum(p, p.max(1, keepdims=True) * np.exp2(most - own - 25)[:, h // G])
        out[:, h] = off @ v[:, h // G]
    return out


COPIES = 304  # as many sequences as there are groups, so that no item is cut


def run(c):
    """The one sequence of c, COPIES times over the same pages."""
    ws = binding.attention_workspace()
    got = binding.paged_attention(c.q.repeat(COPIES, 1, 1).cuda(), kv.gpu_cache(c),
                                  torch.arange(COPIES + 1, dtype=torch.int32).cuda() * c.T, c.kv_len.repeat(COPIES).cuda(),
                                  c.table.repeat(COPIES, 1).cuda(), workspace=ws)
    assert binding.status(ws) == (0, 0)
    return got


def check(c):
    out, lse = (x.cpu().double().numpy() for x in run(c))
    want, wl, mag, dev, ds = kv_bounds.exact(c)
    got, gl = out.reshape((COPIES,) + want.shape), lse.reshape((COPIES,) + wl.shape)
    tol = (2.0 ** -8 + 2.0 ** -18) * mag + 2 * ds[..., None] * dev + 2.0 ** -8 * np.abs(want) + floor(c)
    assert np.isfinite(got).all()
    assert (np.abs(gl - wl) <= ds + np.abs(wl) * 2.0 ** -22).all()
    assert (np.abs(got - want) <= tol).all(), (np.abs(got - want) / tol).max()


@pytest.mark.parametrize("bits", [12, 20, 28])
@pytest.mark.parametrize("tokens", [5, 25, 50])
def test_large_values_of_no_weight(tokens, bits):
    """One large value early on, which no query looks at; forty tiles follow."""
    c = ref.Case([6000], [tokens], 4, 1, 64, 16, True, seed=tokens)
    c.q = c.q.abs()
    p, s = int(c.table[0, 0]), 5
    c.cache["k"].view(torch.uint8)[p, s] = 0xFE  # -448: its scores are far below all others
    c.cache["k_exp"][p, :, s] = 127
    c.values[0][p, s] = -448.0
    scaled(c, [5], bits)
    check(c)


@pytest.mark.parametrize("tokens", [5, 25, 50])
def test_larger_values_unseen(tokens):
    """Each token's value 2^3 times the one's before it, for five tokens of the chunk."""
    c = ref.Case([1300], [tokens], 4, 1, 64, 16, True, seed=tokens)
    for i in range(5):
        scaled(c, [1300 + i], 3 * i)
    check(c)


@pytest.mark.parametrize("tokens", [5, 25, 50])
def test_scales_that_fall_and_rise(tokens):
    """Tiles whose values are 2^40 times others', in turns."""
    c = ref.Case([3000], [tokens], 4, 1, 64, 16, True, seed=tokens)
    scaled(c, [j for j in range(3000) if j // 128 % 3 == 1], 20)
    scaled(c, [j for j in range(3000) if j // 128 % 3 == 2], -20)
    check(c)


@pytest.mark.parametrize("first", [100, 40])
@pytest.mark.parametrize("tokens", [5, 25, 50])
def test_scales_that_fall_far(tokens, first):
    """Values fall by 2^50 a tile, three times: the largest stay what they are."""
    c = ref.Case([600], [tokens], 4, 1, 64, 16, True, seed=tokens)
    for t in range(5):
        scaled(c, range(128 * t, min(128 * (t + 1), 600)), max(first - 50 * t, first - 150))
    check(c)
