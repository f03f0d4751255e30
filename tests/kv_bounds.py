"""Batches whose rows give one slot much of their weight and thousands of slots
the rest, and bounds that allow nothing absolutely: a small weight keeps its bits."""
import math

import numpy as np
import torch

import kv_reference as ref
from speculative_decoding_verification_03_gb300 import binding


class Sink:
    """`batch` sequences over the same pages: slot 0 takes about `share` of a
    row's weight and has small values, the other slots share the rest, their
    scores `spread` (log2) apart and their values around 1.  A row's share
    varies with its query's size."""

    def __init__(self, slots, share, spread, tokens, batch, G=4, D=128, page=64, seed=0):
        rng = np.random.default_rng(seed)
        self.tokens, self.batch, self.Hq, self.D = tokens, batch, G, D
        n = slots + tokens
        pages = -(-n // page)
        sign = np.where(rng.random(D) < 0.5, -1.0, 1.0)
        per = math.sqrt(D)  # nats of a key of ones
        t = -0.125 + spread * math.log(2.0) * rng.standard_normal(pages * page) / per
        t[0] = (math.log(share / (1 - share) * n) + per * -0.125 + (spread * math.log(2.0)) ** 2 / 2) / per
        v = 1.0 + 0.1 * rng.standard_normal((pages * page, D))
        v[0] = 2.0 ** -6 * rng.standard_normal(D)
        store, self.values = {}, []
        for name, x in (("k", t[:, None] * sign), ("v", v)):
            code, byte = ref.quantise(x)
            self.values.append((code * np.exp2(byte - 127.0)[:, None])[:n])
            store[name] = torch.tensor(code).float().to(torch.float8_e4m3fn).view(pages, page, 1, D)
            store[name + "_exp"] = torch.tensor(byte).to(torch.uint8).view(pages, 1, page)
        self.store = store
        size = 1.0 + (np.arange(tokens * G) % 8).reshape(tokens, G, 1) / 64.0
        self.q = torch.tensor(size * sign).bfloat16()
        self.kv_len = slots

    def exact(self):
        """out, sum p |v|, the scores' terms and lse of one sequence, 64 bits."""
        k, v = self.values
        q = self.q.double().numpy()
        s = np.einsum("thd,nd->thn", q, k) / math.sqrt(self.D)
        see = np.arange(len(k)) <= self.kv_len + np.arange(self.tokens)[:, None, None]
        s = np.where(see, s, -np.inf)
        top = s.max(-1, keepdims=True)
        w = np.exp(s - top)
        l = w.sum(-1, keepdims=True)
        terms = np.abs(q).max(-1)[..., None] * np.abs(k).sum(-1) / math.sqrt(self.D)
        self.share = (w / l)[..., 0]
        return (w / l) @ v, (w / l) @ np.abs(v), terms.max(-1), (top + np.log(l))[..., 0]

    def check(self):
        """Run it; every sequence's rows against the one reference."""
        dev = {n: x.cuda() for n, x in self.store.items()}
        pages = dev["k"].shape[0]
        table = torch.arange(pages, dtype=torch.int32).repeat(self.batch, 1).cuda()
        q = self.q.repeat(self.batch, 1, 1).cuda()
        q_start = torch.arange(self.batch + 1, dtype=torch.int32).cuda() * self.tokens
        kv_len = torch.full((self.batch,), self.kv_len, dtype=torch.int32).cuda()
        ws = binding.attention_workspace()
        out, lse = binding.paged_attention(q, binding.KVCache(**dev), q_start, kv_len, table, workspace=ws)
        assert binding.status(ws) == (0, 0)
        want, mag, terms, wl = self.exact()
        # A score is a sum of D products in fp32 (D roundings of at most 2^-24 of the
        # terms' sum, 4 more for scaling and exponent) over queries within 2^-21 of
        # their row's largest; a weight is off by 2^-8 of it, the output is rounded to bf16.
        ds = (self.D + 4) * 2.0 ** -24 * terms + 2.0 ** -21 + 2.0 ** -21 * terms
        tol = (2.0 ** -8 + 2 * ds + 2.0 ** -18)[..., None] * mag + 2.0 ** -8 * np.abs(want)
        got = out.cpu().double().numpy().reshape((self.batch,) + want.shape)
        gl = lse.cpu().double().numpy().reshape((self.batch,) + wl.shape)
        assert np.isfinite(got).all()
        off = np.abs(got - want) / tol
        assert off.max() <= 1, "%.1f times the bound (%.3g of the output at its row)" % (
            off.max(), np.abs(got / want - 1).reshape(-1)[off.argmax()])
        assert (np.abs(gl - wl) <= ds + np.abs(wl) * 2.0 ** -22).all()
