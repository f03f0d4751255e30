"""Bounds on attention's outputs that allow nothing absolutely (a small weight
keeps its bits), the e4m3 cases that they are used on, and batches whose rows give one
slot much of their weight and thousands of slots the rest."""
import math

import numpy as np
import torch

import kv_reference as ref
from speculative_decoding_verification_03_gb300 import binding


def exact(c, scale=None):
    """A batch's exact outputs and what the bounds are made of, 64 bits: out, lse,
    sum p |v|, the values' deviation sqrt(sum p v^2 - out^2), and a bound on the scores' errors."""
    scale = c.D ** -0.5 if scale is None else scale
    G = c.Hq // c.Hkv
    q = c.q.double().numpy()
    out, mag, dev = (np.zeros((c.T, c.Hq, c.D)) for _ in range(3))
    lse, ds = np.full((c.T, c.Hq), -np.inf), np.zeros((c.T, c.Hq))
    for b, n in enumerate(c.chunks):
        if not n:
            continue
        k, v = c.rows(0, b), c.rows(1, b)
        at = slice(int(c.q_start[b]), int(c.q_start[b]) + n)
        see = ref.visible(n, c.lens[b], None if c.parents is None else c.parents[b].tolist())
        for h in range(c.Hq):
            kh, vh, qh = k[:, h // G], v[:, h // G], q[at, h]
            s = np.where(see, scale * (qh @ kh.T), -np.inf)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            l = p.sum(1, keepdims=True)
            p /= l
            out[at, h] = p @ vh
            mag[at, h] = p @ np.abs(vh)
            dev[at, h] = np.sqrt(np.maximum(p @ vh ** 2 - out[at, h] ** 2, 0))
            lse[at, h] = (top + np.log(l))[:, 0]
            # a score is a sum of D products in fp32: D roundings of at most 2^-24 of the
            # terms' sum, and 4 more for scaling and the exponent; over e4m3 caches the
            # query's values are within 2^-21 of their row's largest
            terms = np.where(see, np.abs(qh) @ np.abs(kh).T, 0).max(1)
            ds[at, h] = abs(scale) * (c.D + 4) * 2.0 ** -24 * terms + 2.0 ** -21
            if c.fp8:
                ds[at, h] += abs(scale) * 2.0 ** -21 * np.abs(qh).max(1) * np.abs(kh).sum(1).max()
    return out, lse, mag, dev, ds


def faults(c, out, lse, reference):
    """What is wrong with out and lse ([tokens][heads] ..., padding included) beside
    exact()'s, as text; empty if nothing.  Scores off by ds move an output by
    sum p_j d_j (v_j - out), at most ds times the values' deviation (twice that, for
    what is not linear).  A weight is off by 2^-8 of it (bf16's spacing is 2^-7 of a
    binade's start), the output by 2^-8 of it by the same spacing.  Over all, the
    roundings differ in sign: a spacing's rms rounding is 0.43 of its largest, weights'
    and outputs' together are 0.61 of 2^-8 of the norm; 2^-8 is allowed."""
    n = sum(c.chunks)
    want, wl, mag, dev, ds = (x[:n] for x in reference)
    got, gl = (np.asarray(x, np.float64)[:n] for x in (out, lse))
    by_scores = 2 * ds[..., None] * dev
    tol = (2.0 ** -8 + 2.0 ** -18) * mag + by_scores + 2.0 ** -8 * np.abs(want) + 1e-30
    found = []
    if not np.isfinite(got).all():
        found.append("not finite")
    off = np.abs(got - want) > tol
    if off.any():
        at = np.argwhere(off)[0]
        found.append("%d of %d values, first %s: %r for %r, allowed %.3g" % (
            off.sum(), off.size, at.tolist(), got[tuple(at)], want[tuple(at)], tol[tuple(at)]))
    size, err = (math.sqrt((x ** 2).sum()) for x in (want, got - want))
    allowed = 2.0 ** -8 * size + math.sqrt((by_scores ** 2).sum())
    if not err <= allowed:
        found.append("error %.4g of the norm, allowed %.4g" % (err / size, allowed / size))
    if not (np.abs(gl - wl) <= ds + np.abs(wl) * 2.0 ** -22).all():
        found.append("log-sum-exp off by %.3g" % np.abs(gl - wl).max())
    return found


def _scales_apart():
    c = ref.Case([400], [6], 4, 1, 128, 16, True, seed=7)
    rng = np.random.default_rng(0)
    for j in range(406):
        p, s = int(c.table[0, j // 16]), j % 16
        for which, name in ((0, "k_exp"), (1, "v_exp")):
            byte = int(rng.integers(100, 125)) if which else int(rng.integers(105, 121))
            if j % 50 == 0:
                byte = 1
            old = int(c.cache[name][p, 0, s])
            c.cache[name][p, 0, s] = byte
            c.values[which][p, s, 0] *= 2.0 ** (byte - old)
    return c


def _lengths(seed, lo, hi, n):
    return [int(x) for x in np.random.default_rng(seed).integers(lo, hi, n)]


# name: a batch over an e4m3 cache
E4M3_CASES = {
    "one slot": lambda: ref.Case([0], [1], 1, 1, 16, 8, True, seed=1),
    "two slots": lambda: ref.Case([1], [1], 8, 8, 64, 16, True, seed=2),
    "one token": lambda: ref.Case([1020], [1], 32, 8, 128, 16, True, seed=3),
    "tile ends": lambda: ref.Case([127, 128, 129, 0, 255], [1] * 5, 8, 1, 128, 64, True, seed=4),
    "chunks": lambda: ref.Case([500, 3, 0, 129, 64], [5, 5, 0, 5, 5], 8, 2, 128, 16, True, True, seed=5),
    "head size 80": lambda: ref.Case([33, 700, 90], [6, 17, 1], 6, 2, 80, 24, True, seed=6),
    "trees": lambda: ref.Case([10, 300], [16, 16], 28, 4, 128, 32, True, False, True, seed=7),
    "long trees": lambda: ref.Case([0, 65, 1], [64, 64, 7], 8, 2, 96, 16, True, True, True, seed=8),
    "prompt alone": lambda: ref.Case([0], [300], 4, 2, 128, 64, True, seed=9),
    "prompts": lambda: ref.Case([0, 200, 77], [129, 257, 64], 8, 2, 64, 128, True, seed=10),
    "prompt, head size 112": lambda: ref.Case([1500], [130], 5, 1, 112, 48, True, seed=11),
    "128 heads a key head": lambda: ref.Case([40], [3], 128, 1, 128, 256, True, seed=12),
    "parts": lambda: ref.Case([9000], [2], 4, 1, 128, 64, True, seed=13),
    "parts, wide": lambda: ref.Case([9000], [32], 8, 2, 128, 64, True, seed=14),
    "parts, pair": lambda: ref.Case([6000], [100], 6, 2, 128, 64, True, seed=15),
    "head size 32": lambda: ref.Case([2000] * 3 + [1] * 5, [2] * 8, 12, 4, 32, 16, True, seed=16),
    "equal scores": lambda: ref.Case([800, 3, 260], [7, 1, 90], 8, 2, 128, 16, True, seed=5, sharp=0.0),
    "sharp scores": lambda: ref.Case([800, 3, 260], [7, 1, 90], 8, 2, 128, 16, True, seed=5, sharp=8.0),
    "scores far apart": lambda: ref.Case([800, 3, 260], [7, 1, 90], 8, 2, 128, 16, True, seed=5, sharp=60.0),
    "scales apart": _scales_apart,
    "mixed": lambda: ref.Case([3000, 100, 2500, 0, 600, 40, 1222], [1, 300, 6, 313, 40, 1, 65], 16, 8, 128, 64, True, seed=21),
    "many": lambda: ref.Case(_lengths(1, 0, 700, 150), [4] * 150, 16, 8, 128, 64, True, seed=21),
    "turns": lambda: ref.Case(_lengths(2, 100, 900, 60), [2, 40, 3, 50, 16, 17] * 10, 16, 8, 128, 64, True, seed=21),
}


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
