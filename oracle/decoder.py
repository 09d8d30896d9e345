"""64-bit restatement of what lies between blocks and behind the head.

Block: parts of x added, norm, gate, dropout, scaled residual, norm; its
gradients.  Log probabilities over a vocabulary with entropy, alternatives and
gradient.  Plain loops and numpy; shares no code with the library.
"""
from __future__ import annotations

import numpy as np


def philox(counter, key):
    """Philox4x32-10 on Python integers: four words from a counter of four and a key of two words."""
    c, k = list(counter), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b % 2 ** 32, (a >> 32) ^ c[3] ^ k[1], a % 2 ** 32]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    return c


def keep_mask(rng, tokens, n, p, first=0):
    """[tokens, n] of the elements that dropout keeps; the first token has number ``first``."""
    rng = [int(r) % 2 ** 32 for r in rng]
    below = int(np.floor(float(np.float32(p)) * 2.0 ** 32))
    i = np.arange(first * n, (first + tokens) * n, dtype=np.int64)
    q, inv = np.unique(i >> 2, return_inverse=True)
    lo, hi = (q & 0xFFFFFFFF).astype(np.uint64), (q >> 32).astype(np.uint64)
    m32, s32 = np.uint64(0xFFFFFFFF), np.uint64(32)
    c = [lo, hi, np.full_like(lo, rng[2]), np.full_like(lo, rng[3])]
    k = [rng[0], rng[1]]
    for _ in range(10):
        a, b = c[0] * np.uint64(0xD2511F53), c[2] * np.uint64(0xCD9E8D57)
        c = [(b >> s32) ^ c[1] ^ np.uint64(k[0]), b & m32, (a >> s32) ^ c[3] ^ np.uint64(k[1]), a & m32]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    words = np.stack(c, 1)[inv, i & 3]
    return (words >= np.uint64(below)).reshape(tokens, n)


class Block:
    """Forward values of a block and, from ``backward``, its gradients; fp64, rows [tokens, n].

    Each value v has a companion: the sum of the magnitudes that its formula
    adds up, which bounds what roundings can do to it."""

    def __init__(self, parts, residual=None, post=None, gate=None, pre=None, eps=1e-6, scale=1.0, keep=None, p=0.0):
        s = parts[0].astype(np.float64)
        for x in parts[1:]:
            s = s + x
        self.t, self.n = s.shape
        self.s, self.abs_s = s, sum(np.abs(x) for x in parts)
        self.residual, self.post, self.pre, self.eps, self.scale, self.keep = residual, post, pre, eps, scale, keep
        self.gate = None if gate is None else np.repeat(np.atleast_2d(gate), self.t // np.atleast_2d(gate).shape[0], 0)
        self.gate_shape = None if gate is None else gate.shape
        self.inv = 1.0 / (1.0 - float(np.float32(p))) if keep is not None else 1.0
        one = np.ones((1, self.n))
        self.w = one if post is None else post[None]
        self.g = one if gate is None else self.gate
        self.rx = 1.0 / np.sqrt((s * s).mean(1, keepdims=True) + eps) if post is not None else np.ones((self.t, 1))
        self.mul = self.rx * self.w * self.g * self.inv
        f, abs_f = s * self.mul, self.abs_s * np.abs(self.mul)
        if keep is not None:
            f, abs_f = np.where(keep, f, 0.0), np.where(keep, abs_f, 0.0)
        r = 0.0 if residual is None else scale * residual
        self.h, self.abs_h = r + f, np.abs(r) + abs_f
        if pre is not None:
            self.rh = 1.0 / np.sqrt((self.h ** 2).mean(1, keepdims=True) + eps)
            self.y, self.abs_y = self.h * self.rh * pre, self.abs_h * self.rh * np.abs(pre)

    def backward(self, dh=None, dy=None):
        """{name: (gradient, magnitude)} of dx, dr, dpost, dgate, dpre."""
        g, ag = (0.0, 0.0) if dh is None else (dh, np.abs(dh))
        out = {}
        if dy is not None:
            z = dy * self.pre
            g = g + self.rh * z - self.rh ** 3 * (self.h * z).mean(1, keepdims=True) * self.h
            ag = ag + self.rh * np.abs(z) + self.rh ** 3 * (self.abs_h * np.abs(z)).mean(1, keepdims=True) * self.abs_h
            out["dpre"] = ((dy * self.h * self.rh).sum(0), (np.abs(dy) * self.abs_h * self.rh).sum(0))
        out["dr"] = (self.scale * g, np.abs(self.scale) * ag)
        e, ae = g * self.inv, ag * self.inv
        if self.keep is not None:
            e, ae = np.where(self.keep, e, 0.0), np.where(self.keep, ae, 0.0)

        def kept(v):
            return v if self.keep is None else np.where(self.keep, v, 0.0)

        if self.gate is not None:
            d, ad = kept(e * self.s * self.rx * self.w), kept(ae * self.abs_s * self.rx * np.abs(self.w))
            rows = np.atleast_2d(np.empty(self.gate_shape)).shape[0]
            fold = lambda v: v.reshape(rows, self.t // rows, self.n).sum(1).reshape(self.gate_shape)  # noqa: E731
            out["dgate"] = (fold(d), fold(ad))
        e, ae = e * self.g, ae * np.abs(self.g)
        if self.post is not None:
            out["dpost"] = (kept(e * self.s * self.rx).sum(0), kept(ae * self.abs_s * self.rx).sum(0))
            v, av = e * self.w, ae * np.abs(self.w)
            m, am = kept(self.s * v).mean(1, keepdims=True), kept(self.abs_s * av).mean(1, keepdims=True)
            e, ae = self.rx * v - self.rx ** 3 * m * self.s, self.rx * av + self.rx ** 3 * am * self.abs_s
        out["dx"] = (e, ae)
        return out


def log_probs(z, scale=1.0):
    """(log probabilities [t, v], lse [t], entropy [t]) of fp64 logits; rows of nothing but -inf as documented."""
    x = z * scale
    top = x.max(1, keepdims=True)
    none = np.isneginf(top)
    with np.errstate(invalid="ignore", divide="ignore", over="ignore"):
        e = np.exp(x - np.where(none, 0.0, top))
        total = e.sum(1, keepdims=True)
        ln = np.log(np.where(none, 1.0, total))
        lse = top + ln
        logp = np.where(none, -np.inf, (x - np.where(none, 0.0, top)) - ln)
        p = np.exp(logp)
        ent = -np.where(p > 0, p * logp, np.where(np.isnan(p), np.nan, 0.0)).sum(1)
    return logp, lse[:, 0], np.where(none[:, 0], 0.0, ent)


def top(z, k):
    """Indices [t, k] of the k largest, largest first, ties to the lowest index, NaN above all."""
    out = np.empty((z.shape[0], k), dtype=np.int64)
    for i, row in enumerate(z):
        key = [(0 if np.isnan(v) else 1, 0.0 if np.isnan(v) else -float(v) + 0.0, j) for j, v in enumerate(row)]
        out[i] = [j for _, _, j in sorted(key)[:k]]
    return out


def log_probs_backward(z, ids, dlogp, lse, scale=1.0, dent=None, ent=None):
    """(gradient, magnitude) with respect to the logits; ids [t, c], negative ones add nothing."""
    t, v = z.shape
    with np.errstate(over="ignore", invalid="ignore"):
        logp = z * scale - lse[:, None]
        p = np.where(np.isneginf(lse)[:, None], 0.0, np.exp(logp))
    g = np.where((ids >= 0) & (ids < v), dlogp, 0.0) if ids is not None else np.zeros((t, 0))
    d, a = -p * g.sum(1, keepdims=True), p * np.abs(g).sum(1, keepdims=True)
    if dent is not None:
        lp = np.where(p > 0, logp, 0.0)
        d = d - dent[:, None] * p * (lp + ent[:, None])
        a = a + np.abs(dent[:, None]) * p * (np.abs(lp) + np.abs(ent[:, None]))
    for i in range(t):
        for c in range(g.shape[1]):
            if 0 <= ids[i, c] < v:
                d[i, ids[i, c]] += g[i, c]
                a[i, ids[i, c]] += abs(g[i, c])
    dead = np.isneginf(lse)
    d[dead], a[dead] = 0.0, 0.0
    return d * scale, a * scale
