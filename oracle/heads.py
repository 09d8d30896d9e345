"""Operators on attention heads between the q/k/v and o projections (oracle;
test infrastructure only).

nanotron tutorial, 5.1: attention runs on each rank's heads between the
column-parallel q/k/v and the row-parallel o.  The pages give no formulas for
what happens there; the definitions below are the ones ``include/dt.h`` states:

* norm of each head and position rotation, with its gradients, in fp64;
* the 4-bit record of a token: codes and parameters from fp32 operations that
  each round on their own (so they are compared bit for bit), and the values
  they stand for in fp64;
* attention over the cached keys of a sequence, in fp64, with a bound on what
  a computation with fp32 sums may differ by.
"""
from __future__ import annotations

import numpy as np

from . import bf16


def pairs_of(rotary: int, interleaved: bool):
    """Channel indices (first, second) of the rotated pairs."""
    i = np.arange(rotary // 2)
    return (2 * i, 2 * i + 1) if interleaved else (i, i + rotary // 2)


def rotate(x, cos_sin, pos, interleaved, back=False, dtype=np.float64):
    """x [t, h, d]: channels (a, b) of each pair -> (a c - b s, b c + a s).

    Every product and sum is one operation of ``dtype``.  Positions outside
    the table give zero rows."""
    x = np.asarray(x, dtype=dtype)
    if cos_sin is None:
        return x.copy()
    rows, rotary = cos_sin.shape
    ok = (pos >= 0) & (pos < rows)
    cs = np.asarray(cos_sin, dtype=dtype)[np.where(ok, pos, 0)][:, None, :]
    c, s = cs[..., : rotary // 2], cs[..., rotary // 2:]
    if back:
        s = -s
    ia, ib = pairs_of(rotary, interleaved)
    a, b = x[..., ia], x[..., ib]
    y = x.copy()
    y[..., ia] = a * c - b * s
    y[..., ib] = b * c + a * s
    y[~ok] = 0
    return y


def norm_rope(x, w, cos_sin, pos, interleaved, eps):
    """x [t, h, d] fp64 -> y."""
    x = np.asarray(x, dtype=np.float64)
    z = x if w is None else x / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)
    return rotate(z, cos_sin, pos, interleaved)


def norm_rope_backward(dy, x, w, cos_sin, pos, interleaved, eps):
    """(dx, dw, bound on |dx| terms, bound on |dw| terms) for a gradient dy."""
    x = np.asarray(x, dtype=np.float64)
    dz = rotate(dy, cos_sin, pos, interleaved, back=True)
    if w is None:
        return dz, None, np.abs(dz), None
    w = np.asarray(w, dtype=np.float64)
    r = 1.0 / np.sqrt((x ** 2).mean(-1, keepdims=True) + eps)
    xhat = x * r
    g = dz * w
    dx = r * (g - xhat * (g * xhat).mean(-1, keepdims=True))
    if cos_sin is not None:
        dx[(pos < 0) | (pos >= cos_sin.shape[0])] = 0
    size = r * (np.abs(g) + np.abs(xhat) * np.abs(g * xhat).mean(-1, keepdims=True))
    return dx, (dz * xhat).sum((0, 1)), size, np.abs(dz * xhat).sum((0, 1))


# ---------------------------------------------------------------- the 4-bit record

def record_words(d: int, group: int) -> int:
    n = 2 * (d // 8) + 2 * (d // group)
    return -(-n // 4) * 4


def quantise(x, group):
    """fp32 x [..., d] -> codes [..., d] int, step bits and minimum bits [..., d/group] uint16."""
    x = np.asarray(x, dtype=np.float32)
    g = x.reshape(x.shape[:-1] + (x.shape[-1] // group, group))
    with np.errstate(all="ignore"):
        lo, hi = g.min(-1), g.max(-1)  # NaN propagates
        mb = bf16.round_rne(lo)
        sb = bf16.round_rne((hi - lo) * np.float32(0.06666667014360428))
        m, s = bf16.widen(mb), bf16.widen(sb)
        inv = np.where(s >= np.float32(2.0 ** -126), np.float32(1) / np.where(s > 0, s, np.float32(1)), np.float32(0))
        bad = ~np.isfinite(m) | ~np.isfinite(s)
        c = np.rint((g - m[..., None]) * inv[..., None].astype(np.float32))
        c = np.where(bad[..., None] | np.isnan(c), 0, np.clip(c, 0, 15)).astype(np.int64)
    mb, sb = np.where(bad, np.uint16(0x7FC0), mb), np.where(bad, np.uint16(0x7FC0), sb)
    return c.reshape(x.shape), sb, mb


def pack(k, v, group):
    """Records uint32 [..., words] of fp32 keys and values [..., d]."""
    words, params = [], []
    for x in (k, v):
        c, sb, mb = quantise(x, group)
        c = c.reshape(c.shape[:-1] + (c.shape[-1] // 8, 8)).astype(np.uint32)
        words.append((c << (4 * np.arange(8, dtype=np.uint32))).sum(-1, dtype=np.uint32))
        params.append(sb.astype(np.uint32) | (mb.astype(np.uint32) << np.uint32(16)))
    rec = np.concatenate(words + params, -1)
    pad = record_words(k.shape[-1], group) - rec.shape[-1]
    return np.concatenate([rec, np.zeros(rec.shape[:-1] + (pad,), np.uint32)], -1)


def unpack(rec, d, group):
    """(k, v, key steps, value steps): fp64 values [..., d] and steps [..., d] of records."""
    rec = np.asarray(rec, dtype=np.uint32)
    w, ng = d // 8, d // group
    out, steps = [], []
    for a, pa in ((0, 2 * w), (w, 2 * w + ng)):
        c = (rec[..., a:a + w, None] >> (4 * np.arange(8, dtype=np.uint32))) & 15
        c = c.reshape(c.shape[:-2] + (d,)).astype(np.float64)
        par = rec[..., pa:pa + ng]
        s = np.repeat(bf16.widen64((par & 0xFFFF).astype(np.uint16)), group, -1)
        m = np.repeat(bf16.widen64((par >> 16).astype(np.uint16)), group, -1)
        out.append(m + c * s)
        steps.append(s)
    return out[0], out[1], steps[0], steps[1]


# ---------------------------------------------------------------- attention

def visible(n_q, n_kv, causal, window):
    """bool [n_q, n_kv]: query i (position n_kv - n_q + i) sees key j."""
    at = n_kv - n_q + np.arange(n_q)[:, None]
    j = np.arange(n_kv)[None, :]
    see = np.ones((n_q, n_kv), dtype=bool)
    if causal:
        see = j <= at
        if window:
            see &= j > at - window
    return see


def attention(q, k, v, scale, causal, window, k_step=None, v_step=None):
    """One kv head: q [n, d], k and v [m, d] fp64 -> (out, lse, bounds).

    bounds = (fp32 bound, additional bound for bf16 activations) on |out|'s
    error per query, one for all channels: sums of products in fp32 (relative
    error 2^-18 of the sum of magnitudes: up to 64 roundings) on codes offset
    by up to 128, probability times step in 8 bits.  They hold for the kernels,
    which offset codes by 8 and keep 11 bits, but leave room: ``attention_error``
    bounds what the kernels compute."""
    n, m = q.shape[0], k.shape[0]
    see = visible(n, m, causal, window)
    out, lse, b32, b16 = np.zeros((n, q.shape[1])), np.full(n, -np.inf), np.zeros(n), np.zeros(n)
    for i in range(n):
        j = np.nonzero(see[i])[0]
        if j.size == 0:
            continue
        with np.errstate(all="ignore"):
            s = scale * (k[j] @ q[i])
            p = np.exp(s - s.max())
            out[i] = (p[:, None] * v[j]).sum(0) / p.sum()
            lse[i] = s.max() + np.log(p.sum())
            if k_step is not None:
                mag = scale * ((np.abs(k[j]) + 16 * k_step[j]) @ np.abs(q[i])).max()
                mag16 = scale * (288 * k_step[j] @ np.abs(q[i])).max()
                vmax, smax = np.abs(v[j]).max(), np.abs(v_step[j]).max()
                e = 2.0 ** -18
                b32[i] = (2 * e * (mag + np.abs(s).max()) + e) * (vmax + 15 * smax)
                b16[i] = 2 * e * mag16 * vmax + 2.0 ** -9 * 1.02 * 15 * smax + e * 288 * smax
    return out, lse, b32, b16


def attention_error(q, k, v, scale, causal, window, k_step, v_step, dtype, many=False):
    """One kv head: (bound on |out|'s error [n, d], bound on lse's [n]) of the kernels' arithmetic, before the output's
    rounding.  Every term is weighted by the probabilities, so it shrinks with the result where many keys share it.

    Logit j is off by delta_j: 2^-18 of the magnitudes it is summed from (with |minimum| <= |k| + 15 steps), for bf16
    activations 2^-31 of the row's largest query per step (queries in fp16, the odd codes' 16 times smaller), and with
    many rows 2^-11 of each |q k| (keys in fp16) and 2^-25 of the largest query per |k|.  To first order that moves out
    by sum p delta |v - out|; 1 % more covers the rest, as delta stays far below 0.01.
    Products with V: fp32 sums, 2^-18 of p (|v| + 15 steps).  bf16, few rows: p times step to 11 bits (2^-11), on codes
    centred by 8, or to 2^-36 of the largest step.  Many rows: p and v to 11 bits, or to 2^-31 of 1 and 2^-37 of the
    largest |v|."""
    see = visible(q.shape[0], k.shape[0], causal, window)
    out, log = np.zeros((q.shape[0], q.shape[1])), np.zeros(q.shape[0])
    for i in range(q.shape[0]):
        j = np.nonzero(see[i])[0]
        if j.size == 0:
            continue
        aq, ak, av = np.abs(q[i]), np.abs(k[j]), np.abs(v[j])
        s = scale * (k[j] @ q[i])
        u = np.exp(s - s.max())
        p = u / u.sum()
        delta = 2.0 ** -18 * (scale * ((ak + 30 * k_step[j]) @ aq) + np.abs(s) + 1)
        if many:
            delta += scale * (2.0 ** -11 * (ak @ aq) + 2.0 ** -25 * aq.max() * ak.sum(-1))
        elif dtype == "bf16":
            delta += 2.0 ** -31 * scale * aq.max() * 15 * k_step[j].sum(-1)
        mean = p @ v[j]
        out[i] = 1.01 * ((p * delta) @ np.abs(v[j] - mean)) + 2.0 ** -18 * (p @ (av + 15 * v_step[j]))
        if many:
            out[i] += 2.0 ** -10 * (p @ av) + (2.0 ** -31 * av.sum(0) + 2.0 ** -37 * av.max() * u.sum()) / u.sum()
        elif dtype == "bf16":
            out[i] += 2.0 ** -11 * 8 * (p @ v_step[j]) + 2.0 ** -36 * 8 * v_step[j].max() * j.size / u.sum()
        log[i] = 1.01 * (p @ delta) + 2.0 ** -18 * (1 + abs(s.max() + np.log(u.sum())))
    return out, log


def prompt_bound(q, k, v, scale, causal, window):
    """What fp16 operands may add to ``attention``'s error, per query: keys and
    values rounded to 11 bits (2^-12 of each, K's through the logits, whose
    error counts twice), probabilities to 11 bits, the row's smallest queries
    to 2^-25 of its largest."""
    see = visible(q.shape[0], k.shape[0], causal, window)
    out = np.zeros(q.shape[0])
    for i in range(q.shape[0]):
        j = np.nonzero(see[i])[0]
        if j.size == 0:
            continue
        with np.errstate(all="ignore"):
            logit = scale * 2.0 ** -12 * (np.abs(k[j]) @ np.abs(q[i])).max()
            logit += scale * 2.0 ** -25 * np.abs(q[i]).max() * np.abs(k[j]).sum(-1).max()
            out[i] = (2 * logit * 1.01 + 2.0 ** -10) * np.abs(v[j]).max()
    return out
