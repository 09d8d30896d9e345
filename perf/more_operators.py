"""Cases of the operators around a block of a decoder, and at its end.

Two operators, each with its gradient:

* ``block``  what lies between the output of one block (attention or MLP, with
             its shards' partial sums still apart, if need be) and the input of
             the next: a norm of the output, a gate, dropout whose mask is never
             stored, the scaled residual, and the norm before the next block;
* ``logp``   log probabilities of given tokens from logits whose vocabulary is
             sharded, as a column-parallel head leaves them, with the entropy
             and the top alternatives of each token.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the
library's calls on the same inputs.

The block, per token (parts of x are added first; what a case lacks is left out):

  u = x / sqrt(mean(x^2) + eps) * post      u = u * gate      u = keep ? u / (1 - p) : 0
  h = scale * residual + u                  y = h / sqrt(mean(h^2) + eps) * pre

keep of element e = token * channels + channel is the e % 4th word of
Philox4x32-10 (Salmon, Moraes, Dror and Shaw, "Parallel random numbers: as easy
as 1, 2, 3", 2011) with the key rng[0:2] and the counter (e // 4 low, e // 4
high, rng[2], rng[3]), compared with floor(p * 2^32), p in fp32.

The log probabilities: l = log_softmax(s * logits); an id that is IGNORE gives 0.
"""
import math

import numpy as np
import torch

own = False

EPS = 1e-6
IGNORE = -100
BF16, FP32 = "bf16", "fp32"
_DT = {BF16: torch.bfloat16, FP32: torch.float32}
REP, SHARD, PARTIAL = "replicate", "shard", "partial"


# ------------------------------------------------------------------ the cases

def _block(name, tokens, n, parts, place, dtype=BF16, stream=None, post=False, gate=0, drop=0.0, scale=1.0,
           backward=False, out=SHARD):
    """``place``: how x lies on the shards; ``out``: residual and outputs; ``stream``: dtype of the residual stream;
    ``gate``: 0 none, -1 one for all tokens, else the number of its rows, each for as many consecutive tokens."""
    return {"name": name, "op": "block", "tokens": tokens, "n": n, "parts": parts, "place": place, "out": out,
            "dtype": dtype, "stream": dtype if stream is None else stream, "post": post, "gate": gate, "drop": drop,
            "scale": scale, "backward": backward}


def _logp(name, tokens, vocab, parts, dtype=BF16, given=1, top=0, entropy=False, scale=1.0, masked=False,
          backward=False):
    """``given``: tokens per row whose log probability is asked for; ``masked``: part of the logits are -inf."""
    return {"name": name, "op": "logp", "tokens": tokens, "vocab": vocab, "parts": parts, "dtype": dtype,
            "given": given, "top": top, "entropy": entropy, "scale": scale, "masked": masked, "backward": backward}


def listed():
    return [
        # the smallest call: a decode step of 8 sequences behind a row-parallel layer that left its partial sums
        _block("block decode 8 tokens", 8, 4096, 4, PARTIAL, post=True, out=REP),
        # the attention workload of the benchmark, tokens sharded: residual, dropout and the next block's norm
        _block("block train dropout", 8192, 4096, 4, SHARD, drop=0.1),
        # partial sums of 8 shards reduced and scattered on the way, a wide model with norms on both sides
        _block("block reduce wide", 2048, 8192, 8, PARTIAL, post=True, scale=0.5),
        # images of 1031 patches, a gate for each of them, the residual stream in fp32
        _block("block image gates", 13 * 1031, 1152, 1, REP, stream=FP32, gate=13, out=REP),
        # gradients of a block with both norms and a gate per channel
        _block("block train backward", 8192, 4096, 4, SHARD, post=True, gate=-1, backward=True),
        # a small model in fp32, odd sizes, dropout, gates per sequence: gradients
        _block("block fp32 odd backward", 7 * 219, 1000, 2, SHARD, FP32, post=True, gate=7, drop=0.25, backward=True),
        # one user, one token: what a server reports beside the sampled token
        _logp("logp decode one", 1, 128256, 4, top=20, entropy=True),
        # a serving batch at a temperature, under a mask of allowed tokens, fp32 logits
        _logp("logp decode batch", 64, 128256, 8, FP32, top=5, scale=1.25, masked=True),
        # scoring prompts: every token's log probability and entropy, the embedding workload's vocabulary
        _logp("logp prompt", 4096, 128256, 8, entropy=True),
        # an odd vocabulary, not sharded, three candidates and ten alternatives per row
        _logp("logp odd vocabulary", 777, 50257, 1, given=3, top=10),
        # the gradient of a training loss, the largest case
        _logp("logp train backward", 4096, 128256, 8, backward=True),
        # a policy's gradient, entropy bonus included, odd shards in fp32
        _logp("logp odd backward", 301, 50257, 2, FP32, given=4, entropy=True, backward=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    parts = rng.choice([1, 2, 4, 8])
    backward = rng.random() < 0.5
    if rng.random() < 0.5:
        n = rng.choice([_log(rng, 8, 2048) * 8, _log(rng, 8, 2048) * 8, _log(rng, 8, 2048) * 8, 1024, 2048, 4096, 5120,
                        8192, _log(rng, 33, 8191) | 1])
        place = rng.choice([REP, SHARD, SHARD, PARTIAL])
        budget = 8192 * 4096 * 2 // (parts + 3 if place == PARTIAL else 4)
        tokens = max(1, min(_log(rng, 1, 16384), budget // n))
        gate = rng.choice([0, 0, -1, -1, 1, 3, 8])
        if gate > 0:
            tokens = max(gate, tokens // gate * gate)
        dtype, stream = rng.choice([(BF16, BF16), (BF16, BF16), (BF16, FP32), (FP32, FP32)])
        if FP32 in (dtype, stream):
            tokens = max(max(gate, 1), tokens // 2 // max(gate, 1) * max(gate, 1))
        c = _block("", tokens, n, parts, place, dtype, stream, rng.random() < 0.5, gate, rng.choice([0.0, 0.0, 0.1, 0.5]),
                   rng.choice([1.0, 1.0, 0.5, 2.25]), backward, rng.choice([REP, SHARD]))
    else:
        vocab = rng.choice([_log(rng, 1000, 262144), _log(rng, 1000, 262144), 32000, 50257, 65536, 128256])
        dtype = rng.choice([BF16, BF16, FP32])
        given = rng.choice([1, 1, 1, 2, 5])
        tokens = max(1, min(_log(rng, 1, 16384), 4096 * 128256 // vocab // (1 if dtype == BF16 else 2)))
        top = 0 if backward else rng.choice([0, 0, 1, 5, 20])
        if top:
            tokens = min(tokens, max(1, (1 << 27) // vocab))
        c = _logp("", tokens, vocab, parts, dtype, given, top, rng.random() < 0.5, rng.choice([1.0, 1.0, 0.7, 1.25]),
                  rng.random() < 0.2, backward)
    del c["name"]
    return c


def work(case):
    b = 2 if case["dtype"] == BF16 else 4
    t = case["tokens"]
    if case["op"] == "logp":
        x = t * case["vocab"]
        small = 4 * t * (2 * case["given"] + 1 + bool(case["entropy"]) + 2 * case["top"])
        # forward: read each logit once; backward: read each and write its gradient
        return {"bytes": (2 if case["backward"] else 1) * x * b + small,
                "flops": x * (4 + (2 if case["entropy"] else 0) + (2 if case["backward"] else 0))}
    n, rb = case["n"], 2 if case["stream"] == BF16 else 4
    copies = case["parts"] if case["place"] == PARTIAL else 1
    rows = max(0, case["gate"]) or (1 if case["gate"] else 0)
    vectors = n * (1 + bool(case["post"]) + rows) * 4
    # forward: read x and the residual, write h and y; backward: read x, the residual and the gradients of h and y,
    # write those of x and the residual
    if case["backward"]:
        return {"bytes": t * n * ((copies + 2) * b + 3 * rb) + 2 * vectors, "flops": t * n * (copies + 24)}
    return {"bytes": t * n * ((copies + 1) * b + 2 * rb) + vectors, "flops": t * n * (copies + 12)}


# ------------------------------------------------------------------ inputs

def _rows(x, parts):
    """The slots of a tensor split over its rows."""
    return [s.contiguous() for s in x.chunk(parts, dim=0)] + [x[:0]] * (parts - len(x.chunk(parts, dim=0)))


def _slots(x, place, parts):
    return _rows(x, parts) if place == SHARD else [x]


def _whole(slots, place):
    """All rows in fp32, parts of a sum added in their order."""
    if place == PARTIAL:
        s = slots[0].float()
        for p in slots[1:]:
            s = s + p.float()
        return s
    return torch.cat(slots).float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    st = {"case": case}
    (_prepare_block if case["op"] == "block" else _prepare_logp)(st, case, gen)
    if own:
        (_block_handles if case["op"] == "block" else _logp_handles)(st)
    return st


def _randn(gen, *shape):
    return torch.randn(*shape, generator=gen, device="cuda")


def _prepare_block(st, case, gen):
    t, n, p, dt, rt = case["tokens"], case["n"], case["parts"], _DT[case["dtype"]], _DT[case["stream"]]
    # activations with channels of their own scale; a residual stream that has grown over some layers
    ch = torch.exp(0.4 * _randn(gen, n))
    if case["place"] == PARTIAL:
        st["x"] = [(_randn(gen, t, n) * ch / math.sqrt(p)).to(dt) for _ in range(p)]
    else:
        st["x"] = _slots((_randn(gen, t, n) * ch).to(dt), case["place"], p)
    st["r"] = _slots((2.0 * _randn(gen, t, n) * torch.exp(0.3 * _randn(gen, n))).to(rt), case["out"], p)
    st["pre"] = 1 + 0.1 * _randn(gen, n)
    st["post"] = 1 + 0.1 * _randn(gen, n) if case["post"] else None
    st["gate"] = None
    if case["gate"]:
        st["gate"] = 0.5 + 0.3 * (_randn(gen, n) if case["gate"] < 0 else _randn(gen, case["gate"], n))
    st["rng"] = None
    if case["drop"]:
        st["rng"] = torch.randint(-2 ** 31, 2 ** 31, (4,), generator=gen, device="cuda").to(torch.int32)
    if case["backward"]:
        st["dh"] = _slots(_randn(gen, t, n).to(rt), case["out"], p)
        st["dy"] = _slots((3.0 * _randn(gen, t, n)).to(dt), case["out"], p)


def _prepare_logp(st, case, gen):
    t, v, p, dt, g = case["tokens"], case["vocab"], case["parts"], _DT[case["dtype"]], case["given"]
    ids = torch.randint(0, v, (t, g), generator=gen, device="cuda")
    z = torch.empty(t, v, device="cuda", dtype=dt)
    step = max(1, (1 << 27) // v)
    likely = torch.randn(2, v, generator=gen, device="cuda")  # by token: what is set twice is set alike
    for a in range(0, t, step):
        e = min(t, a + step)
        # a bulk of unlikely tokens, a few likely ones, the given tokens mostly among these
        y = 2.0 * _randn(gen, e - a, v)
        if case["masked"]:
            y[torch.rand(e - a, v, generator=gen, device="cuda") < 0.5] = -math.inf
        hot = torch.randint(0, v, (e - a, 8), generator=gen, device="cuda")
        y.scatter_(1, hot, 8.0 + 3.0 * likely[0][hot])
        y.scatter_(1, ids[a:e], 6.0 + 4.0 * likely[1][ids[a:e]])
        z[a:e] = y.to(dt)
    # a tenth of the rows is padding
    pad = torch.rand(t, generator=gen, device="cuda") < 0.1
    ids[pad] = IGNORE
    st["z"] = [c.contiguous() for c in z.chunk(p, dim=1)]
    st["ids"] = ids.to(torch.int32) if g > 1 else ids[:, 0].to(torch.int32)
    if case["backward"]:
        st["dlp"] = (_randn(gen, t, g) if g > 1 or case["entropy"] else torch.full((t, 1), -1.0, device="cuda")) / t
        if g == 1:
            st["dlp"] = st["dlp"][:, 0].contiguous()
        st["dent"] = 0.01 * _randn(gen, t) / t if case["entropy"] else None
        # what the forward pass returned
        st["lse"] = torch.empty(t, device="cuda")
        st["ent"] = torch.empty(t, device="cuda") if case["entropy"] else None
        for a in range(0, t, step):
            x = z[a:a + step].double() * _f32(case["scale"])
            l = torch.logsumexp(x, 1)
            st["lse"][a:a + step] = l.float()
            if case["entropy"]:
                lp = x - l[:, None]
                st["ent"][a:a + step] = -(lp.exp() * lp.clamp(min=-1e30)).sum(1).float()


def _f32(x):
    """x as the fp32 number that a call takes."""
    return float(np.float32(x))


def _mesh(st):
    import tensor_sharded_linear_gb300 as tsl
    return tsl, tsl.DeviceMesh((st["case"]["parts"],), ("tp",))


def _block_handles(st):
    """What a user of the library keeps: distributed tensors over the slots above, outputs and the workspace."""
    tsl, mesh = _mesh(st)
    c = st["case"]
    shape, dt, rt = (c["tokens"], c["n"]), _DT[c["dtype"]], _DT[c["stream"]]
    pl = {REP: [tsl.Replicate()], SHARD: [tsl.Shard(0)], PARTIAL: [tsl.Partial()]}
    h = st["h"] = {"tsl": tsl}
    h["x"] = tsl.DTensor(st["x"], mesh, pl[c["place"]], shape, dt)
    h["r"] = tsl.DTensor(st["r"], mesh, pl[c["out"]], shape, rt)
    for name in ("pre", "post", "gate", "rng"):
        v = st[name]
        h[name] = None if v is None else tsl.DTensor([v], mesh, pl[REP], tuple(v.shape), v.dtype)
    if not c["backward"]:
        h["out"] = tuple(tsl.DTensor.empty(mesh, pl[c["out"]], shape, d) for d in (rt, dt))
        return
    h["dh"] = tsl.DTensor(st["dh"], mesh, pl[c["out"]], shape, rt)
    h["dy"] = tsl.DTensor(st["dy"], mesh, pl[c["out"]], shape, dt)
    like = lambda t: None if t is None else tsl.DTensor.empty(mesh, pl[REP], t.gshape, t.dtype)  # noqa: E731
    h["out"] = (tsl.DTensor.empty(mesh, pl[REP if c["place"] == PARTIAL else c["place"]], shape, dt),
                tsl.DTensor.empty(mesh, pl[c["out"]], shape, rt), like(h["post"]), like(h["gate"]), like(h["pre"]))
    h["workspace"] = torch.empty(max(256, tsl.tp_block_norm_backward_workspace_bytes(
        h["x"], h["post"], h["gate"], h["pre"])), dtype=torch.uint8, device="cuda")


def _logp_handles(st):
    tsl, mesh = _mesh(st)
    c = st["case"]
    t, rep = c["tokens"], [tsl.Replicate()]
    h = st["h"] = {"tsl": tsl}
    h["z"] = tsl.DTensor(st["z"], mesh, [tsl.Shard(1)], (t, c["vocab"]), _DT[c["dtype"]])
    for name in ("ids", "dlp", "dent", "lse", "ent"):
        v = st.get(name)
        h[name] = None if v is None else tsl.DTensor([v], mesh, rep, tuple(v.shape), v.dtype)
    if c["backward"]:
        h["out"] = tsl.DTensor.empty(mesh, [tsl.Shard(1)], (t, c["vocab"]), _DT[c["dtype"]])
    else:
        empty = lambda *s, dtype=torch.float32: tsl.DTensor.empty(mesh, rep, s, dtype)  # noqa: E731
        h["out"] = (empty(*st["ids"].shape), empty(t), empty(t) if c["entropy"] else None,
                    empty(t, c["top"]) if c["top"] else None,
                    empty(t, c["top"], dtype=torch.int32) if c["top"] else None)


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return (_own_block if st["case"]["op"] == "block" else _own_logp)(st)
    return (_plain_block if st["case"]["op"] == "block" else _plain_logp)(st)


def _own_block(st):
    c, h = st["case"], st["h"]
    tsl = h["tsl"]
    kw = dict(eps=EPS, residual_scale=c["scale"], dropout=c["drop"], rng=h["rng"], out=h["out"])
    if not c["backward"]:
        hh, y = tsl.tp_block_norm(h["x"], h["r"], h["post"], h["gate"], h["pre"], **kw)
        return {"h": hh.slots, "y": y.slots}
    out = tsl.tp_block_norm_backward(h["dh"], h["dy"], h["x"], h["r"], h["post"], h["gate"], h["pre"],
                                     workspace=h["workspace"], **kw)
    return {k: v.slots for k, v in zip(("dx", "dr", "dpost", "dgate", "dpre"), out) if v is not None}


def _own_logp(st):
    c, h = st["case"], st["h"]
    tsl = h["tsl"]
    if c["backward"]:
        d = tsl.tp_log_probs_backward(h["dlp"], h["dent"], h["z"], h["ids"], h["lse"], h["ent"], scale=c["scale"],
                                      ignore_index=IGNORE, out=h["out"])
        return {"dz": d.slots}
    r = tsl.tp_log_probs(h["z"], h["ids"], scale=c["scale"], top=c["top"], entropy=c["entropy"], ignore_index=IGNORE,
                         out=h["out"])
    return {k: v.slots[0] for k, v in zip(("logp", "lse", "entropy", "top", "top_ids"), r) if v is not None}


# -- the plain forms

def _philox_keep(rng, tokens, n, p):
    """[tokens, n] booleans: the elements that dropout keeps."""
    m = 0xFFFFFFFF
    k0, k1, c2, c3 = [rng[i].long() & m for i in range(4)]
    i = torch.arange((tokens * n + 3) // 4, device="cuda")
    a, b = i & m, i >> 32
    c, d = c2.expand_as(i), c3.expand_as(i)
    for _ in range(10):
        x, y = a * 0xD2511F53, c * 0xCD9E8D57  # low 64 bits; the arithmetic shift's sign is masked off
        a, b, c, d = (y >> 32 & m) ^ b ^ k0, y & m, (x >> 32 & m) ^ d ^ k1, x & m
        k0, k1 = (k0 + 0x9E3779B9) & m, (k1 + 0xBB67AE85) & m
    words = torch.stack([a, b, c, d], dim=1).flatten()[:tokens * n].view(tokens, n)
    return words >= int(_f32(p) * 2.0 ** 32)


def _plain_block(st):
    c = st["case"]
    t, n, p, dt, rt = c["tokens"], c["n"], c["parts"], _DT[c["dtype"]], _DT[c["stream"]]
    x, r = _whole(st["x"], c["place"]), _whole(st["r"], c["out"])
    post, gate, pre = st["post"], st["gate"], st["pre"]
    if c["gate"] > 0:
        gate = gate.repeat_interleave(t // c["gate"], 0)
    rx = 1.0 / (x.square().mean(1, keepdim=True) + EPS).sqrt() if c["post"] else None
    xhat = x * rx if c["post"] else x
    u = xhat * post if c["post"] else xhat
    if c["drop"]:
        mask = torch.where(_philox_keep(st["rng"], t, n, c["drop"]), 1.0 / (1.0 - _f32(c["drop"])), 0.0)
    f = u * gate if c["gate"] else u
    if c["drop"]:
        f = f * mask
    h = r * c["scale"] + f
    rh = 1.0 / (h.square().mean(1, keepdim=True) + EPS).sqrt()
    hhat = h * rh
    if not c["backward"]:
        return {"h": _slots(h.to(rt), c["out"], p), "y": _slots((hhat * pre).to(dt), c["out"], p)}
    dh, dy = _whole(st["dh"], c["out"]), _whole(st["dy"], c["out"])
    out = {"dpre": [(dy * hhat).sum(0)]}
    g = dy * pre
    g = dh + rh * (g - hhat * (g * hhat).mean(1, keepdim=True))
    out["dr"] = _slots((g * c["scale"]).to(rt), c["out"], p)
    if c["drop"]:
        g = g * mask
    if c["gate"]:
        dg = g * u
        out["dgate"] = [dg.sum(0) if c["gate"] < 0 else dg.view(c["gate"], -1, n).sum(1)]
        g = g * gate
    if c["post"]:
        out["dpost"] = [(g * xhat).sum(0)]
        g = g * post
        g = rx * (g - xhat * (g * xhat).mean(1, keepdim=True))
    out["dx"] = _slots(g.to(dt), REP if c["place"] == PARTIAL else c["place"], p)
    return out


def _plain_logp(st):
    c = st["case"]
    s, k = _f32(c["scale"]), c["top"]
    z = torch.cat(st["z"], dim=1).float()
    ids = st["ids"].long().view(c["tokens"], -1)
    there = ids != IGNORE
    at = ids.clamp(min=0)
    if c["backward"]:
        lp = z * s - st["lse"][:, None]
        p = lp.exp()
        g = torch.where(there, st["dlp"].view_as(ids), 0.0)
        d = p * -g.sum(1, keepdim=True)
        if c["entropy"]:
            d = d - st["dent"][:, None] * p * (lp.clamp(min=-1e30) + st["ent"][:, None])
        d.scatter_add_(1, at, g)
        return {"dz": [x.contiguous() for x in (d * s).to(_DT[c["dtype"]]).chunk(c["parts"], dim=1)]}
    m = z.amax(1, keepdim=True)
    d = (z - m) * s
    e = d.exp()
    total = e.sum(1, keepdim=True)
    ln = total.log()
    out = {"logp": torch.where(there, d.gather(1, at) - ln, 0.0).view(st["ids"].shape), "lse": (m * s + ln)[:, 0]}
    if c["entropy"]:
        out["entropy"] = (ln - (e * d.clamp(min=-1e30)).sum(1, keepdim=True) / total)[:, 0]
    if k:
        # ties go to the lowest id
        idx = torch.sort(z, dim=1, descending=True, stable=True).indices[:, :k]
        out["top"] = d.gather(1, idx) - ln
        out["top_ids"] = idx.to(torch.int32)
    return out


# ------------------------------------------------------------------ the definition, in 64 bits

def _kept(rng, tokens, n, p):
    """The same choice from the generator's definition, on the host."""
    key = [int(v) & 0xFFFFFFFF for v in rng.tolist()]
    blocks = -(-tokens * n // 4)
    words = np.empty((blocks, 4), dtype=np.uint32)
    step = 1 << 20
    for lo in range(0, blocks, step):
        i = np.arange(lo, min(blocks, lo + step), dtype=np.uint64)
        ctr = [(i & np.uint64(0xFFFFFFFF)).astype(np.uint32), (i >> np.uint64(32)).astype(np.uint32),
               np.full(len(i), key[2], np.uint32), np.full(len(i), key[3], np.uint32)]
        for r in range(10):
            k = [np.uint32((key[0] + r * 0x9E3779B9) % 2 ** 32), np.uint32((key[1] + r * 0xBB67AE85) % 2 ** 32)]
            m0 = ctr[0].astype(np.uint64) * np.uint64(0xD2511F53)
            m1 = ctr[2].astype(np.uint64) * np.uint64(0xCD9E8D57)
            hi = lambda m: (m >> np.uint64(32)).astype(np.uint32)  # noqa: E731
            ctr = [hi(m1) ^ ctr[1] ^ k[0], m1.astype(np.uint32), hi(m0) ^ ctr[3] ^ k[1], m0.astype(np.uint32)]
        words[lo:lo + len(i)] = np.stack(ctr, 1)
    keep = words.reshape(-1)[:tokens * n].reshape(tokens, n).astype(np.float64) >= math.floor(_f32(p) * 2.0 ** 32)
    return torch.from_numpy(keep).cuda()


def _exact_block(case, st):
    t, n, p = case["tokens"], case["n"], case["parts"]
    grad = case["backward"]
    leaf = lambda v: v.double().requires_grad_(grad)  # noqa: E731
    parts = torch.stack([s.double() for s in st["x"]]).sum(0) if case["place"] == PARTIAL else \
        torch.cat([s.double() for s in st["x"]])
    leaves = {"dx": leaf(parts), "dr": leaf(torch.cat(st["r"])), "dpre": leaf(st["pre"])}
    if case["post"]:
        leaves["dpost"] = leaf(st["post"])
    if case["gate"]:
        leaves["dgate"] = leaf(st["gate"])

    def norm(v, w):
        return v * w / torch.sqrt(torch.sum(v * v, dim=-1, keepdim=True) / n + EPS)

    u = norm(leaves["dx"], leaves["dpost"]) if case["post"] else leaves["dx"]
    if case["gate"]:
        g = leaves["dgate"]
        u = u * g if case["gate"] < 0 else (u.view(case["gate"], -1, n) * g[:, None]).view(t, n)
    if case["drop"]:
        u = u * _kept(st["rng"], t, n, case["drop"]) / (1.0 - _f32(case["drop"]))
    h = u + case["scale"] * leaves["dr"]
    y = norm(h, leaves["dpre"])
    cut = lambda v, place: _slots(v, place, p)  # noqa: E731
    if not grad:
        return {"h": cut(h, case["out"]), "y": cut(y, case["out"])}
    names = list(leaves)
    dh, dy = (torch.cat([s.double() for s in st[k]]) for k in ("dh", "dy"))
    got = dict(zip(names, torch.autograd.grad((h, y), [leaves[k] for k in names], (dh, dy))))
    out = {k: [v] for k, v in got.items()}
    out["dr"] = cut(got["dr"], case["out"])
    out["dx"] = cut(got["dx"], REP if case["place"] == PARTIAL else case["place"])
    return out


def _exact_logp(case, st):
    s, v, k = _f32(case["scale"]), case["vocab"], case["top"]
    t = case["tokens"]
    ids = st["ids"].view(t, -1).long()
    pieces = []
    step = max(1, (1 << 26) // v)
    for a in range(0, t, step):
        e = min(t, a + step)
        z = torch.cat([c[a:e].double() for c in st["z"]], dim=1)
        own_ids = ids[a:e]
        hit = own_ids >= 0
        if case["backward"]:
            logp = z * s - st["lse"][a:e, None].double()
            prob = torch.exp(logp)
            d = torch.zeros_like(z)
            for j in range(ids.shape[1]):
                w = torch.where(hit[:, j], st["dlp"].view(t, -1)[a:e, j].double(), 0.0)
                d -= w[:, None] * prob
                d[torch.arange(e - a, device="cuda"), own_ids[:, j].clamp(min=0)] += w
            if case["entropy"]:
                ent = torch.where(prob > 0, prob * (logp + st["ent"][a:e, None].double()), 0.0)
                d -= st["dent"][a:e, None].double() * ent
            pieces.append({"dz": d * s})
            continue
        logp = torch.log_softmax(z * s, dim=1)
        one = {"logp": torch.where(hit, torch.gather(logp, 1, own_ids.clamp(min=0)), 0.0),
               "lse": torch.logsumexp(z * s, dim=1)}
        if case["entropy"]:
            prob = torch.exp(logp)
            one["entropy"] = -torch.where(prob > 0, prob * logp, 0.0).sum(1)
        if k:
            at, place = torch.arange(v, device="cuda"), []
            left = z.clone()
            for _ in range(k):
                best = left.max(1, keepdim=True).values
                i = torch.where(left == best, at, v).min(1).values
                place.append(i)
                left[torch.arange(e - a, device="cuda"), i] = -math.inf
            idx = torch.stack(place, 1)
            one["top"], one["top_ids"] = torch.gather(logp, 1, idx), idx.to(torch.int32)
        pieces.append(one)
    out = {name: torch.cat([q[name] for q in pieces]) for name in pieces[0]}
    if case["backward"]:
        return {"dz": list(out["dz"].chunk(case["parts"], dim=1))}
    out["logp"] = out["logp"].view(st["ids"].shape)
    return out


def exact(case, seed):
    st = prepare(case, seed)
    return (_exact_block if case["op"] == "block" else _exact_logp)(case, st)
