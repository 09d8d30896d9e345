"""Cases of the operators between the q/k/v projections and the o projection.

Three operators, all tensor-parallel over heads (slot i of ``parts`` holds the
heads of chunk i, as ``tp_attention_projections`` leaves them):

* ``norm``    norms of queries and keys for each head with the position
              rotation in the same pass (forward, and backward with the
              gradients of the two norm weights);
* ``append``  keys and values of new tokens written into a paged cache held
              in 4 bits, with the rotation applied on the way to the keys and
              to the queries that go with them;
* ``attn``    attention of each sequence's newest queries over its part of
              that cache.

``own`` false: elementary torch operations in 32 bits.  ``own`` true: the
library's calls on the same inputs.

The cache: int32 [pages, kv heads, page size, words].  The record of one token
and head is  D/8 words of key codes, D/8 of value codes (nibble i of word w is
channel 8 w + i), then one word per group of ``group`` channels for the keys
and one for the values (bf16 step in the low half, bf16 minimum in the high
half), padded to a multiple of 4 words.  A code c stands for
minimum + c * step.
"""
import math

import torch

own = False

EPS = 1e-6
THETA = 10000.0
BF16, FP32 = "bf16", "fp32"
_DT = {BF16: torch.bfloat16, FP32: torch.float32}


# ------------------------------------------------------------------ the cases

def _norm(name, tokens, hq, hk, d, parts, dtype=BF16, backward=False, rotary=None, interleaved=False, table=8192):
    return {"name": name, "op": "norm", "tokens": tokens, "hq": hq, "hk": hk, "d": d, "parts": parts, "dtype": dtype,
            "backward": backward, "rotary": d if rotary is None else rotary, "interleaved": interleaved,
            "table": table}


def _append(name, batch, q_len, kv_len, hq, hk, d, parts, page, group=64, dtype=BF16, ragged=True,
            interleaved=False):
    return {"name": name, "op": "append", "batch": batch, "q_len": q_len, "kv_len": kv_len, "hq": hq, "hk": hk,
            "d": d, "parts": parts, "page": page, "group": group, "dtype": dtype, "ragged": ragged,
            "interleaved": interleaved}


def _attn(name, batch, q_len, kv_len, hq, hk, d, parts, page, group=64, dtype=BF16, ragged=True, window=0,
          causal=True):
    return {"name": name, "op": "attn", "batch": batch, "q_len": q_len, "kv_len": kv_len, "hq": hq, "hk": hk,
            "d": d, "parts": parts, "page": page, "group": group, "dtype": dtype, "ragged": ragged,
            "window": window, "causal": causal}


def listed():
    return [
        # the smallest call: one decode step of 8 sequences, 32 query and 8 key heads over 4 shards
        _norm("norm decode 8 tokens", 8, 32, 8, 128, 4),
        # the attention workload of the benchmark: 8192 tokens, 32 heads of 128 over 4 shards
        _norm("norm train forward", 8192, 32, 32, 128, 4),
        _norm("norm train backward", 8192, 32, 32, 128, 4, backward=True),
        # a small model in fp32: odd token count, a rotation of interleaved pairs over half of the head
        _norm("norm fp32 odd backward", 1531, 12, 4, 64, 1, FP32, backward=True, rotary=32, interleaved=True,
              table=2048),
        # one decode step of 32 sequences
        _append("append decode 32", 32, 1, 4000, 32, 8, 128, 4, 16),
        # three prompts of different lengths, 8000 tokens or so together
        _append("append prompts", 3, 4096, 4500, 32, 8, 128, 4, 64),
        # one user, one token: the latency of a single stream
        _attn("attn decode one", 1, 1, 4097, 32, 8, 128, 4, 16),
        # a serving batch with contexts of all lengths
        _attn("attn decode batch", 48, 1, 8192, 32, 8, 128, 4, 16),
        # few long contexts, the largest read
        _attn("attn decode long", 5, 1, 131071, 32, 8, 128, 1, 64),
        # verifying drafts of up to 5 tokens, fp32 activations, no shared key heads, odd pages
        _attn("attn drafts fp32", 7, 5, 2000, 12, 12, 64, 2, 24, 32, FP32),
        # wide heads with a sliding window
        _attn("attn window wide", 16, 1, 6000, 16, 2, 256, 2, 32, window=1024),
        # chunks of long prompts against their context so far, the largest product
        _attn("attn prompt chunks", 3, 1024, 8000, 32, 8, 128, 4, 64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "append", "append", "attn", "attn", "attn", "attn"])
    hk = rng.choice([1, 2, 4, 5, 8])
    hq = hk * rng.choice([1, 2, 4, 5, 7, 8])
    parts = rng.choice([p for p in (1, 2, 4, 8) if hk % p == 0])
    dtype = rng.choice([BF16, BF16, BF16, FP32])
    if op == "norm":
        d = rng.choice([64, 80, 128, 128, 256])
        rotary = d if rng.random() < 0.7 else d // 4
        tokens = _log(rng, 1, 16384)
        tokens = max(1, min(tokens, 8192 * 64 * 128 // ((hq + hk) * d)))
        c = _norm("", tokens, hq, hk, d, parts, dtype, rng.random() < 0.5, rotary, rng.random() < 0.3,
                  max(tokens, 512))
    else:
        d = rng.choice([64, 128, 128, 128, 256])
        group = rng.choice([32, 64, 64])
        page = rng.choice([8, 16, 16, 32, 64, 24])
        if op == "append":
            batch = _log(rng, 1, 64)
            q_len = 1 if rng.random() < 0.5 else _log(rng, 2, 4096)
            kv = _log(rng, 16, 8192)
            q_len = max(1, min(q_len, 8192 * 48 * 128 // (batch * (hq + 2 * hk) * d)))
            c = _append("", batch, q_len, max(kv, q_len), hq, hk, d, parts, page, group, dtype, True,
                        rng.random() < 0.3)
        else:
            kind = rng.choice(["one", "one", "few", "chunk"])
            batch = _log(rng, 1, 64) if kind != "chunk" else _log(rng, 1, 8)
            q_len = 1 if kind == "one" else _log(rng, 2, 16) if kind == "few" else _log(rng, 64, 1024)
            if kind == "chunk":
                dtype = BF16
            kv = _log(rng, 16, 32768)
            budget = 131071 * 5 * 8 * 128 // 2
            kv = max(1, min(kv, budget // (batch * hk * d)))
            pairs = 3 * 1024 * 8000 * 32 * 128 // 2
            if dtype == FP32:
                pairs //= 64
            kv = max(1, min(kv, pairs // (batch * q_len * hq * d)))
            q_len = min(q_len, kv)
            window = rng.choice([0, 0, 0, 128, 1000])
            c = _attn("", batch, q_len, kv, hq, hk, d, parts, page, group, dtype, rng.random() < 0.8, window,
                      rng.random() < 0.85)
    del c["name"]
    return c


def _lengths(case):
    """New tokens and cached tokens (the new ones among them) of each sequence."""
    n, q, kv = case["batch"], case["q_len"], case["kv_len"]
    frac = [((i + 1) * 0.6180339887498949) % 1.0 if case["ragged"] else 1.0 for i in range(n)]
    if case["ragged"]:
        frac[0] = 1.0
    kvs = [max(1, int(kv * (0.1 + 0.9 * f))) if f < 1.0 else kv for f in frac]
    qs = [max(1, int(math.ceil(q * (0.25 + 0.75 * f)))) if f < 1.0 else q for f in frac]
    return [min(a, b) for a, b in zip(qs, kvs)], kvs


def _words(case):
    w = 2 * (case["d"] // 8) + 2 * (case["d"] // case["group"])
    return (w + 3) // 4 * 4


def _visible(case):
    """(keys that some query of the sequence sees, (query, key) pairs) over the batch."""
    keys = pairs = 0
    for q, kv in zip(*_lengths(case)):
        off, w = kv - q, case["window"]
        if not case["causal"]:
            keys, pairs = keys + kv, pairs + q * kv
            continue
        lo = max(0, off - w + 1) if w else 0
        keys += kv - lo
        full = q * off + q * (q + 1) // 2
        if w:  # query i sees min(off + i + 1, w) keys
            n = max(0, min(q, w - off))
            full = n * off + n * (n + 1) // 2 + (q - n) * w
        pairs += full
    return keys, pairs


def work(case):
    b = 2 if case["dtype"] == BF16 else 4
    d, hq, hk = case["d"], case["hq"], case["hk"]
    if case["op"] == "norm":
        t = case["tokens"]
        x = t * (hq + hk) * d
        table = t * case["rotary"] * 4 + t * 4
        # forward: read and write each element once; backward: read the gradient and the input, write one gradient
        return {"bytes": (3 if case["backward"] else 2) * x * b + table + 8 * d * (2 if case["backward"] else 1),
                "flops": x * (16 if case["backward"] else 8)}
    qs, kvs = _lengths(case)
    t = sum(qs)
    meta = sum((k + case["page"] - 1) // case["page"] for k in kvs) * 4 + case["batch"] * 8
    record = d + 8 * (d // case["group"])
    if case["op"] == "append":
        # read q, k, v; write q, the stored values of k and v, and the records
        return {"bytes": t * (2 * hq * d * b + 4 * hk * d * b + hk * record + d * 4) + meta,
                "flops": t * (hq * 3 + hk * 14) * d}
    keys, pairs = _visible(case)
    return {"bytes": keys * hk * record + 2 * t * hq * d * b + meta, "flops": 4.0 * pairs * hq * d}


# ------------------------------------------------------------------ inputs

def _split(x, parts):
    """The slots of a tensor split over its last dim."""
    return [s.contiguous() for s in x.chunk(parts, dim=-1)]


def _table(rows, rotary, device):
    """[rows, rotary] fp32: cosines, then sines, of position * theta^(-2 i / rotary)."""
    freq = THETA ** (-torch.arange(0, rotary, 2, device=device, dtype=torch.float64) / rotary)
    a = torch.arange(rows, device=device, dtype=torch.float64)[:, None] * freq
    return torch.cat([a.cos(), a.sin()], dim=1).float()


def _heads(gen, t, h, d, dtype):
    """Activations of a projection: unit scale, some heads and channels larger."""
    x = torch.randn(t, h, d, generator=gen, device="cuda")
    x *= torch.exp(0.3 * torch.randn(h, 1, generator=gen, device="cuda"))
    x *= torch.exp(0.5 * torch.randn(h, d, generator=gen, device="cuda"))
    return x.reshape(t, h * d).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(int(seed))
    d, hq, hk, p, dt = case["d"], case["hq"], case["hk"], case["parts"], _DT[case["dtype"]]
    st = {"case": case}
    if case["op"] == "norm":
        t = case["tokens"]
        st["q"], st["k"] = (_split(_heads(gen, t, h, d, dt), p) for h in (hq, hk))
        st["qw"], st["kw"] = (1 + 0.1 * torch.randn(d, generator=gen, device="cuda") for _ in range(2))
        st["table"] = _table(case["table"], case["rotary"], "cuda")
        # consecutive positions that begin somewhere in the table
        start = torch.randint(0, max(1, case["table"] - t + 1), (1,), generator=gen, device="cuda")
        st["pos"] = (torch.arange(t, device="cuda") + start).to(torch.int32)
        if case["backward"]:
            st["dq"], st["dk"] = (_split(torch.randn(t, h * d, generator=gen, device="cuda").to(dt), p)
                                  for h in (hq, hk))
    else:
        _prepare_cache(st, case, gen)
    if own:
        _handles(st)
    return st


def _prepare_cache(st, case, gen):
    d, hq, hk, p, dt = case["d"], case["hq"], case["hk"], case["parts"], _DT[case["dtype"]]
    qs, kvs = _lengths(case)
    n, t, ps = case["batch"], sum(qs), case["page"]
    need = [(k + ps - 1) // ps for k in kvs]
    pages, width = sum(need) + 3, max(need) + 1
    order = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)
    at = torch.full((n, width), -1, dtype=torch.int64)
    run_ = 0
    for i, c in enumerate(need):
        at[i, :c] = torch.arange(run_, run_ + c)
        run_ += c
    at = at.cuda()
    st["pages"] = torch.where(at >= 0, order[at.clamp(min=0)], torch.zeros_like(order[:1]))
    st["kv_lens"] = torch.tensor(kvs, dtype=torch.int32).cuda()
    starts = [0]
    for c in qs:
        starts.append(starts[-1] + c)
    st["q_starts"] = torch.tensor(starts, dtype=torch.int32).cuda()
    st["uniform"] = all(c == qs[0] for c in qs)
    st["q"] = _split(_heads(gen, t, hq, d, dt), p)
    # what the pages hold: keys with channels of their own scale and offset, values of unit scale
    ks = torch.exp(0.4 * torch.randn(hk, 1, d, generator=gen, device="cuda"))
    ko = 0.5 * torch.randn(hk, 1, d, generator=gen, device="cuda")
    cache = torch.empty(pages, hk, ps, _words(case), dtype=torch.int32, device="cuda")
    step = max(1, (1 << 25) // (hk * ps * d))
    for a in range(0, pages, step):
        e = min(pages, a + step)
        k = torch.randn(e - a, hk, ps, d, generator=gen, device="cuda") * ks + ko
        v = torch.randn(e - a, hk, ps, d, generator=gen, device="cuda")
        cache[a:e] = _pack(k, v, case)
    st["cache"] = [c.contiguous() for c in cache.chunk(p, dim=1)] if p > 1 else [cache]
    if case["op"] == "append":
        st["k"], st["v"] = (_split(_heads(gen, t, hk, d, dt), p) for _ in range(2))
        st["table"] = _table(max(kvs), d, "cuda")
    st["seq"] = torch.repeat_interleave(torch.arange(n), torch.tensor(qs)).cuda()
    st["row"] = torch.cat([torch.arange(c) for c in qs]).cuda()
    st["max_q"], st["max_kv"] = max(qs), max(kvs)


def _handles(st):
    """What a user of the library keeps: its distributed tensors over the slots above, outputs and workspaces."""
    import tensor_sharded_linear_gb300 as tsl
    c = st["case"]
    d, hq, hk, p, dt = c["d"], c["hq"], c["hk"], c["parts"], _DT[c["dtype"]]
    mesh = tsl.DeviceMesh((p,), ("tp",))
    rep, last = [tsl.Replicate()], [tsl.Shard(1)]

    def sharded(slots):
        return tsl.DTensor(slots, mesh, last, (slots[0].shape[0], sum(s.shape[1] for s in slots)), slots[0].dtype)

    def whole(x):
        return tsl.DTensor([x], mesh, rep, tuple(x.shape), x.dtype)

    h = st["h"] = {"tsl": tsl}
    t = st["q"][0].shape[0]
    for name in ("q", "k", "v", "dq", "dk"):
        if name in st:
            h[name] = sharded(st[name])
    if c["op"] == "norm":
        for name in ("qw", "kw", "table", "pos"):
            h[name] = whole(st[name])
        h["out"] = tuple(tsl.DTensor.empty(mesh, last, (t, n * d), dt) for n in (hq, hk))
        if c["backward"]:
            h["out"] += tuple(tsl.DTensor.empty(mesh, rep, (d,), torch.float32) for _ in range(2))
            h["workspace"] = torch.empty(max(256, tsl.tp_qk_norm_rope_backward_workspace_bytes(
                h["q"], h["k"], head_dim=d)), dtype=torch.uint8, device="cuda")
        return
    gshape = (st["cache"][0].shape[0], hk) + tuple(st["cache"][0].shape[2:])
    h["cache"] = tsl.DTensor(st["cache"], mesh, last, gshape, torch.int32)
    for name in ("pages", "kv_lens", "q_starts"):
        h[name] = whole(st[name])
    if st["uniform"]:
        h["q_starts"] = None
    h["out"] = tsl.DTensor.empty(mesh, last, (t, hq * d), dt)
    if c["op"] == "append":
        h["table"] = whole(st["table"])
        h["stored"] = tuple(tsl.DTensor.empty(mesh, last, (t, hk * d), dt) for _ in range(2))
    else:
        h["workspace"] = torch.empty(max(256, tsl.tp_kv4_attention_workspace_bytes(
            h["q"], h["cache"], h["pages"], head_dim=d, group=c["group"])), dtype=torch.uint8, device="cuda")


# ------------------------------------------------------------------ one pass

def run(st):
    if own:
        return _run_own(st)
    return {"norm": _plain_norm, "append": _plain_append, "attn": _plain_attention}[st["case"]["op"]](st)


def _run_own(st):
    c, h = st["case"], st["h"]
    tsl, d = h["tsl"], c["d"]
    if c["op"] == "norm":
        if c["backward"]:
            dq, dk, dqw, dkw = tsl.tp_qk_norm_rope_backward(
                h["dq"], h["dk"], h["q"], h["k"], h["qw"], h["kw"], h["table"], h["pos"], head_dim=d, eps=EPS,
                interleaved=c["interleaved"], out=h["out"], workspace=h["workspace"])
            return {"dq": dq.slots, "dk": dk.slots, "dqw": dqw.slots[0], "dkw": dkw.slots[0]}
        q, k = tsl.tp_qk_norm_rope(h["q"], h["k"], h["qw"], h["kw"], h["table"], h["pos"], head_dim=d, eps=EPS,
                                   interleaved=c["interleaved"], out=h["out"])
        return {"q": q.slots, "k": k.slots}
    if c["op"] == "append":
        q = tsl.tp_kv4_append(h["k"], h["v"], h["cache"], h["pages"], h["kv_lens"], h["q_starts"], q=h["q"],
                              cos_sin=h["table"], head_dim=d, group=c["group"], interleaved=c["interleaved"],
                              q_out=h["out"], stored=h["stored"])
        return {"q": q.slots, "k": h["stored"][0].slots, "v": h["stored"][1].slots, "cache": h["cache"].slots}
    o = tsl.tp_kv4_attention(h["q"], h["cache"], h["pages"], h["kv_lens"], h["q_starts"], head_dim=d,
                             group=c["group"], causal=c["causal"], window=c["window"], out=h["out"],
                             workspace=h["workspace"])
    return {"o": o.slots}


# -- the plain forms

def _rotate(x, cos, sin, interleaved, back=False):
    """x [..., D] with its first 2 * cos.shape[-1] channels rotated in pairs (back: by minus the angle)."""
    r = cos.shape[-1]
    if back:
        sin = -sin
    if interleaved:
        a, b = x[..., 0:2 * r:2], x[..., 1:2 * r:2]
        y = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :r], x[..., r:2 * r]
        y = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([y, x[..., 2 * r:]], dim=-1)


def _angles(table, pos):
    row = table[pos.long()][:, None, :]
    return row.chunk(2, dim=-1)


def _plain_norm(st):
    c = st["case"]
    d, dt = c["d"], _DT[c["dtype"]]
    cos, sin = _angles(st["table"], st["pos"])
    out = {}
    for name, w in (("q", st["qw"]), ("k", st["kw"])):
        x = torch.cat(st[name], dim=-1).float().unflatten(-1, (-1, d))
        rstd = 1.0 / (x.square().mean(-1, keepdim=True) + EPS).sqrt()
        if not c["backward"]:
            y = _rotate(x * rstd * w, cos, sin, c["interleaved"])
            out[name] = _split(y.flatten(-2).to(dt), c["parts"])
            continue
        g = torch.cat(st["d" + name], dim=-1).float().unflatten(-1, (-1, d))
        g = _rotate(g, cos, sin, c["interleaved"], back=True)
        xhat = x * rstd
        out["d" + name + "w"] = (g * xhat).sum((0, 1))
        g = g * w
        dx = rstd * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        out["d" + name] = _split(dx.flatten(-2).to(dt), c["parts"])
    return out


def _quantise(x, group):
    """x [..., D] as codes [..., D/G, G] (float), steps and minima [..., D/G, 1], bf16-rounded."""
    x = x.unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    m = lo.to(torch.bfloat16).float()
    s = ((hi - lo) * 0.06666667014360428).to(torch.bfloat16).float()
    one = torch.ones_like(s)
    inv = torch.where(s >= 2.0 ** -126, one / s, torch.zeros_like(s))
    return ((x - m) * inv).round().clamp(0, 15), s, m


def _pack(k, v, case):
    """Records [..., words] of keys and values [..., D]."""
    words = []
    params = []
    for x in (k, v):
        c, s, m = _quantise(x, case["group"])
        c = c.to(torch.int32).flatten(-2).unflatten(-1, (-1, 8))
        shift = torch.arange(0, 32, 4, device=x.device, dtype=torch.int32)
        words.append((c << shift).sum(-1, dtype=torch.int32))
        sb, mb = (z.squeeze(-1).to(torch.bfloat16).view(torch.int16).to(torch.int32) for z in (s, m))
        params.append((sb & 0xFFFF) | (mb << 16))
    rec = torch.cat(words + params, dim=-1)
    pad = _words(case) - rec.shape[-1]
    return torch.cat([rec, rec.new_zeros(rec.shape[:-1] + (pad,))], dim=-1) if pad else rec


def _plain_append(st):
    c = st["case"]
    d, dt, p, ps = c["d"], _DT[c["dtype"]], c["parts"], c["page"]
    q_lens = st["q_starts"][1:] - st["q_starts"][:-1]
    pos = (st["kv_lens"] - q_lens)[st["seq"]] + st["row"]
    cos, sin = _angles(st["table"], pos)
    q, k, v = (torch.cat(st[n], dim=-1).float().unflatten(-1, (-1, d)) for n in ("q", "k", "v"))
    q, k = (_rotate(x, cos, sin, c["interleaved"]) for x in (q, k))
    rec = _pack(k, v, c)
    cache = torch.cat(st["cache"], dim=1) if p > 1 else st["cache"][0].clone()
    cache[st["pages"][st["seq"], pos // ps].long(), :, pos % ps] = rec
    stored = []
    for x in (k, v):
        code, s, m = _quantise(x, c["group"])
        stored.append(_split((code * s + m).flatten(-3).to(dt), p))
    return {"q": _split(q.flatten(-2).to(dt), p), "k": stored[0], "v": stored[1],
            "cache": [x.contiguous() for x in cache.chunk(p, dim=1)]}


def _unpack(words, params, group):
    """fp32 values [..., D] of code words [..., D/8] and parameter words [..., D/G]."""
    shift = torch.arange(0, 32, 4, device=words.device, dtype=torch.int32)
    c = ((words[..., None] >> shift) & 15).flatten(-2).float().unflatten(-1, (-1, group))
    s = (params & 0xFFFF).to(torch.int16).view(torch.bfloat16).float()
    m = (params >> 16).to(torch.int16).view(torch.bfloat16).float()
    return (c * s[..., None] + m[..., None]).flatten(-2)


def _plain_attention(st):
    c = st["case"]
    d, dt, p, ps, hk = c["d"], _DT[c["dtype"]], c["parts"], c["page"], c["hk"]
    n, g = c["batch"], c["hq"] // c["hk"]
    w, ng = d // 8, d // c["group"]
    mq, mk = st["max_q"], st["max_kv"]
    # each sequence's records, padded to the longest: [n, mk, hk, words]
    key = torch.arange(mk, device="cuda")
    cache = torch.cat(st["cache"], dim=1) if p > 1 else st["cache"][0]
    rec = cache[st["pages"][:, key // ps].long(), :, (key % ps)[None, :]].transpose(1, 2)
    k = _unpack(rec[..., :w], rec[..., 2 * w:2 * w + ng], c["group"])
    v = _unpack(rec[..., w:2 * w], rec[..., 2 * w + ng:2 * w + 2 * ng], c["group"])
    # the queries, padded to the longest: [n, hk, g * mq, d]
    x = torch.cat(st["q"], dim=-1).float().unflatten(-1, (hk, g, d))
    q = x.new_zeros(n, mq, hk, g, d)
    q[st["seq"], st["row"]] = x
    s = torch.matmul(q.permute(0, 2, 3, 1, 4).reshape(n, hk, g * mq, d), k.transpose(-1, -2)) * (1.0 / math.sqrt(d))
    s = s.unflatten(2, (g, mq))
    kv = st["kv_lens"][:, None, None]
    at = (kv - (st["q_starts"][1:] - st["q_starts"][:-1])[:, None, None]) + torch.arange(mq, device="cuda")[:, None]
    see = (key < kv) & torch.ones_like(at, dtype=torch.bool)
    if c["causal"]:
        see = see & (key <= at)
        if c["window"]:
            see = see & (key > at - c["window"])
    s = s.masked_fill_(~see[:, None, None], -math.inf)
    top = s.amax(-1, keepdim=True).clamp(min=-3e38)
    s = s.sub_(top).exp_()
    o = torch.matmul(s.flatten(2, 3), v) / s.sum(-1).flatten(2, 3).unsqueeze(-1).clamp(min=1e-30)
    o = o.unflatten(2, (g, mq)).permute(0, 3, 1, 2, 4)[st["seq"], st["row"]]
    return {"o": _split(o.flatten(1).to(dt), p)}


# ------------------------------------------------------------------ the definition, in 64 bits

def _turn(x, table, pos, interleaved):
    """Each pair (a, b) of x [t, h, d] as the complex number a + i b, times e^(i angle) from the table's row."""
    r = table.shape[1] // 2
    e = torch.complex(table[:, :r].double(), table[:, r:].double())[pos.long()][:, None, :]
    y = x.clone()
    ia = torch.arange(r, device=x.device) * (2 if interleaved else 1)
    ib = ia + (1 if interleaved else r)
    z = torch.complex(x[..., ia], x[..., ib]) * e
    y[..., ia], y[..., ib] = z.real, z.imag
    return y


def exact(case, seed):
    st = prepare(case, seed)
    d, p = case["d"], case["parts"]
    cut = lambda y: list(y.flatten(1).chunk(p, dim=1))  # noqa: E731
    whole = lambda s: torch.cat([t.double() for t in s], dim=1).reshape(s[0].shape[0], -1, d)  # noqa: E731
    if case["op"] == "norm":
        out = {}
        for name, w in (("q", st["qw"]), ("k", st["kw"])):
            x = whole(st[name]).requires_grad_(case["backward"])
            wd = w.double().requires_grad_(case["backward"])
            if not case["backward"]:
                out[name] = cut(_turn(x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * wd, st["table"],
                                      st["pos"], case["interleaved"]))
                continue
            # <dy, R z> = <R^T dy, z>: the rotation is undone with the conjugate table
            r = st["table"].shape[1] // 2
            conj = torch.cat([st["table"][:, :r], -st["table"][:, r:]], dim=1)
            dz = _turn(whole(st["d" + name]), conj, st["pos"], case["interleaved"])
            z = x / (x.pow(2).sum(-1, keepdim=True) / d + EPS).sqrt() * wd
            dx, dw = torch.autograd.grad((z * dz).sum(), (x, wd))
            out["d" + name], out["d" + name + "w"] = cut(dx), dw
        return out
    qs, kvs = _lengths(case)
    ps = case["page"]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(kv - q, kv) for q, kv in zip(qs, kvs)]).cuda()
        k = _turn(whole(st["k"]), st["table"], pos, case["interleaved"])
        out = {"q": cut(_turn(whole(st["q"]), st["table"], pos, case["interleaved"])),
               "cache": [None for _ in range(p)]}
        for name, x in (("k", k), ("v", whole(st["v"]))):
            x = x.reshape(x.shape[0], x.shape[1], d // case["group"], case["group"])
            lo, hi = x.min(-1, keepdim=True).values, x.max(-1, keepdim=True).values
            m, s = lo.bfloat16().double(), ((hi - lo) / 15).bfloat16().double()
            code = torch.where(s > 0, ((x - m) / s.clamp(min=1e-300)).round().clamp(0, 15), torch.zeros_like(x))
            out[name] = cut((m + code * s).flatten(-2))
        return out
    hk, g = case["hk"], case["hq"] // case["hk"]
    w, ng = d // 8, d // case["group"]
    q = whole(st["q"])
    cache = torch.cat(st["cache"], dim=1)
    outs, t0 = [], 0
    for b, (nq, kv) in enumerate(zip(qs, kvs)):
        pos = torch.arange(kv, device="cuda")
        rec = cache[st["pages"][b].long()[pos // ps], :, pos % ps]  # [kv, hk, words]
        vals = []
        for a, pa in ((0, 2 * w), (w, 2 * w + ng)):
            code = torch.stack([(rec[..., a:a + w] >> (4 * i)) & 15 for i in range(8)], -1)
            par = rec[..., pa:pa + ng].contiguous().view(torch.bfloat16).reshape(kv, hk, ng, 2).double()
            code = code.reshape(kv, hk, ng, case["group"]).double()
            vals.append((par[..., 1:2] + code * par[..., 0:1]).reshape(kv, hk, d))
        at = torch.arange(kv - nq, kv, device="cuda")
        see = torch.ones(nq, kv, dtype=torch.bool, device="cuda")
        if case["causal"]:
            see = pos[None, :] <= at[:, None]
            if case["window"]:
                see = see & (pos[None, :] > at[:, None] - case["window"])
        rows = []
        for h in range(case["hq"]):
            s = q[t0:t0 + nq, h] @ vals[0][:, h // g].T / math.sqrt(d)
            rows.append(torch.softmax(s.masked_fill(~see, -math.inf), -1) @ vals[1][:, h // g])
        outs.append(torch.stack(rows, 1))
        t0 += nq
    return {"o": cut(torch.cat(outs, 0))}
