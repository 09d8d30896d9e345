"""Block norms (norm, gate, dropout, residual, norm) and their gradients against the 64-bit restatement.

Bounds.  An output is rounded once to its type (half a step).  Before that it
is computed in fp32 (half a step is 2^-24): each term of its formula is a
product of at most 10 factors that are each rounded once or twice, and of up to
three reciprocal roots and means, each of a sum over n channels.  Such a sum
adds at most ceil(n / 32) numbers in a row (a thread's own) and 16 on the way
through the CTA, so it is off by (ceil(n / 32) + 16) half steps of the sum of
magnitudes, and what it enters by as many.  K below counts all of them; where a
formula's terms cancel (parts of x, residual and branch), what a rounding does
is relative to their magnitudes, so K multiplies the sum of magnitudes that the
restatement returns with each value, times the worst row's ratio of magnitudes
to values in the norms.  Sums over tokens add as many numbers in a row as a CTA
has tokens, and 40 more.
"""
import numpy as np
import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from heads_helpers import DT, draw, full, strided, whole
from oracle import decoder

pytestmark = pytest.mark.gpu
HALF = {"bf16": 2.0 ** -8, "fp32": 2.0 ** -24}
R, S0, PART = tsl.Replicate(), tsl.Shard(0), tsl.Partial()


def rows(x, mesh, dtype, place, extra=0, offset=0):
    """[tokens, n] values (a list of them: parts) as a DTensor of row blocks."""
    xs = x if isinstance(x, list) else [x]
    ts = [torch.from_numpy(np.ascontiguousarray(v)).cuda().to(DT[dtype]) for v in xs]
    if place == S0:
        c = -(-ts[0].shape[0] // mesh.shape[0])
        ts = [ts[0][min(i * c, len(ts[0])):(i + 1) * c] for i in range(mesh.shape[0])]
    shape = xs[0].shape
    return tsl.DTensor([strided(t, extra, offset) for t in ts], mesh, [place], shape, DT[dtype])


def got(d):
    return np.concatenate([s.detach().double().cpu().numpy() for s in d.slots], 0)


class Case:
    def __init__(self, seed, t, n, p=1, place=R, out=R, dtype="bf16", stream=None, res=True, post=True, gate=0,
                 pre=True, drop=0.0, scale=1.0, eps=1e-6, extra=0, offset=0, wdtype="fp32", zero_row=False, x_scale=None):
        rng = np.random.default_rng(seed)
        self.mesh = mesh = tsl.DeviceMesh((p,), ("tp",))
        self.t, self.n, self.dtype, self.stream = t, n, dtype, stream or dtype
        x_scale = 1 / np.sqrt(p) if x_scale is None else x_scale
        parts = [draw(rng, (t, n), dtype, x_scale) for _ in range(p if place == PART else 1)]
        r = draw(rng, (t, n), self.stream, 2.0) if res else None
        if zero_row:
            for x in parts:
                x[t // 2] = 0
            if res:
                r[t // 2] = 0
        vec = lambda *s: draw(rng, s, wdtype)  # noqa: E731
        post, pre = vec(n) if post else None, vec(n) if pre else None
        gate = (vec(n) if gate < 0 else vec(gate, n)) if gate else None
        seed4 = rng.integers(-2 ** 31, 2 ** 31, 4)
        keep = decoder.keep_mask(seed4, t, n, drop) if drop else None
        self.ref = decoder.Block(parts, r, post, gate, pre, eps, scale, keep, drop)
        lay = dict(extra=extra, offset=offset)
        self.x = rows(parts if place == PART else parts[0], mesh, dtype, place, **lay)
        self.r = None if r is None else rows(r, mesh, self.stream, out, **lay)
        w = lambda v: None if v is None else whole(v, mesh, DT[wdtype])  # noqa: E731
        self.post, self.gate, self.pre = w(post), w(gate), w(pre)
        self.rng = whole(torch.tensor(seed4, dtype=torch.int32), mesh) if drop else None
        self.dh, self.dy = draw(rng, (t, n), self.stream), draw(rng, (t, n), dtype) if self.pre else None
        self.gh = rows(self.dh, mesh, self.stream, out, **lay)
        self.gy = rows(self.dy, mesh, dtype, out, **lay) if self.pre else None
        self.kw = dict(eps=eps, residual_scale=scale, dropout=drop, rng=self.rng)
        z = lambda d, pl: rows(np.zeros((t, n)), mesh, d, pl, **lay)  # noqa: E731
        self.fwd_out = (z(self.stream, out), z(dtype, out) if self.pre else None)
        self.bwd_out = (z(dtype, R if place == PART else place), z(self.stream, out) if res else None,
                        *(None if v is None else whole(torch.zeros(v.gshape), mesh, DT[wdtype])
                          for v in (self.post, self.gate, self.pre)))
        self.wdtype = wdtype
        ref = self.ref
        with np.errstate(divide="ignore", invalid="ignore"):
            ratio = [(ref.abs_s ** 2).sum(1) / (ref.s ** 2).sum(1), (ref.abs_h ** 2).sum(1) / (ref.h ** 2).sum(1)]
        ratio = np.nanmax(np.where(np.isfinite(ratio), ratio, 1.0)) if t and n else 1.0
        self.k = (10 * 2 + len(parts) + 3 * (-(-n // 32) + 16)) * ratio * 2.0 ** -24

    def operands(self):
        return self.x, self.r, self.post, self.gate, self.pre

    def forward(self):
        return tsl.tp_block_norm(*self.operands(), out=self.fwd_out, **self.kw)

    def backward(self):
        return tsl.tp_block_norm_backward(self.gh, self.gy, *self.operands(), out=self.bwd_out, **self.kw)

    def check_forward(self, h, y):
        ref = self.ref
        err = np.abs(got(h) - ref.h)
        assert (err <= HALF[self.stream] * np.abs(ref.h) + self.k * ref.abs_h + 1e-37).all(), ("h", err.max())
        if y is not None:
            err = np.abs(got(y) - ref.y)
            assert (err <= HALF[self.dtype] * np.abs(ref.y) + self.k * ref.abs_y + 1e-37).all(), ("y", err.max())

    def check_backward(self, out):
        ref = self.ref.backward(self.dh, self.dy)
        chain = (-(-self.t // 152) + 40) * 2.0 ** -24
        for name, d in zip(("dx", "dr", "dpost", "dgate", "dpre"), out):
            if d is None:
                continue
            e, mag = ref[name]
            g = got(d) if name in ("dx", "dr") else d.slots[0].double().cpu().numpy()
            half = HALF[self.dtype if name == "dx" else self.stream if name == "dr" else self.wdtype]
            k = self.k * 2 if name in ("dx", "dr") else self.k * 2 + chain  # (gradients: two norms, one in the other)
            err = np.abs(g - e)
            assert (err <= half * np.abs(e) + k * mag + 1e-37).all(), (name, err.max(), (err / (mag + 1e-30)).max())


CASES = [
    dict(t=1, n=4096), dict(t=8, n=4096, p=4, place=PART), dict(t=5, n=1), dict(t=3, n=2, gate=-1), dict(t=9, n=7),
    dict(t=2, n=8, gate=2), dict(t=37, n=64, p=2, place=S0, out=S0), dict(t=300, n=1000, p=4, place=S0, out=R, gate=3),
    dict(t=301, n=1001, p=4, place=R, out=S0, gate=-1), dict(t=33, n=8192, p=8, place=PART, out=S0, scale=0.5),
    dict(t=7, n=16384, gate=7), dict(t=5, n=20000, p=2, place=PART), dict(t=6, n=4093, p=3, place=PART, out=S0),
    dict(t=700, n=128, gate=-1, drop=0.5), dict(t=513, n=1152, stream="fp32", gate=9, drop=0.1),
    dict(t=330, n=512, dtype="fp32", p=2, place=S0, out=S0, gate=165, drop=0.25, scale=-1.5),
    dict(t=19, n=8200, dtype="fp32", drop=0.9), dict(t=40, n=4096, post=False, drop=0.1, p=4, place=S0, out=S0),
    dict(t=40, n=4096, post=False, pre=False, res=False, drop=0.3), dict(t=64, n=2048, post=False, res=False),
    dict(t=12, n=1024, pre=False, gate=-1), dict(t=12, n=1024, res=False, gate=12), dict(t=12, n=1024, wdtype="bf16",
                                                                                        gate=4),
    dict(t=50, n=4096, extra=8), dict(t=50, n=4096, extra=3, offset=1), dict(t=21, n=1000, offset=4, drop=0.5, gate=3),
    dict(t=20, n=256, zero_row=True, gate=-1), dict(t=3, n=4096, p=64, place=PART, out=S0),
    dict(t=70, n=96, p=64, place=S0, out=S0), dict(t=2000, n=32, gate=1000), dict(t=1700, n=5120, gate=-1, p=4,
                                                                                 place=S0, out=S0, drop=0.1),
    dict(t=640, n=16384, p=2, place=S0, out=S0, gate=-1), dict(t=9, n=12288, dtype="fp32", gate=-1, drop=0.2),
]


def ids(c):
    return "-".join(f"{k}{type(v).__name__ if k in ('place', 'out') else v}" for k, v in c.items())


@pytest.mark.parametrize("c", CASES, ids=ids)
def test_block_norm(c):
    case = Case(11, **c)
    case.check_forward(*case.forward())
    case.check_backward(case.backward())
    assert tsl.read_device_status() == 0


@pytest.mark.parametrize("c", CASES[6:20:3], ids=ids)
def test_same_inputs_same_bits(c):
    case = Case(12, **c)
    first = [[s.clone() for s in d.slots] for d in (*case.forward(), *case.backward()) if d is not None]
    case.forward()
    again = [d.slots for d in (*case.fwd_out, *case.backward()) if d is not None]
    for a, b in zip(first, again):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_results_do_not_depend_on_the_layout():
    """Dropout's mask and every sum of a row are those of the row, wherever it lies."""
    outs = []
    for p, place, out in ((1, R, R), (4, S0, R), (4, R, S0), (3, S0, S0)):
        case = Case(13, 50, 768, p=p, place=place, out=out, drop=0.4, gate=5, x_scale=1.0)
        outs.append([got(d) for d in case.forward()])
    for o in outs[1:]:
        assert all(np.array_equal(a, b) for a, b in zip(o, outs[0]))


@pytest.mark.parametrize("n", [1024, 1001])
def test_dropped_elements_do_not_reach_anything(n):
    """Infinities and NaN of x in dropped places, without a norm over x."""
    case = Case(14, 30, n, post=False, drop=0.5, gate=-1)
    bad = torch.from_numpy(~case.ref.keep).cuda()
    for v in (float("nan"), float("inf")):
        case.x.slots[0][bad] = v
        case.check_forward(*case.forward())
        case.check_backward(case.backward())


@pytest.mark.parametrize("n", [512, 333])
def test_rows_keep_to_themselves(n):
    """A row of NaN and one of infinities spoil their own results only, and the sums over tokens."""
    case = Case(15, 40, n, p=2, place=S0, out=S0)
    case.x.slots[0][3] = float("nan")
    case.r.slots[1][5] = float("inf")
    h, y = case.forward()
    dx, dr = case.backward()[:2]
    ok = np.ones(40, bool)
    ok[[3, 25]] = False
    ref = case.ref.backward(case.dh, case.dy)
    for d, e in ((h, case.ref.h), (y, case.ref.y), (dx, ref["dx"][0]), (dr, ref["dr"][0])):
        g = got(d)
        assert np.isfinite(g[ok]).all() and np.abs(g[ok] - e[ok]).max() <= 0.05 * np.abs(e[ok]).max()
    assert np.isnan(got(y)[3]).all() and np.isnan(got(y)[25]).any()


@pytest.mark.parametrize("n", [1024, 999])
def test_what_lies_beside_the_rows_stays(n):
    case = Case(16, 21, n, extra=24, offset=8, gate=-1)
    outs = [d for d in (*case.fwd_out, *case.bwd_out[:2])]
    case.forward()
    case.backward()
    for d in outs:
        s = d.slots[0]
        base = torch.as_strided(s, (21, n + 24), (n + 24, 1))[:-1, n:]
        assert (base == 7).all()


def test_outputs_that_are_not_wanted():
    case = Case(17, 10, 640, gate=-1)
    h, y = case.forward()
    none, y2 = tsl.tp_block_norm(*case.operands(), out=(None, rows(np.zeros((10, 640)), case.mesh, "bf16", R)), **case.kw)
    assert none is None and torch.equal(y2.slots[0], y.slots[0])
    want = [d.slots[0].clone() for d in case.backward()]
    out = (None, None, *case.bwd_out[2:])
    again = tsl.tp_block_norm_backward(case.gh, case.gy, *case.operands(), out=out, **case.kw)
    assert again[0] is None and all(torch.equal(a.slots[0], b) for a, b in zip(again[2:], want[2:]))
    # without dh: the gradient of y alone
    dx = tsl.tp_block_norm_backward(None, case.gy, *case.operands(), **case.kw)[0]
    e, mag = case.ref.backward(None, case.dy)["dx"]
    assert (np.abs(got(dx) - e) <= HALF["bf16"] * np.abs(e) + 2 * case.k * mag).all()


def test_default_outputs_and_leading_dims():
    mesh = tsl.DeviceMesh((2, 2), ("dp", "tp"))
    rng = np.random.default_rng(18)
    x = [draw(rng, (4, 6, 64), "bf16") for _ in range(2)]
    r = draw(rng, (4, 6, 64), "fp32")
    pre = draw(rng, (64,), "fp32")
    t = lambda v, d: torch.from_numpy(v).cuda().to(DT[d])  # noqa: E731
    xd = tsl.DTensor([t(x[p][2 * i:2 * i + 2], "bf16") for i in range(2) for p in range(2)], mesh, [S0, PART],
                     (4, 6, 64), torch.bfloat16)
    rd = tsl.DTensor([t(r[i:i + 1], "fp32") for i in range(4)], mesh, [S0, S0], (4, 6, 64), torch.float32)
    w = tsl.DTensor([t(pre, "fp32")], mesh, [R, R], (64,), torch.float32)
    h, y = tsl.tp_block_norm(xd, rd, pre_weight=w)
    assert h.placements == y.placements == (S0, S0) and h.dtype == torch.float32 and y.dtype == torch.bfloat16
    ref = decoder.Block([v.reshape(24, 64) for v in x], r.reshape(24, 64), pre=pre)
    assert np.abs(got(h).reshape(24, 64) - ref.h).max() <= 2.0 ** -20
    assert (np.abs(got(y).reshape(24, 64) - ref.y) <= 2.0 ** -8 * np.abs(ref.y) + 2.0 ** -18).all()
    dx, dr, _, _, dw = tsl.tp_block_norm_backward(h, y, xd, rd, pre_weight=w)
    assert dx.placements == (S0, R) and dx.dtype == torch.bfloat16 and dr.placements == (S0, S0)
    e = ref.backward(got(h).reshape(24, 64), got(y).reshape(24, 64))
    assert (np.abs(got(dr).reshape(24, 64) - e["dr"][0]) <= 2.0 ** -18 * (1 + e["dr"][1])).all()
    assert (np.abs(dw.slots[0].double().cpu().numpy() - e["dpre"][0]) <= 2.0 ** -18 * (1 + e["dpre"][1])).all()


def test_gradient_against_differences():
    """The directional derivative of the library's own forward in fp32, central differences."""
    case = Case(19, 12, 256, dtype="fp32", gate=3, drop=0.25, eps=1e-3)
    grads = case.backward()
    rng = np.random.default_rng(20)

    def loss():
        h, y = case.forward()
        return (got(h) * case.dh).sum() + (got(y) * case.dy).sum()

    for d, g in zip(case.operands(), grads):
        v = torch.from_numpy(rng.standard_normal(d.slots[0].shape)).float().cuda()
        step = 2.0 ** -8
        d.slots[0] += step * v
        up = loss()
        d.slots[0] -= 2 * step * v
        down = loss()
        d.slots[0] += step * v
        want = (g.slots[0].double() * v.double()).sum().item()
        size = (g.slots[0].double() * v.double()).abs().sum().item()
        # the third derivative's share is about step^2; the forward's roundings, 2^-22 of the loss's terms, over 2 step
        noise = 2.0 ** -22 * (np.abs(case.ref.h * case.dh).sum() + np.abs(case.ref.y * case.dy).sum()) / (2 * step)
        assert abs((up - down) / (2 * step) - want) <= 2.0 ** -8 * size + noise


@pytest.mark.parametrize("n", [768, 771])
def test_captured_with_new_inputs_and_masks(n):
    case = Case(21, 24, n, drop=0.5, gate=-1)
    case.forward(), case.backward()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    g = torch.cuda.CUDAGraph()
    ws = torch.empty(tsl.tp_block_norm_backward_workspace_bytes(case.x, case.post, case.gate, case.pre),
                     dtype=torch.uint8, device="cuda")
    with torch.cuda.graph(g, stream=stream):
        case.forward()
        tsl.tp_block_norm_backward(case.gh, case.gy, *case.operands(), out=case.bwd_out, workspace=ws, **case.kw)
    new = Case(22, 24, n, drop=0.5, gate=-1)
    for a, b in zip((*case.operands(), case.rng, case.gh, case.gy), (*new.operands(), new.rng, new.gh, new.gy)):
        a.slots[0].copy_(b.slots[0])
    for _ in range(2):
        g.replay()
    torch.cuda.synchronize()
    new.check_forward(*case.fwd_out)
    new.check_backward(case.bwd_out)


def test_two_streams_with_their_own_workspaces():
    cases = [Case(23 + i, 500, 1536, gate=-1) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(5):
        for c, s in zip(cases, streams):
            with torch.cuda.stream(s):
                c.forward()
                c.backward()
    torch.cuda.synchronize()
    for c in cases:
        c.check_forward(*c.fwd_out)
        c.check_backward(c.bwd_out)


def test_no_tokens_give_zero_weight_gradients():
    case = Case(25, 0, 48, gate=-1)
    case.forward()
    out = [d.slots[0] for d in tsl.tp_block_norm_backward(case.gh, case.gy, *case.operands(), out=case.bwd_out,
                                                          **case.kw)[2:]]
    for d in out:
        d.fill_(3)
    case.backward()
    assert all((d == 0).all() for d in out)


@pytest.mark.parametrize("dtype,stream", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("n", [9, 255, 263, 1003, 4096])
def test_rows_at_every_distance_from_a_16_byte_boundary(n, dtype, stream):
    """Rows 1 to 8 elements off the boundary, with other numbers between them that have to stay."""
    for offset in range(1, 9):
        case = Case(28 + offset, 11, n, p=2, place=S0, out=S0, dtype=dtype, stream=stream, gate=-1, extra=offset % 3,
                    offset=offset, wdtype=dtype)
        beside = []
        for d in case.fwd_out:
            for s in d.slots:
                flat = torch.as_strided(s, (s.untyped_storage().size() // s.element_size(),), (1,), 0)
                flat.fill_(7)
                mask = torch.ones_like(flat, dtype=torch.bool)
                torch.as_strided(mask, s.shape, s.stride(), s.storage_offset()).fill_(False)
                beside.append((flat, mask))
        case.check_forward(*case.forward())
        for flat, mask in beside:
            assert (flat[mask] == 7).all()


IN_PLACE = [dict(t=7, n=512), dict(t=700, n=4096, drop=0.1), dict(t=600, n=1001, p=2, place=S0, out=S0, gate=3),
            dict(t=9, n=20000), dict(t=300, n=1152, dtype="fp32"), dict(t=320, n=16384, gate=-1)]


@pytest.mark.parametrize("c", IN_PLACE, ids=ids)
def test_results_in_place_of_operands(c):
    """The same bits as with outputs of their own."""
    def fresh():
        return Case(27, **c)

    def same(a, b):
        assert all(torch.equal(u, v) for u, v in zip(a.slots, b.slots))

    one = fresh()
    h, y = one.forward()
    want = one.backward()
    case = fresh()
    got_h, got_y = tsl.tp_block_norm(*case.operands(), out=(case.r, case.x), **case.kw)
    same(got_h, h)
    same(got_y, y)
    for over in (lambda k: (k.x, k.r), lambda k: (k.gy, k.gh), lambda k: (k.gy, k.r)):
        case = fresh()
        dx, dr = over(case)
        out = tsl.tp_block_norm_backward(case.gh, case.gy, *case.operands(), out=(dx, dr, *case.bwd_out[2:]), **case.kw)
        for a, b in zip(out, want):
            if b is not None:
                same(a, b)


@pytest.mark.parametrize("n,wdtype", [(1001, "bf16"), (77, "fp32"), (1024, "bf16"), (20001, "bf16")])
def test_a_gate_for_every_token(n, wdtype):
    """Its gradient has the tokens' rows, off 16-byte boundaries too, and goes out without sums over tokens."""
    case = Case(40, 23, n, p=2, place=S0, out=R, gate=23, wdtype=wdtype, drop=0.2)
    case.check_forward(*case.forward())
    case.check_backward(case.backward())


@pytest.mark.parametrize("n", [512, 1001])
def test_one_row_for_all_tokens(n):
    """Rows without a step between them (x and the residual broadcast), and one replica of several."""
    case = Case(41, 9, n, gate=-1)
    for d in (case.x, case.r):
        d.slots[0].copy_(d.slots[0][:1].clone().expand(9, n))
    want = [d.slots[0] for d in case.forward()] + [d.slots[0] for d in case.backward()]
    mesh = tsl.DeviceMesh((2,), ("tp",))

    def again(d, broadcast=False):
        t = d.slots[0]
        t = t[:1].expand(9, n) if broadcast else t
        return tsl.DTensor([t, t.clone()], mesh, [R], d.gshape, d.dtype, materialize_replicas=True)

    ops = (again(case.x, True), again(case.r, True), again(case.post), again(case.gate), again(case.pre))
    out = tsl.tp_block_norm(*ops, **case.kw) + tsl.tp_block_norm_backward(again(case.gh), again(case.gy), *ops, **case.kw)
    assert all(torch.equal(a.slots[0], b) for a, b in zip(out, want))


def test_empty_sequences_give_zero_gate_gradients():
    mesh = tsl.DeviceMesh((1,), ("tp",))
    empty = lambda: whole(torch.zeros(5, 0, 64), mesh, torch.bfloat16)  # noqa: E731
    w, gate = whole(torch.ones(64), mesh), whole(torch.ones(5, 64), mesh)
    out = (empty(), None, None, whole(torch.full((5, 64), 3.0), mesh), whole(torch.full((64,), 3.0), mesh))
    tsl.tp_block_norm_backward(None, empty(), empty(), None, None, gate, w, out=out)
    assert all((d.slots[0] == 0).all() for d in out[3:])


def test_offsets_past_32_bits():
    """Rows beyond 2^32 bytes and elements beyond 2^32, dropout's counter among them."""
    n, t = 8192, (1 << 32) // 8192 + 3
    mesh = tsl.DeviceMesh((1,), ("tp",))
    x = torch.empty(t, n, dtype=torch.bfloat16, device="cuda").normal_()
    rng = whole(torch.tensor([1, 2, 3, 4], dtype=torch.int32), mesh)
    pre = torch.randn(n, device="cuda")
    y = tsl.DTensor([torch.empty_like(x)], mesh, [R], x.shape, x.dtype)
    xd = tsl.DTensor([x], mesh, [R], x.shape, x.dtype)
    tsl.tp_block_norm(xd, pre_weight=whole(pre, mesh), dropout=0.5, rng=rng, out=(None, y))
    keep = decoder.keep_mask([1, 2, 3, 4], 3, n, 0.5, first=t - 3)
    ref = decoder.Block([x[-3:].double().cpu().numpy()], pre=pre.double().cpu().numpy(), keep=keep, p=0.5)
    g = y.slots[0][-3:].double().cpu().numpy()
    assert (np.abs(g - ref.y) <= 2.0 ** -8 * np.abs(ref.y) + 2.0 ** -14 * ref.abs_y).all()
