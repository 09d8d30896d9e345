"""Calls that share a kernel and differ in the shared memory they need: from native threads at once, and in one graph."""
import ctypes as C
import subprocess

import pytest
import torch

import tensor_sharded_linear_gb300 as tsl
from tensor_sharded_linear_gb300 import _lib
from tensor_sharded_linear_gb300.api import _ref

pytestmark = pytest.mark.gpu
R = tsl.Replicate()

# Python's threads hand each other the interpreter between calls; these call without it.
CALLER = r"""
#include <cstddef>
#include <cstdint>
#include <thread>
#include <vector>
typedef int (*Gradients)(const void*, const void*, const void*, const void*, const void*, const void*, const void*,
                         const void*, const void*, const void*, const void*, const void*, const void*, float, float, float,
                         int32_t, void*, size_t, int32_t*, void*);
typedef int (*LogProbs)(const void*, const void*, const void*, const void*, const void*, const void*, const void*, float,
                        int32_t, int32_t, int32_t*, void*);
struct Call {
  void* entry;
  int32_t gradients, rounds, status;
  const void* d[13];
  void* workspace;
  size_t bytes;
  void* stream;
};
extern "C" void run(Call* calls, int n) {
  std::vector<std::thread> threads;
  for (Call* c = calls; c != calls + n; ++c)
    threads.emplace_back([c] {
      const void* const* d = c->d;
      for (int i = 0; i < c->rounds && c->status == 0; ++i)
        c->status = c->gradients
                        ? ((Gradients)c->entry)(d[0], d[1], d[2], d[3], d[4], d[5], d[6], d[7], d[8], d[9], d[10], d[11],
                                                d[12], 1e-6f, 1.f, 0.f, 0, c->workspace, c->bytes, nullptr, c->stream)
                        : ((LogProbs)c->entry)(d[0], d[1], d[2], d[3], d[4], d[5], d[6], 1.f, -100, 0, nullptr, c->stream);
    });
  for (auto& t : threads) t.join();
}
"""


class Call(C.Structure):
    _fields_ = [("entry", C.c_void_p), ("gradients", C.c_int32), ("rounds", C.c_int32), ("status", C.c_int32),
                ("d", C.c_void_p * 13), ("workspace", C.c_void_p), ("bytes", C.c_size_t), ("stream", C.c_void_p)]


def whole(t, mesh):
    return tsl.DTensor([t], mesh, [R], tuple(t.shape), t.dtype)


class Gradients:
    """Gradients of a block norm, with outputs and workspace of their own."""

    def __init__(self, n, parts, dtype, t=9):
        mesh = tsl.DeviceMesh((parts,), ("tp",))
        new = lambda: torch.randn(t, n, device="cuda").to(dtype)  # noqa: E731
        x = tsl.DTensor([new() for _ in range(parts)], mesh, [tsl.Partial() if parts > 1 else R], (t, n), dtype)
        r, dh, dy = (whole(new(), mesh) for _ in range(3))
        post, pre = (whole(torch.randn(n, device="cuda"), mesh) for _ in range(2))
        self.out = (whole(new(), mesh), whole(new(), mesh), whole(torch.zeros(n, device="cuda"), mesh), None,
                    whole(torch.zeros(n, device="cuda"), mesh))
        self.ws = torch.empty(tsl.tp_block_norm_backward_workspace_bytes(x, post, None, pre), dtype=torch.uint8,
                              device="cuda")
        self.call = lambda: tsl.tp_block_norm_backward(dh, dy, x, r, post, None, pre, out=self.out, workspace=self.ws)
        self.operands = (dh, dy, x, r, post, None, pre, None, *self.out)

    def native(self, stream, rounds):
        entry = C.cast(_lib.load().dt_tp_block_norm_backward, C.c_void_p)
        return Call(entry, 1, rounds, 0, pointers(self.operands), self.ws.data_ptr(), self.ws.numel(), stream.cuda_stream)

    def results(self):
        return [d.slots[0] for d in self.out if d is not None]


class Alternatives:
    def __init__(self, v, t=350):
        z = whole(torch.randn(t, v, device="cuda"), tsl.DeviceMesh((1,), ("tp",)))
        self.out = tsl.tp_log_probs(z, top=3)
        self.call = lambda: tsl.tp_log_probs(z, top=3, out=self.out)
        self.operands = (z, None, *self.out)

    def native(self, stream, rounds):
        entry = C.cast(_lib.load().dt_tp_log_probs, C.c_void_p)
        return Call(entry, 0, min(rounds, 300), 0, pointers(self.operands), None, 0, stream.cuda_stream)

    def results(self):
        return [d.slots[0] for d in self.out if d is not None]


def pointers(operands):
    p = [None if d is None else C.addressof(_ref(d)._obj) for d in operands]
    return (C.c_void_p * 13)(*p, *[None] * (13 - len(p)))


BF, FP = torch.bfloat16, torch.float32
SETS = [  # calls of one kernel each, with different needs
    lambda: [Gradients(n, p, BF) for n, p in ((4096, 2), (8192, 6), (5120, 3), (8192, 3))],
    lambda: [Gradients(n, 1, BF) for n in (4096, 4224, 6144)],
    lambda: [Gradients(n, p, FP) for n, p in ((2560, 2), (8192, 2), (4096, 5))],
    lambda: [Alternatives(v) for v in (1200000, 2000000)],
]


def expected(calls):
    want = []
    for c in calls:
        c.call()
        want.append([t.clone() for t in c.results()])
        for t in c.results():
            t.zero_()
    torch.cuda.synchronize()
    return want


def check(calls, want):
    torch.cuda.synchronize()
    for c, w in zip(calls, want):
        assert all(torch.equal(a, b) for a, b in zip(c.results(), w))


@pytest.fixture(scope="module")
def caller(tmp_path_factory):
    at = tmp_path_factory.mktemp("caller")
    (at / "caller.cpp").write_text(CALLER)
    subprocess.run(["g++", "-O1", "-shared", "-fPIC", "-pthread", "-o", str(at / "caller.so"), str(at / "caller.cpp")],
                   check=True)
    return C.CDLL(str(at / "caller.so")).run


@pytest.mark.parametrize("which", range(len(SETS)))
def test_from_many_threads(lib, caller, which):
    calls = SETS[which]()
    want = expected(calls)
    streams = [torch.cuda.Stream() for _ in calls]
    natives = (Call * len(calls))(*[c.native(s, 20000) for c, s in zip(calls, streams)])
    caller(natives, len(calls))
    torch.cuda.synchronize()
    assert [n.status for n in natives] == [0] * len(calls)
    check(calls, want)


@pytest.mark.parametrize("which", range(len(SETS)))
def test_in_one_graph(which):
    calls = SETS[which]()
    want = expected(calls)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for c in calls + calls[::-1]:
            c.call()
    g.replay()
    check(calls, want)
