"""The 8-bit operators captured in graphs, on several streams, in two host threads and
with the binding's own workspaces: every result equals the eager call bitwise."""
import numpy as np
import pytest
import torch

from moe_experts_amd import datagen
from tests.gpu_util import dev, to_dev
from tests.test_gpu_threads import together

pytestmark = pytest.mark.gpu


class Setup:
    """One call of every operator on buffers of its own (M rows)."""

    def __init__(self, M, K=1040, N=264, seed=1):
        import moe_experts_amd as q4
        r = datagen.rng(seed)
        self.W, self.sw = q4.i8_quantize(to_dev(r.standard_normal((N, K)).astype(np.float32)))
        e = lambda t, *s: torch.empty(s, dtype=t, device=dev())
        self.inputs = {"x": e(torch.float32, M, K), "dY": e(torch.bfloat16, M, N)}
        i = self.inputs
        self.outs = [e(torch.int8, M, K), e(torch.float32, M), e(torch.bfloat16, M, K),
                     e(torch.float16, M, N), e(torch.bfloat16, M, K), e(torch.bfloat16, N, K)]
        o = self.outs
        self.calls = [
            lambda: q4.i8_quantize(i["x"], Q=o[0], scale=o[1]),
            lambda: q4.i8_dequantize(o[0], o[1], X=o[2]),
            lambda: q4.i8_gemm(o[0], o[1], self.W, self.sw, Y=o[3]),
            lambda: q4.i8_gemm_backward(i["dY"], self.W, self.sw, dX=o[4]),
            lambda: q4.i8_gemm_backward_weight(i["dY"], o[0], o[1], dW=o[5]),
        ]
        if M <= 8:
            o.append(e(torch.float32, M, N))
            self.calls.append(lambda: q4.i8_gemv(i["x"], self.W, self.sw, y=o[6]))
        self.refill(seed + 1)

    def refill(self, seed):
        r = datagen.rng(seed)
        for t in self.inputs.values():
            t.copy_(to_dev(r.standard_normal(tuple(t.shape)).astype(np.float32)))

    def run(self):
        for f in self.calls:
            f()

    def results(self):
        torch.cuda.synchronize()
        return [o.clone() for o in self.outs]

    def eager(self):
        for o in self.outs:
            o.fill_(77)
        self.run()
        return self.results()

    def capture(self):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        return g


def equal(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("M,K", [(1, 1040), (5, 1040), (8, 11008), (40, 1040), (300, 1040),
                                 (300, 8208)])
def test_replays_equal_eager(M, K):
    s = Setup(M, K)
    s.run()
    torch.cuda.synchronize()
    g = s.capture()
    for seed in (11, 12, 13, 14):
        s.refill(seed)
        g.replay()
        got = s.results()
        assert equal(got, s.eager())  # eager work between the replays
        assert all(torch.isfinite(t.float()).all() for t in got)


def test_two_graphs_at_once_and_a_larger_call_between():
    """Two graphs replayed on two streams without waiting for one another, after an eager call
    that needs a larger workspace than either: neither sees the other's scratch memory."""
    a, b = Setup(8, 4112, seed=21), Setup(130, 4112, seed=25)
    for s in (a, b):
        s.run()
    torch.cuda.synchronize()
    ga, gb = a.capture(), b.capture()
    Setup(1000, K=8208, N=1024, seed=23).run()
    junk = torch.full((64 << 20,), 7, dtype=torch.uint8, device=dev())  # takes freed memory, if any
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for seed in (31, 32, 33):
        a.refill(seed)
        b.refill(seed + 100)
        torch.cuda.synchronize()
        for _ in range(4):
            with torch.cuda.stream(s1):
                ga.replay()
            with torch.cuda.stream(s2):
                gb.replay()
        got = a.results(), b.results()
        assert equal(got[0], a.eager()) and equal(got[1], b.eager())
    assert bool((junk == 7).all())


def test_streams_do_not_share_workspaces():
    a, b = Setup(5, 4112, seed=41), Setup(130, seed=45)
    want = a.eager(), b.eager()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
    assert equal(a.results(), want[0]) and equal(b.results(), want[1])


@pytest.mark.parametrize("rows", [(5, 8), (130, 130), (300, 8)])
def test_threads_on_the_default_stream(rows):
    sets = [Setup(M, 4112, seed=61 + 10 * i) for i, M in enumerate(rows)]
    want = [s.eager() for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def calls(i):
        def f():
            for _ in range(30):
                sets[i].run()
                if not equal(sets[i].results(), want[i]):
                    wrong.append(rows[i])
        return f

    together(calls(0), calls(1))
    assert not wrong


def test_calls_are_bitwise_repeatable():
    for M, N in ((3, 264), (70, 264), (260, 72), (1100, 4104)):
        s = Setup(M, N=N, seed=51)
        first = s.eager()
        assert all(equal(first, s.eager()) for _ in range(3))
