"""The dense feed-forward operators captured in graphs, on several streams and
with the binding's own workspaces: every result equals the eager call bitwise."""
import numpy as np
import pytest
import torch

from moe_experts_amd import datagen
from tests.gpu_util import dev, to_dev

pytestmark = pytest.mark.gpu


class Setup:
    """One call of every operator on buffers of its own (M rows)."""

    def __init__(self, M, K=512, N=256, R=16, L=3, seed=1):
        import moe_experts_amd as q4
        self.M, self.K, self.N, self.L = M, K, N, L
        r = datagen.rng(seed)
        f16 = lambda *s: to_dev(r.standard_normal(s).astype(np.float16))
        self.Wg, self.Wu = (to_dev(datagen.q4_0_random(seed + i, K, N)) for i in (1, 2))
        self.A, self.Bl = f16(L, R, K), f16(L, N, R)
        self.scale = to_dev(r.uniform(0.5, 2, L).astype(np.float32))
        self.G, self.U = f16(M, N), f16(M, N)
        self.inputs = {"X": f16(M, K), "dY": f16(M, N).bfloat16(),
                       "ids": torch.zeros(M, dtype=torch.int32, device=dev())}
        e = lambda n, t: torch.empty((M, n), dtype=t, device=dev())
        i = self.inputs
        self.outs = [e(N, torch.float16), e(K, torch.bfloat16), e(K, torch.bfloat16),
                     e(N, torch.float16)]
        o = self.outs
        self.calls = [
            lambda: q4.q4_0_glu_gemm(i["X"], self.Wg, self.Wu, N, H=o[0]),
            lambda: q4.q4_0_glu_backward(i["dY"], self.G, self.U, self.Wg, self.Wu, K, dX=o[1]),
            lambda: q4.q4_0_gemm_backward(i["dY"], self.Wg, K, dX=o[2]),
            lambda: q4.q4_0_gemm_lora(i["X"], self.Wg, N, self.A, self.Bl, i["ids"], self.scale,
                                      Y=o[3]),
        ]
        if M <= 8:
            i["x"] = i["X"].float()
            o += [e(N, torch.float32), e(N, torch.float32)]
            self.calls += [
                lambda: q4.q4_0_glu(i["x"], self.Wg, self.Wu, N, h=o[4]),
                lambda: q4.q4_0_gemv_lora(i["x"], self.Wg, N, self.A, self.Bl, i["ids"],
                                          self.scale, y=o[5]),
            ]

    def refill(self, seed):
        r = datagen.rng(seed)
        for k, t in self.inputs.items():
            if k == "ids":
                t.copy_(to_dev(r.integers(-1, self.L, self.M).astype(np.int32)))
            else:
                t.copy_(to_dev(r.standard_normal(tuple(t.shape)).astype(np.float32)))

    def run(self):
        for f in self.calls:
            f()

    def results(self):
        torch.cuda.synchronize()
        return [o.clone() for o in self.outs]

    def eager(self):
        for o in self.outs:
            o.fill_(float("nan"))
        self.run()
        return self.results()

    def capture(self):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            self.run()
        return g


def equal(a, b):
    return all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("M", [1, 5, 40, 300])
def test_replays_equal_eager(M):
    s = Setup(M)
    s.run()
    torch.cuda.synchronize()
    g = s.capture()
    for seed in (11, 12, 13, 14):
        s.refill(seed)
        g.replay()
        got = s.results()
        assert equal(got, s.eager())   # eager work between the replays
        assert all(torch.isfinite(t.float()).all() for t in got)


def test_two_graphs_at_once_and_a_larger_call_between():
    """Two graphs replayed on two streams without waiting for one another, after an eager call
    that needs a larger workspace than either: neither sees the other's scratch memory."""
    a, b = Setup(40, seed=21), Setup(40, seed=22)
    for s in (a, b):
        s.run()
    torch.cuda.synchronize()
    ga, gb = a.capture(), b.capture()
    Setup(300, K=2048, N=1024, seed=23).run()
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
    a, b = Setup(5, seed=41), Setup(40, seed=42)
    want = a.eager(), b.eager()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        with torch.cuda.stream(s1):
            a.run()
        with torch.cuda.stream(s2):
            b.run()
    assert equal(a.results(), want[0]) and equal(b.results(), want[1])


def test_calls_are_bitwise_repeatable():
    for M in (3, 70, 260):
        s = Setup(M, K=1024, N=320, seed=51)
        s.refill(52)
        first = s.eager()
        assert all(equal(first, s.eager()) for _ in range(3))
