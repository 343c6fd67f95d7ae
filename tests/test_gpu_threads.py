"""Host threads that call the operators at the same time, on one stream: every
result equals the one computed alone, bitwise."""
import threading

import pytest
import torch

from moe_experts_amd import datagen
from tests.gpu_util import dev, to_dev
from tests.test_gpu_ffn_graphs import Setup

pytestmark = pytest.mark.gpu


def together(*work):
    """Runs each function in a thread of its own, started at the same time."""
    start, errors = threading.Barrier(len(work)), []

    def go(f):
        try:
            start.wait(60)
            f()
        except BaseException as e:  # noqa: BLE001 - reported below
            errors.append(e)

    threads = [threading.Thread(target=go, args=(f,)) for f in work]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not errors, errors


@pytest.mark.parametrize("rows", [(1, 5), (40, 40), (300, 8), (300, 300)])
def test_dense_feed_forward_on_the_default_stream(rows):
    sets = [Setup(M, seed=61 + 10 * i) for i, M in enumerate(rows)]
    for i, s in enumerate(sets):
        s.refill(71 + i)
    want = [s.eager() for s in sets]
    torch.cuda.synchronize()
    wrong = []

    def calls(i):
        def f():
            for _ in range(30):
                sets[i].run()
                got = sets[i].results()
                if not all(torch.equal(a, b) for a, b in zip(got, want[i])):
                    wrong.append(rows[i])
        return f

    together(calls(0), calls(1))
    assert not wrong


def test_decode_products_on_the_default_stream():
    """The same of an entry point that takes its workspace by device: K split, so that partial
    sums pass through it."""
    from moe_experts_amd import q4_0_gemv
    K, N = 4096, 512
    B = to_dev(datagen.q4_0_random(81, K, N))
    xs = [to_dev(datagen.activations(82 + i, 4, K)) for i in range(2)]
    ys = [torch.empty((4, N), dtype=torch.float32, device=dev()) for _ in xs]
    want = [q4_0_gemv(x, B, N) for x in xs]
    torch.cuda.synchronize()
    wrong = []

    def calls(i):
        def f():
            for _ in range(100):
                q4_0_gemv(xs[i], B, N, y=ys[i])
                torch.cuda.synchronize()
                if not torch.equal(ys[i], want[i]):
                    wrong.append(i)
        return f

    together(calls(0), calls(1))
    assert not wrong
