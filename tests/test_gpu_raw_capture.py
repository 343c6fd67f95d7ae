"""Calls captured by HIP's own stream capture, not through torch's graphs: the
graph's scratch memory is not given to anyone else while the graph lives."""
import ctypes

import pytest
import torch

from tests.gpu_util import dev
from tests.test_gpu_ffn_graphs import Setup, equal

pytestmark = pytest.mark.gpu
RELAXED = 2


def hip():
    """The HIP runtime that the library has loaded."""
    from moe_experts_amd import binding
    lib, p = binding._lib, ctypes.c_void_p
    lib.hipStreamBeginCapture.argtypes = [p, ctypes.c_int]
    lib.hipStreamEndCapture.argtypes = [p, ctypes.POINTER(p)]
    lib.hipGraphInstantiate.argtypes = [ctypes.POINTER(p), p, p, p, ctypes.c_size_t]
    lib.hipGraphLaunch.argtypes = [p, p]
    lib.hipGraphExecDestroy.argtypes = [p]
    lib.hipGraphDestroy.argtypes = [p]
    return lib


@pytest.mark.parametrize("M", [5, 40, 300])
def test_graph_of_a_raw_capture_keeps_its_memory(M):
    h, s = hip(), Setup(M, seed=91)
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        s.run()  # outside the capture first
        torch.cuda.synchronize()
        graph, run = ctypes.c_void_p(), ctypes.c_void_p()
        assert h.hipStreamBeginCapture(stream.cuda_stream, RELAXED) == 0
        s.run()
        assert h.hipStreamEndCapture(stream.cuda_stream, ctypes.byref(graph)) == 0
        assert h.hipGraphInstantiate(ctypes.byref(run), graph, None, None, 0) == 0
        # takes what memory the allocator has free on this stream
        junk = [torch.full((1 << n,), 7, dtype=torch.uint8, device=dev())
                for n in range(9, 27) for _ in range(4)]
        for seed in (92, 93, 94):
            s.refill(seed)
            torch.cuda.synchronize()
            for o in s.outs:
                o.fill_(float("nan"))
            assert h.hipGraphLaunch(run, stream.cuda_stream) == 0
            got = s.results()
            assert equal(got, s.eager())
            assert all(bool((j == 7).all()) for j in junk)
        assert h.hipGraphExecDestroy(run) == 0 and h.hipGraphDestroy(graph) == 0
