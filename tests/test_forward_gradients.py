"""Tangents of forward-mode differentiation, which the calls without a gradient of their own would
quietly drop: refused, without a GPU. (CPU tensors; the check of the device and the library's calls
are stand-ins.)"""
import pytest
import torch
from torch.autograd import forward_ad

import tests.built  # noqa: F401  (binding loads the library)
import moe_experts_amd as q4
from moe_experts_amd import binding

M, N, K = 3, 64, 64
MAT = K * (N // 32) * binding.BLOCK_BYTES


@pytest.fixture
def ran(monkeypatch):
    calls = []
    monkeypatch.setattr(binding, "_dev", lambda t, *a: t.data_ptr())
    monkeypatch.setattr(binding, "_run", lambda *a: calls.append(a))
    monkeypatch.setattr(binding, "_call", lambda *a: calls.append(a))
    return calls


def cases():
    x, x16 = torch.zeros(M, K), torch.zeros(M, K, dtype=torch.float16)
    X, W = torch.zeros(M, K, dtype=torch.int8), torch.zeros(N, K, dtype=torch.int8)
    sx, sw = torch.zeros(M), torch.zeros(N)
    dY = torch.zeros(M, N, dtype=torch.bfloat16)
    B = torch.zeros(MAT, dtype=torch.uint8)
    yield (x,), lambda x: q4.i8_quantize(x)
    yield (sx,), lambda s: q4.i8_dequantize(X, s)
    yield (x, sw), lambda x, s: q4.i8_gemv(x, W, s)
    yield (sx, sw), lambda a, b: q4.i8_gemm(X, a, W, b)
    yield (dY, sw), lambda d, s: q4.i8_gemm_backward(d, W, s)
    yield (dY, sx), lambda d, s: q4.i8_gemm_backward_weight(d, X, s)
    yield (x,), lambda x: q4.q4_0_glu(x, B, B, N)
    yield (x16,), lambda x: q4.q4_0_glu_gemm(x, B, B, N)
    yield (dY,), lambda d: q4.q4_0_gemm_backward(d, B, K)


@pytest.mark.parametrize("at", range(9))
def test_a_tangent_that_would_be_lost_is_refused(at, ran):
    inputs, call = list(cases())[at]
    for i, t in enumerate(inputs):
        with forward_ad.dual_level():
            call(*inputs)  # a level alone is none of an input's
            assert ran.pop()
            dual = [forward_ad.make_dual(u, torch.ones_like(u)) if j == i else u
                    for j, u in enumerate(inputs)]
            with pytest.raises(ValueError, match="tangent"):
                call(*dual)
            with torch.no_grad(), pytest.raises(ValueError, match="tangent"):
                call(*dual)  # no_grad leaves tangents be
            assert not ran
        call(*inputs)
        assert ran.pop()


def test_a_function_of_its_own_may_call(ran):
    """In the forward of a torch.autograd.Function, which brings its own jvp."""

    class Rows(torch.autograd.Function):
        @staticmethod
        def forward(ctx, x):
            return q4.i8_quantize(x)[1]

        @staticmethod
        def jvp(ctx, t):
            return t.sum(1)

    x = torch.zeros(M, K)
    with forward_ad.dual_level():
        y = Rows.apply(forward_ad.make_dual(x, torch.ones_like(x)))
        assert ran.pop()
        assert torch.equal(forward_ad.unpack_dual(y).tangent, torch.full((M,), float(K)))
