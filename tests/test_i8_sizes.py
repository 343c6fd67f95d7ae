"""Sizes below the C ints' range, which would lose their upper bits as those above it would."""
import pytest

import tests.built  # noqa: F401  (binding loads the library)
from moe_experts_amd import binding

EINVAL = -1
#: name: (M, N, K)
CALLS = ("i8_gemv", "i8_gemm", "i8_gemm_backward", "i8_gemm_backward_weight")
LOW = -(1 << 32) + 64  # its lower 32 bits are 64


@pytest.mark.parametrize("at", range(3))
@pytest.mark.parametrize("name", CALLS)
def test_sizes_below_c_ints(name, at):
    sizes = [64, 64, 64]
    sizes[at] = LOW
    with pytest.raises(binding.Q4Error) as e:
        getattr(binding, name + "_workspace_bytes")(*sizes)
    assert e.value.status == EINVAL
    if name in binding.I8_FORMS:
        with pytest.raises(binding.Q4Error) as e:
            binding.i8_gemm_plan(name, *sizes)
        assert e.value.status == EINVAL


def test_the_lowest_c_int_is_the_librarys_to_refuse():
    assert binding.i8_gemm_workspace_bytes(-(1 << 31), 64, 64) == 0
    with pytest.raises(binding.Q4Error) as e:
        binding.i8_gemm_plan("i8_gemm", -(1 << 31), 64, 64)
    assert e.value.status == EINVAL
