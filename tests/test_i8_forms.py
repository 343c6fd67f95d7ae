"""The shapes that the 8-bit operators' GPU tests check by value reach every compiled form of the
row kernels, by i8_rows_plan (CPU)."""
import ctypes

import pytest

import tests.built  # noqa: F401
from moe_experts_amd import i8_rows_plan
from moe_experts_amd.binding import LIB_PATH, Q4Error
from tests import test_gpu_i8 as gpu
from tests import test_gpu_i8_forms as forms
from tests.test_ffn_registers import descriptions

EINVAL, ESHAPE, EBIG = -1, -2, -6


def built(tmp_path, kernel):
    """The template arguments of a kernel's variants in the built library, as they are mangled."""
    return [n.split(kernel + "I")[1].split("EEEv")[0].replace("Ei", "").split("EL")
            for n, _ in descriptions(tmp_path) if kernel + "I" in n]


def numbers(parts):
    return tuple(int(p.lstrip("Lib")) for p in parts)


def test_every_form_that_quantizes(tmp_path):
    want = {numbers(v) for v in built(tmp_path, "i8_quantize_kernel")}
    shapes = [(M, K) for M, K in gpu.ROW_SHAPES] + [(forms.MANY, K) for K in forms.LONG]
    got = {i8_rows_plan("i8_quantize", M, 8, K) for M, K in shapes}
    # of every type: type, threads, pieces, whether there is a second pass
    got = {(t, *p[:2], p[2] - 1) for t in range(3) for p in got if p[1]}
    assert got == want and len(want) == 27


def test_every_form_of_the_inputs_left_operand(tmp_path):
    want = {numbers(v) for v in built(tmp_path, "i8_gradient_rows_kernel")}
    got = {i8_rows_plan("i8_gemm_backward", *s) for s in forms.ROWS}
    assert {(*p[:2], p[2] - 1) for p in got} == want and len(want) == 7


def test_every_form_of_the_weights_left_operand(tmp_path):
    want = {numbers(v) for v in built(tmp_path, "i8_gradient_columns_once_kernel")}
    got = {i8_rows_plan("i8_gemm_backward_weight", *s) for s in forms.COLUMNS}
    assert {(p[0], p[1] // 2) for p in got if p[2] == 1} == want and len(want) == 6
    assert any(p[2] == 2 for p in got)


def test_odd_lengths_of_every_transposition():
    """Tokens that end inside a lane's pair of rows."""
    got = [(i8_rows_plan("i8_gemm_backward_weight", M, N, K), M % 2) for M, N, K in forms.COLUMNS]
    assert {p for p, odd in got if odd} == {p for p, _ in got}


def test_broken_values_and_far_sizes_reach_both_transpositions():
    for form, *s in forms.BROKEN:
        assert i8_rows_plan(form, *s)[0] > 0
    assert {i8_rows_plan(f, *s)[2] for f, *s in forms.BROKEN if f.endswith("weight")} == {1, 2}


def test_a_gradient_of_little_work_has_no_row_kernel():
    assert i8_rows_plan("i8_gemm_backward", 8, 4096, 64) == (0, 0, 0)
    assert i8_rows_plan("i8_gemm_backward_weight", 64, 24, 64) == (0, 0, 0)


def test_refusals():
    with pytest.raises(ValueError, match="form"):
        i8_rows_plan("i8_gemm", 1, 8, 16)
    for args, status in ((("i8_quantize", 0, 8, 16), EINVAL), (("i8_quantize", 1, 8, 0), EINVAL),
                         (("i8_quantize", 1 << 20, 8, 1 << 20), EBIG),
                         (("i8_quantize", 1 << 32, 8, 16), EBIG),
                         (("i8_gemm_backward", 1, 8, 8), ESHAPE),
                         (("i8_gemm_backward_weight", 1, 4, 16), ESHAPE),
                         (("i8_gemm_backward_weight", 1 << 27, 8, 16), EBIG)):
        with pytest.raises(Q4Error) as e:
            i8_rows_plan(*args)
        assert e.value.status == status, args
    lib, i = ctypes.CDLL(LIB_PATH), ctypes.c_int
    out = [ctypes.byref(i(7)) for _ in range(3)]
    for form in (-1, 3):
        assert lib.i8_rows_plan(form, 65, 64, 64, *out) == EINVAL
    for at in range(3):
        assert lib.i8_rows_plan(0, 65, 64, 64, *out[:at], None, *out[at + 1:]) == EINVAL
