"""The 8-bit calls' way to the library, without a GPU: on which device and stream a call is
made, and what the compiler made of their kernels."""
import re

import pytest

import tests.built  # noqa: F401  (binding loads the library)
from moe_experts_amd import binding
from tests.test_binding_workspaces import FakeTorch
from tests.test_ffn_registers import OBJDUMP, descriptions, said_of_objects, unwaited

#: kernels of the matrix cores, and how many variants of each are built
KERNELS = {"i8_gemm_kernel": 18, "i8_gradient_kernel": 4, "i8_few_rows_kernel": 7,
           "i8_few_gradient_kernel": 6}


@pytest.mark.parametrize("index", [0, 3])
def test_calls_without_a_workspace_run_on_their_own_device(index, monkeypatch):
    fake = FakeTorch()
    monkeypatch.setattr(binding, "torch", fake)
    monkeypatch.setattr(binding, "_raw_stream", lambda i: 1000 + i)
    seen = []
    binding._call(lambda *a: seen.append((fake.current, a)) or 0, index, 7, 8)
    assert seen == [(index, (7, 8, 1000 + index))] and fake.current == 0
    with pytest.raises(binding.Q4Error) as e:
        binding._call(lambda *a: -2, index)
    assert e.value.status == -2 and fake.current == 0


def test_accumulators_are_in_vector_registers(tmp_path):
    found = descriptions(tmp_path)
    for kernel, count in KERNELS.items():
        mine = [agprs for name, agprs in found if kernel in name]
        assert mine == [0] * count, kernel


def bodies(tmp_path, kernel):
    for text in said_of_objects(tmp_path, OBJDUMP, "-d"):
        yield from re.findall(r"^[0-9a-f]+ <(\S*%s\S*)>:\n(.*?)(?=^[0-9a-f]+ <|\Z)" % kernel, text,
                              re.S | re.M)


@pytest.mark.parametrize("kernel", KERNELS)
def test_lds_is_waited_for_at_every_barrier(kernel, tmp_path):
    """A wave's reads of LDS are done before each barrier that hands a stage over."""
    found = list(bodies(tmp_path, kernel))
    assert len(found) == KERNELS[kernel]
    for name, body in found:
        barriers, bad = unwaited(body.splitlines())
        assert barriers >= 1 and not bad, (name, bad[:4])


@pytest.mark.parametrize("kernel", ["i8_gemm_kernel", "i8_gradient_kernel"])
def test_copies_stay_in_flight_over_reads_of_other_stages(kernel, tmp_path):
    """Between the loop's barriers no wait is for copies but the one that stands right before a
    barrier: with all stages in one array the compiler waits for all of them before every read."""
    for name, body in bodies(tmp_path, kernel):
        lines = [l.split("//")[0].strip() for l in body.splitlines()]
        barriers = [i for i, l in enumerate(lines) if l.startswith("s_barrier")]
        waits = [i for i in range(barriers[0], barriers[2])  # the first two steps of the loop
                 if lines[i].startswith("s_waitcnt") and "vmcnt" in lines[i]]
        assert len(waits) == 2, (name, [lines[i] for i in waits])
        for i in waits:
            assert any(l.startswith("s_barrier") for l in lines[i + 1:i + 4]), (name, lines[i])
