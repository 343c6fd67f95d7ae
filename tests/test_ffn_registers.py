"""What the compiler made of the dense feed-forward's matrix-core kernels, read from
the built library, without a GPU.

The matrix-core kernels of the dense feed-forward keep their accumulators in
ordinary vector registers. With accumulation registers the compiler (AMD clang
22.0.0, ROCm 7.2.0) gave one LDS store of lora_shrink_tile_kernel a wrong offset:
row 1 of a tile went to row 0. And every wave of a GEMM tile waits for its own LDS
reads and writes before each barrier that hands LDS over."""
import os
import re
import subprocess

import numpy as np
import pytest

import tests.built  # noqa: F401
from tests import ffn_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_experts_amd", "libq4moe.so")
READELF, OBJDUMP = ("/opt/rocm/llvm/bin/llvm-" + t for t in ("readelf", "objdump"))
KERNELS = {"ffn_gemm_kernel": 9, "strip_kernel": 5, "lora_shrink_tile_kernel": 1}


def said_of_objects(tmp_path, *command):
    """What a tool prints of each gfx950 object in the library."""
    if not os.path.exists(command[0]):
        pytest.skip(f"{command[0]} is not installed")
    data = open(LIB, "rb").read()
    starts = [m.start() for m in re.finditer(b"\x7fELF\x02\x01\x01\x40", data)]  # AMDGPU's
    for a, b in zip(starts, starts[1:] + [len(data)]):
        obj = tmp_path / "object.elf"
        obj.write_bytes(data[a:b])
        yield subprocess.run([*command, str(obj)], capture_output=True, text=True).stdout


def descriptions(tmp_path):
    """(kernel, accumulation registers) of every gfx950 kernel in the library."""
    found = []
    for notes in said_of_objects(tmp_path, READELF, "--notes"):
        for part in notes.split("- .agpr_count:")[1:]:
            name = re.search(r"\.name:\s+(\S+)", part)
            found.append((name.group(1), int(part.split()[0])))
    return found


def test_accumulators_are_in_vector_registers(tmp_path):
    found = descriptions(tmp_path)
    for kernel, count in KERNELS.items():
        mine = [agprs for name, agprs in found if kernel in name]
        assert len(mine) == count, kernel
        assert mine == [0] * count, kernel


@pytest.mark.parametrize("source", ["ffn_gemm.hip", "ffn_rows.hip", "ffn_strip.hip"])
def test_every_source_of_them_is_built_so(source):
    from moe_experts_amd import build
    assert "-amdgpu-mfma-vgpr-form" in build.EXTRA.get(source, [])


@pytest.mark.parametrize("M,K,N,R,L", [(65, 256, 192, 24, 7), (64 + 64, 64, 64, 8, 3)])
def test_mixed_up_rows_of_a_tile_are_seen(M, K, N, R, L):
    """What that fault did, planted in the reference: row 0 of each tile of 64 with the narrow
    product of row 1 is far outside the bound that the results are held to."""
    from tests.test_gpu_ffn import adapters, row_ids, weights
    from moe_experts_amd import datagen
    x, B = datagen.to_f16(datagen.activations(55, M, K)), weights(56, K, N)
    A, Bl, scale = adapters(57, L, R, K, N)
    ids = row_ids("one", M, L)
    right = ref.gemm_lora(x, B, A, Bl, ids, scale)
    ref.check(right[0], right)
    y, _ = ref.product16(x, B)
    own, _ = ref.adapters(x, A, Bl, ids, scale, True)
    own[::64][:M // 64] = own[1::64][:M // 64]
    with pytest.raises(AssertionError, match="of the bound"):
        ref.check(y + own, right)
    assert np.abs(own).max() > 0


def unwaited(lines):
    """LDS accesses between the last full LDS wait (or the block's start) and a barrier."""
    since, bad, barriers = [], [], 0
    for line in lines:
        t = line.split("//")[0].strip()
        if t.startswith("ds_"):
            since.append(t)
        elif t == "s_endpgm" or t.startswith("s_waitcnt") and "lgkmcnt(0)" in t:
            since = []
        elif t.startswith("s_barrier"):
            barriers += 1
            bad += since
            since = []
    return barriers, bad


def test_lds_is_waited_for_at_every_barrier(tmp_path):
    kernels = 0
    for text in said_of_objects(tmp_path, OBJDUMP, "-d"):
        for name, body in re.findall(r"^[0-9a-f]+ <(\S*ffn_gemm_kernel\S*)>:\n(.*?)(?=^[0-9a-f]+ <|\Z)",
                                     text, re.S | re.M):
            barriers, bad = unwaited(body.splitlines())
            kernels += 1
            assert barriers >= 4 and not bad, (name, bad[:4])
    assert kernels == KERNELS["ffn_gemm_kernel"]


def test_an_access_behind_the_wait_is_seen():
    right = ["ds_write_b128 v1, v[2:5]", "s_waitcnt lgkmcnt(0)", "v_mov_b32 v0, 0", "s_barrier"]
    assert unwaited(right) == (1, [])
    wrong = [right[1], right[0], right[3]]
    assert unwaited(wrong) == (1, [right[0]])
