"""The matrix-core kernels of the dense feed-forward keep their accumulators in
ordinary vector registers. With accumulation registers the compiler (AMD clang
22.0.0, ROCm 7.2.0) gave one LDS store of lora_shrink_tile_kernel a wrong offset:
row 1 of a tile went to row 0. Read here from the built library's own kernel
descriptions, without a GPU."""
import os
import re
import subprocess

import numpy as np
import pytest

from tests import ffn_ref as ref

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
LIB = os.path.join(ROOT, "moe_experts_amd", "libq4moe.so")
READELF = "/opt/rocm/llvm/bin/llvm-readelf"
KERNELS = {"ffn_gemm_kernel": 9, "strip_kernel": 5, "lora_shrink_tile_kernel": 1}


def descriptions(lib, tmp_path):
    """(kernel, accumulation registers) of every gfx950 kernel in a library."""
    data = open(lib, "rb").read()
    starts = [m.start() for m in re.finditer(b"\x7fELF\x02\x01\x01\x40", data)]  # AMDGPU's
    found = []
    for a, b in zip(starts, starts[1:] + [len(data)]):
        obj = tmp_path / "object.elf"
        obj.write_bytes(data[a:b])
        notes = subprocess.run([READELF, "--notes", str(obj)], capture_output=True,
                               text=True).stdout
        for part in notes.split("- .agpr_count:")[1:]:
            name = re.search(r"\.name:\s+(\S+)", part)
            found.append((name.group(1), int(part.split()[0])))
    return found


def test_accumulators_are_in_vector_registers(tmp_path):
    if not os.path.exists(READELF):
        pytest.skip("llvm-readelf is not installed")
    if not os.path.exists(LIB):
        from moe_experts_amd import build
        build.build()
    found = descriptions(LIB, tmp_path)
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
