"""The 8-bit entry points' argument checks, workspace sizing and plans (every check of
test_i8_refusals.py at the C boundary, the sweep over extreme shapes among them) under
AddressSanitizer and UndefinedBehaviorSanitizer, on the CPU."""
import glob
import os
import shutil

import pytest

from tests.test_sanitizers import run_child

pytestmark = pytest.mark.slow


def test_i8_host_code_under_asan_ubsan(tmp_path):
    from moe_experts_amd import build
    if not shutil.which(build.HIPCC) and not os.path.exists(build.HIPCC):
        pytest.skip("hipcc not available")
    rts = sorted(glob.glob("/opt/rocm/llvm/lib/clang/*/lib/linux/libclang_rt.asan-x86_64.so"))
    if not rts:
        pytest.skip("clang's ASan runtime is not installed")
    lib = build.build_sanitized(str(tmp_path / "libq4moe_san.so"))
    out = run_child(["tests/test_i8_refusals.py", "-k", "not binding and not lost"],
                    {"LD_PRELOAD": rts[-1], "Q4MOE_ABI_LIB": lib})
    assert "passed" in out
