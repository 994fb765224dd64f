"""Decode-step entry points without a GPU: null handles and sizes are refused on the host."""
import pytest

from consumer_movement_gemm_gb300 import build as tovl_build
from consumer_movement_gemm_gb300 import tovl


@pytest.fixture(scope="module")
def lib():
    tovl_build.build()
    return tovl.load()


def test_null_handles_are_refused(lib):
    for name in ("tovl_add_rmsnorm", "tovl_route_topk", "tovl_moe_decode", "tovl_moe_decode_q4", "tovl_matvec_q4",
                 "tovl_quantize_q4"):
        args = [0 if a is not tovl._P else None for a in tovl.SIGNATURES[name][0]]
        assert getattr(lib, name)(*args) == tovl.TOVL_ERR_INVALID, name
    assert lib.tovl_moe_decode_workspace(None, 1, 1, 8, 8) == -1
    assert lib.tovl_matvec_q4_workspace(None, 1, 8) == -1


def test_the_binding_and_the_header_agree_on_types():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(tovl.__file__))), "include", "tovl.h")).read()
    for name in ("TOVL_BF16", "TOVL_F32", "TOVL_E4M3"):
        assert int(re.search(name + r" = (\d+)", text).group(1)) == getattr(tovl, name)


def test_importing_the_binding_does_not_import_torch():
    import subprocess
    import sys
    code = "import sys; import consumer_movement_gemm_gb300; sys.exit(1 if 'torch' in sys.modules else 0)"
    assert subprocess.run([sys.executable, "-c", code]).returncode == 0
