"""What the host hands to the kernels of the paged attention step (csrc/paged_api.cu, its launches replaced by ones that keep
their parameters), at the ends of what the header allows."""
import ctypes
import subprocess

import pytest

from consumer_movement_gemm_gb300 import build as tovl_build
from consumer_movement_gemm_gb300 import tovl
from tests.test_paged_abi import ATTN, INVALID, OK, P, ROPE, call


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("limits")
    src = at / "limits.cu"
    src.write_text('#include "paged_api.cu"\n'
                   "static int launches, together;\n"
                   "static AttnParams last;\n"
                   "namespace tovl {\n"
                   "cudaError_t launch_page_plan(const PagePlanParams&, int, cudaStream_t, bool) { ++launches; return cudaSuccess; }\n"
                   "cudaError_t launch_rope_append(const RopeParams&, bool, int, cudaStream_t, bool) { ++launches; return cudaSuccess; }\n"
                   "cudaError_t launch_attn_decode(const AttnParams& p, bool, int, cudaStream_t, bool) { ++launches; last = p; return cudaSuccess; }\n"
                   "AttnShape attn_decode_shape(int, bool, int, bool) { return {16, 128, 8, 8, 1040}; }\n"
                   "int attn_decode_together(const AttnShape&, int, int, bool) { return together; }\n"
                   "bool attn_decode_pairs(int, bool, int) { return false; }\n"
                   "long long attn_decode_workspace(int, int, int, int) { return 4096; }\n"
                   "}\n"
                   "static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,\n"
                   "                       const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill)\n"
                   "{\n"
                   "    return CUDA_SUCCESS;\n"
                   "}\n"
                   "TOVL_API void* make() { auto* h = new tovl_ctx(); h->num_sms = 152; h->encode = encode; return h; }\n"
                   "TOVL_API int count() { return launches; }\n"
                   "TOVL_API void side_by_side(int n) { together = n; }\n"
                   "TOVL_API unsigned most_tiles() { return last.most_tiles; }\n")
    so = at / "limits.so"
    subprocess.run([tovl_build._nvcc(), *tovl_build._flags(), "-shared", "-cudart", "shared", "-o", str(so), str(src)], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(str(so))
    for n in ("tovl_rope_append", "tovl_attn_decode", "tovl_attn_decode_workspace"):
        getattr(lib, n).argtypes, getattr(lib, n).restype = tovl.SIGNATURES[n]
    lib.make.restype = ctypes.c_void_p
    lib.most_tiles.restype = ctypes.c_uint
    return lib


@pytest.mark.parametrize("heads,Hq,together", [(1, 1, 1), (1, 8, 1), (2, 2, 2), (1, 9, 1), (2, 4, 1), (8, 8, 4), (3, 120, 1)])
def test_a_call_of_more_tiles_than_ints_count_is_over_the_limit(lib, heads, Hq, together):
    """The kernel's sums of tiles stop at 2^31 - 1, so that number has to be over the limit, and what is not has to fit."""
    lib.side_by_side(together)
    wide = heads * 64
    assert call(lib, "tovl_attn_decode", ATTN, Hq=Hq, ldq=Hq * 64, ldo=Hq * 64,
                cache=dict(heads=heads, slot_stride=wide, page_stride=16 * wide)) == (OK, 1)
    groups = heads * -(-Hq // heads // 8) // together
    assert lib.most_tiles() < 2 ** 31 - 1
    assert lib.most_tiles() * groups < 2 ** 31 - 1 <= (lib.most_tiles() + 1) * groups


def test_angles_are_looked_at_where_something_is_rotated(lib):
    assert call(lib, "tovl_rope_append", ROPE, cos_sin=P + 4) == (INVALID, 0)
    for table in (P + 4, None):
        assert call(lib, "tovl_rope_append", ROPE, rot=0, cos_sin=table) == (OK, 1)
