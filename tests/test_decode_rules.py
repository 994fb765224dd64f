"""Which form of a decode-step operator a call takes, without a GPU: the rules of csrc/ops.cuh are host code."""
import ctypes
import subprocess

import pytest

from consumer_movement_gemm_gb300 import build as tovl_build


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    at = tmp_path_factory.mktemp("rules")
    src = at / "rules.cu"
    src.write_text('#include "ops.cuh"\n'
                   'extern "C" __attribute__((visibility("default"))) int direct_moe(int T, int k, int E, int H, int I, int group)\n'
                   "{ return tovl::use_direct_moe(T, k, E, H, I, group); }\n")
    lib = at / "rules.so"
    subprocess.run([tovl_build._nvcc(), *tovl_build._flags(), "-shared", "-cudart", "shared", "-o", str(lib), str(src)], check=True,
                   capture_output=True)
    return ctypes.CDLL(str(lib))


# (T, k, E, H, I), the small form's time and the rings', us, one GB300, calls in a row over three sets of inputs
BF16 = [((1, 2, 8, 4096, 2048), 23.7, 30.7), ((2, 8, 64, 1024, 512), 18.0, 21.6), ((4, 4, 32, 2048, 1024), 40.6, 34.8),
        ((8, 4, 32, 1024, 1024), 39.0, 32.6), ((8, 16, 128, 512, 256), 35.2, 25.8), ((8, 8, 64, 1024, 512), 41.4, 34.3),
        ((9, 8, 64, 512, 256), 25.8, 21.2), ((16, 2, 16, 512, 256), 11.7, 17.0), ((16, 8, 64, 512, 256), 31.1, 22.3),
        ((20, 4, 32, 512, 256), 22.0, 17.9), ((20, 4, 32, 256, 128), 11.4, 16.3), ((32, 4, 32, 512, 256), 23.6, 18.5),
        ((33, 2, 16, 512, 256), 14.9, 17.2), ((48, 8, 64, 256, 128), 24.5, 19.7), ((64, 2, 4, 1024, 512), 17.7, 28.5),
        ((64, 2, 8, 1024, 512), 28.6, 23.0), ((64, 8, 64, 256, 128), 27.2, 21.1), ((64, 1, 32, 512, 256), 20.7, 17.0)]
Q4 = [((1, 2, 8, 4096, 2048), 15.8, 20.0), ((1, 4, 8, 4096, 4096), 47.2, 34.5), ((8, 4, 32, 512, 256), 9.5, 17.5),
      ((8, 8, 64, 1024, 512), 29.7, 25.6), ((8, 16, 128, 512, 256), 27.6, 21.2), ((20, 8, 64, 256, 128), 15.8, 18.7),
      ((32, 2, 8, 1024, 512), 15.8, 20.4), ((48, 8, 64, 256, 128), 23.9, 21.4), ((64, 4, 32, 256, 128), 16.7, 20.3),
      ((64, 8, 64, 256, 128), 28.9, 22.2)]


@pytest.mark.parametrize("shape,direct,rings,group", [(*c, 0) for c in BF16] + [(*c, 128) for c in Q4])
def test_expert_layers_take_the_faster_form(rules, shape, direct, rings, group):
    """Every measured size whose two forms differ by a tenth."""
    assert max(direct, rings) > 1.1 * min(direct, rings)
    T, k, E, H, I = shape
    assert bool(rules.direct_moe(T, k, E, H, I, group)) == (direct < rings)
