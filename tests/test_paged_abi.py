"""The paged attention step's entry points without a GPU: the host's argument checks (csrc/paged_api.cu, its launches
replaced by ones that count) refuse what the kernels do not take, and nothing else."""
import ctypes
import subprocess

import pytest

from consumer_movement_gemm_gb300 import build as tovl_build
from consumer_movement_gemm_gb300 import tovl

OK, INVALID, UNSUPPORTED = tovl.TOVL_OK, tovl.TOVL_ERR_INVALID, tovl.TOVL_ERR_UNSUPPORTED
NAMES = ("tovl_page_plan", "tovl_rope_append", "tovl_attn_decode")
BIG = 1 << 20


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    at = tmp_path_factory.mktemp("paged")
    src = at / "paged.cu"
    src.write_text('#include "paged_api.cu"\n'
                   "static int launches;\n"
                   "namespace tovl {\n"
                   "cudaError_t launch_page_plan(const PagePlanParams&, int, cudaStream_t, bool) { ++launches; return cudaSuccess; }\n"
                   "cudaError_t launch_rope_append(const RopeParams&, bool, int, cudaStream_t, bool) { ++launches; return cudaSuccess; }\n"
                   "cudaError_t launch_attn_decode(const AttnParams&, bool, int, cudaStream_t, bool) { ++launches; return cudaSuccess; }\n"
                   "AttnShape attn_decode_shape(int, bool, int, bool) { return {16, 128, 8, 8, 1040}; }\n"
                   "int attn_decode_together(const AttnShape&, int, int, bool) { return 1; }\n"
                   "bool attn_decode_pairs(int, bool, int) { return false; }\n"
                   "long long attn_decode_workspace(int, int, int, int) { return 4096; }\n"
                   "}\n"
                   "static long long maps[16];      // of the last map: dims, strides, box, how many\n"
                   "static CUresult encode(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t* dims, const cuuint64_t* strides,\n"
                   "                       const cuuint32_t* box, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,\n"
                   "                       CUtensorMapFloatOOBfill)\n"
                   "{\n"
                   "    for (int i = 0; i < 4; ++i) maps[i] = dims[i], maps[4 + i] = i < 3 ? strides[i] : 0, maps[8 + i] = box[i];\n"
                   "    ++maps[12];\n"
                   "    return CUDA_SUCCESS;\n"
                   "}\n"
                   'TOVL_API void* make() { auto* h = new tovl_ctx(); h->num_sms = 152; h->encode = encode; maps[12] = 0; return h; }\n'
                   'TOVL_API const long long* last_map() { return maps; }\n'
                   'TOVL_API int count() { return launches; }\n'
                   'TOVL_API int size_of_args(int i) { return i == 0 ? sizeof(tovl_page_plan_args) : i == 1 ? sizeof(tovl_rope_append_args) : sizeof(tovl_attn_decode_args); }\n'
                   'TOVL_API int divide(unsigned x, unsigned d) { return FastDiv(d).div(x); }\n')
    so = at / "paged.so"
    subprocess.run([tovl_build._nvcc(), *tovl_build._flags(), "-shared", "-cudart", "shared", "-o", str(so), str(src)], check=True,
                   capture_output=True)
    lib = ctypes.CDLL(str(so))
    for n in NAMES + ("tovl_attn_decode_workspace",):
        getattr(lib, n).argtypes, getattr(lib, n).restype = tovl.SIGNATURES[n]
    lib.make.restype = ctypes.c_void_p
    lib.last_map.restype = ctypes.POINTER(ctypes.c_longlong)
    return lib


# addresses that are never followed
P = 1 << 16


def cache(**change):
    f = dict(k=P, v=P, k_scale=None, v_scale=None, type=tovl.TOVL_BF16, pages=9, page=16, heads=2, dim=64, page_stride=2048,
             slot_stride=128, head_stride=64)
    f.update(change)
    c = tovl.tovl_kv_cache(**f)
    cache.alive = c
    return ctypes.addressof(c)


PLAN = dict(length=P, add=P, B=3, table=P, ldt=5, width=5, ring=P, pages=9, page=16, state=P, length_out=P, state_out=P, slots=P,
            positions=P, cap=8, starts=P, stream=None)
ROPE = dict(q=P, ldq=256, k=P, ldk=128, v=P, ldv=128, positions=P, slots=P, cos_sin=P, max_pos=7, rot=64, interleaved=0, T=3, Hq=4,
            cache={}, q_out=P, ldqo=256, stream=None)
ATTN = dict(q=P, ldq=256, B=3, Hq=4, cache={}, table=P, ldt=5, width=5, length=P, scale=0.125, window=0, out=P, ldo=256, lse=P,
            workspace=P, workspace_bytes=4096, stream=None)


PACK = {"tovl_page_plan": (tovl._PLAN_ARGS, "length add table ring state length_out state_out slots positions starts ldt B width pages page cap"),
        "tovl_rope_append": (tovl._ROPE_ARGS, "q k v q_out positions slots cos_sin cache ldq ldk ldv ldqo T Hq max_pos rot interleaved"),
        "tovl_attn_decode": (tovl._ATTN_ARGS, "q out lse table length cache workspace ldq ldo ldt workspace_bytes B Hq width window scale")}


def call(lib, name, base, **change):
    a = {**base, **change}
    if "cache" in a and a["cache"] is not None:
        a["cache"] = cache(**a["cache"])
    before = lib.count()
    pack, names = PACK[name]
    rc = getattr(lib, name)(lib.make(), pack(*(0 if a[n] is None else a[n] for n in names.split())), a["stream"])
    return rc, lib.count() - before


def test_the_binding_packs_the_structs_that_the_header_declares(lib):
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(tovl.__file__))), "include", "tovl.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    for i, (name, (pack, names)) in enumerate(PACK.items()):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + "_args;", text).group(1)
        fields = [n.strip(" *") for line in body.split(";") if line.strip()
                  for n in re.sub(r"^\s*(const )?(void|float|int|long long|tovl_kv_cache)", "", line).split(",")]
        assert fields == names.split(), name
        assert pack.__self__.size == lib.size_of_args(i), name
    for name in PACK:
        assert getattr(lib, name)(lib.make(), None, None) == INVALID


def test_what_fits_is_launched(lib):
    e4m3 = dict(type=tovl.TOVL_E4M3, k_scale=P, v_scale=P)
    for name, base, changes in (
            ("tovl_page_plan", PLAN, [{}, dict(B=4096), dict(cap=0, slots=None, positions=None), dict(ldt=700)]),
            ("tovl_rope_append", ROPE, [{}, dict(rot=0, cos_sin=None, max_pos=0), dict(rot=16), dict(ldq=264, ldk=1024), dict(cache=e4m3)]),
            ("tovl_attn_decode", ATTN, [{}, dict(lse=None), dict(window=1 << 30), dict(cache=e4m3), dict(cache=dict(page=1, slot_stride=0)),
                                        dict(cache=dict(page=1000, page_stride=128000)), dict(cache=dict(head_stride=1024, slot_stride=64)),
                                        dict(cache=dict(heads=1, head_stride=3, slot_stride=64, page_stride=1024)), dict(B=65536)])):
        for c in changes:
            assert call(lib, name, base, **c) == (OK, 1), (name, c)


def test_nothing_to_do_is_not_launched(lib):
    for name, base, n in (("tovl_page_plan", PLAN, "B"), ("tovl_rope_append", ROPE, "T"), ("tovl_attn_decode", ATTN, "B")):
        nothing = {k: None for k, v in base.items() if v == P}
        assert call(lib, name, base, **{**nothing, n: 0, **({"cos_sin": P} if n == "T" else {})}) == (OK, 0), name


@pytest.mark.parametrize("name,base", [("tovl_page_plan", PLAN), ("tovl_rope_append", ROPE), ("tovl_attn_decode", ATTN)])
def test_null_and_misaligned_pointers_are_refused(lib, name, base):
    for k, v in base.items():
        if v != P:
            continue
        if k != "lse":
            assert call(lib, name, base, **{k: None}) == (INVALID, 0), k
        assert call(lib, name, base, **{k: P + 2}) == (INVALID, 0), k


def test_caches_are_mapped_in_boxes_where_their_layout_allows_it(lib):
    """Dimensions of a map: columns, the smaller of head and slot stride, the larger, pages; every stride a multiple of
    the one before.  Boxes lie in one page and have 8 rows at least."""
    def mapped(**c):
        assert call(lib, "tovl_attn_decode", ATTN, cache=c, Hq=4 * c.get("heads", 2), ldq=4096, ldo=4096) == (OK, 1)
        m = lib.last_map()
        return None if m[12] == 0 else (list(m[0:4]), list(m[4:7]), list(m[8:12]))

    assert mapped() == ([64, 2, 16, 9], [128, 256, 4096], [64, 1, 16, 1])
    assert mapped(head_stride=1024, slot_stride=64) == ([64, 16, 2, 9], [128, 2048, 4096], [64, 16, 1, 1])      # heads first
    assert mapped(page=24, page_stride=24 * 128) == ([64, 2, 24, 9], [128, 256, 24 * 256], [64, 1, 8, 1])
    assert mapped(page=64, page_stride=2 * 64 * 128) == ([64, 2, 64, 9], [128, 256, 4 * 64 * 128], [64, 1, 16, 1])
    assert mapped(heads=1, head_stride=5, slot_stride=64, page_stride=1024) == ([64, 1, 16, 9], [128, 128, 2048], [64, 1, 16, 1])
    assert mapped(pages=1, page_stride=3) == ([64, 2, 16, 1], [128, 256, 4096], [64, 1, 16, 1])
    for c in (dict(page=4, page_stride=512), dict(page=1, page_stride=128), dict(page=20, page_stride=2560), dict(page=1000 // 8 * 8 + 4, page_stride=1 << 20),
              dict(slot_stride=136, page_stride=136 * 16), dict(page_stride=2056), dict(head_stride=72, slot_stride=160)):
        assert mapped(**c) is None, c


def test_plan_refusals(lib):
    for c, rc in ((dict(B=-1), INVALID), (dict(B=4097), UNSUPPORTED), (dict(width=0), INVALID), (dict(ldt=4), INVALID),
                  (dict(pages=0), INVALID), (dict(page=0), INVALID), (dict(cap=-1), INVALID), (dict(cap=(1 << 30) + 1), UNSUPPORTED), (dict(pages=BIG, page=2048), UNSUPPORTED)):
        assert call(lib, "tovl_page_plan", PLAN, **c) == (rc, 0), c


def test_append_refusals(lib):
    for c, rc in ((dict(T=-1), INVALID), (dict(Hq=0), INVALID), (dict(rot=-16), INVALID), (dict(rot=80), INVALID), (dict(rot=24), UNSUPPORTED),
                  (dict(max_pos=0), INVALID), (dict(ldq=248), INVALID), (dict(ldq=260), INVALID), (dict(ldk=120), INVALID),
                  (dict(ldv=132), INVALID), (dict(ldqo=192), INVALID), (dict(q=P + 8), INVALID), (dict(cos_sin=P + 8), INVALID),
                  (dict(Hq=4098, ldq=4098 * 64, ldqo=4098 * 64), UNSUPPORTED), (dict(cache=None), INVALID)):
        assert call(lib, "tovl_rope_append", ROPE, **c) == (rc, 0), c


def test_attention_refusals(lib):
    for c, rc in ((dict(B=-1), INVALID), (dict(B=65537), UNSUPPORTED), (dict(Hq=3), INVALID), (dict(Hq=0), INVALID), (dict(Hq=4098), UNSUPPORTED),
                  (dict(window=-1), INVALID), (dict(width=0), INVALID), (dict(ldt=4), INVALID), (dict(ldq=252), INVALID), (dict(ldo=248), INVALID),
                  (dict(workspace=P + 128), INVALID), (dict(workspace_bytes=4095), INVALID), (dict(cache=None), INVALID)):
        assert call(lib, "tovl_attn_decode", ATTN, **c) == (rc, 0), c


@pytest.mark.parametrize("name,base", [("tovl_rope_append", ROPE), ("tovl_attn_decode", ATTN)])
def test_cache_refusals(lib, name, base):
    e4m3 = dict(type=tovl.TOVL_E4M3, k_scale=P, v_scale=P)
    for c, rc in ((dict(type=tovl.TOVL_F32), INVALID), (dict(k=None), INVALID), (dict(v=P + 8), INVALID), (dict(pages=0), INVALID),
                  (dict(page=0), INVALID), (dict(heads=0), INVALID), (dict(dim=0), INVALID), (dict(dim=260), UNSUPPORTED),
                  (dict(dim=264), UNSUPPORTED), (dict(dim=60), UNSUPPORTED), (dict(pages=BIG, page=2048), UNSUPPORTED), (dict(head_stride=56), INVALID),
                  (dict(slot_stride=132), INVALID), (dict(page_stride=-2048), INVALID), (dict(heads=5000), UNSUPPORTED),
                  ({**e4m3, "dim": 72}, UNSUPPORTED), ({**e4m3, "k_scale": None}, INVALID), ({**e4m3, "v_scale": P + 2}, INVALID),
                  ({**e4m3, "slot_stride": 136}, INVALID)):
        assert call(lib, name, base, cache=c) == (rc, 0), c


def test_workspace_sizes(lib):
    h = lib.make()
    assert lib.tovl_attn_decode_workspace(h, 8, 2, 64) == 4096
    for a in ((0, 1, 64), (8, 0, 64), (8, 3, 64), (8, 2, 0), (8, 2, 260), (8, 2, 60), (8192, 2, 64)):
        assert lib.tovl_attn_decode_workspace(h, *a) == -1, a


def test_division_by_a_number_the_host_knows(lib):
    import random
    rng = random.Random(3)
    lib.divide.argtypes = [ctypes.c_uint, ctypes.c_uint]
    for d in [*range(1, 70), 4095, 4096, 4097, 2 ** 30 - 1, 2 ** 30, 2 ** 31 - 1, *(rng.randrange(1, 2 ** 31) for _ in range(300))]:
        top = (2 ** 31 - 1) // d * d
        for x in {0, 1, d - 1, d, min(d + 1, 2 ** 31 - 1), top, top - 1 if top else 0, 2 ** 31 - 1, rng.randrange(2 ** 31)}:
            assert lib.divide(x, d) == x // d, (x, d)


def test_null_handles_are_refused():
    tovl_build.build()
    for name in NAMES:
        args = [0 if a is not tovl._P else None for a in tovl.SIGNATURES[name][0]]
        assert getattr(tovl.load(), name)(*args) == INVALID, name
    assert tovl.load().tovl_attn_decode_workspace(None, 8, 2, 64) == -1


def test_the_binding_and_the_header_agree_on_the_cache():
    import os
    import re
    text = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(tovl.__file__))), "include", "tovl.h")).read()
    body = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} tovl_kv_cache;", body).group(1)
    names = [n.strip(" *") for line in body.split(";") if line.strip() for n in re.sub(r"^\s*(void|float|int|long long)", "", line).split(",")]
    assert names == [n for n, _ in tovl.tovl_kv_cache._fields_]
