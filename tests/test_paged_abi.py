"""The paged cache's C ABI without a GPU: struct layouts, refusals before any device work."""
import ctypes
import os
import subprocess

import pytest

from clustered_sparse_decode_b200 import _lib as L
from clustered_sparse_decode_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLASSES = {"mp_paged_config": L.MpPagedConfig, "mp_paged_cache": L.MpPagedCache, "mp_paged_plan_args": L.MpPagedPlanArgs,
           "mp_paged_attend_args": L.MpPagedAttendArgs}


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def test_struct_layouts_match_the_header(tmp_path):
    lines = ['#include <stdio.h>', '#include <stddef.h>', '#include "mpattn.h"', "int main(void){"]
    for s, cls in CLASSES.items():
        lines.append(f'printf("{s} %zu\\n", sizeof({s}));')
        lines += [f'printf("{s}.{f[0]} %zu\\n", offsetof({s}, {f[0]}));' for f in cls._fields_]
    (tmp_path / "p.c").write_text("\n".join(lines + ["return 0;}"]))
    subprocess.run(["gcc", "-std=c99", "-I", os.path.join(ROOT, "include"), str(tmp_path / "p.c"), "-o", str(tmp_path / "p")],
                   check=True)
    got = dict(x.split() for x in subprocess.run([str(tmp_path / "p")], capture_output=True, text=True).stdout.splitlines())
    for s, cls in CLASSES.items():
        assert int(got[s]) == ctypes.sizeof(cls)
        for f in cls._fields_:
            assert int(got[f"{s}.{f[0]}"]) == getattr(cls, f[0]).offset, f"{s}.{f[0]}"
    assert L.PLAN_ARGS.size == int(got["mp_paged_plan_args"]) and L.ATTEND_ARGS.size == int(got["mp_paged_attend_args"])


FAKE = 1 << 20                                       # an address that no refused call looks at


@pytest.mark.parametrize("kw,status", [
    (dict(kv_heads=0), L.MP_EINVAL), (dict(num_pages=0), L.MP_EINVAL), (dict(page_tokens=0), L.MP_EINVAL),
    (dict(dtype=3), L.MP_EINVAL), (dict(reserved=1), L.MP_EINVAL), (dict(head_dim=96), L.MP_EUNSUPPORTED),
    (dict(page_tokens=24), L.MP_EUNSUPPORTED), (dict(page_tokens=512), L.MP_EUNSUPPORTED),
    (dict(page_tokens=8), L.MP_EUNSUPPORTED), (dict(kv_heads=1 << 20), L.MP_EUNSUPPORTED),
    (dict(token_stride=64, head_stride=1024, page_stride=0), L.MP_EINVAL),
    (dict(token_stride=65, head_stride=1040, page_stride=2080), L.MP_EINVAL),
    (dict(token_stride=64, head_stride=1024, page_stride=1 << 40), L.MP_EUNSUPPORTED),
])
def test_init_refusals(lib, kw, status):
    c = L.MpPagedConfig(kv_heads=2, head_dim=64, num_pages=4, page_tokens=16, dtype=L.MP_BF16)
    for k, v in kw.items():
        setattr(c, k, v)
    out = L.MpPagedCache()
    assert lib.mp_paged_init(ctypes.byref(c), FAKE, FAKE, FAKE, ctypes.byref(out)) == status


def test_null_and_misaligned_pointers(lib):
    c = L.MpPagedConfig(kv_heads=2, head_dim=64, num_pages=4, page_tokens=16, dtype=L.MP_BF16)
    out = L.MpPagedCache()
    for k, v, e in ((0, FAKE, FAKE), (FAKE, 0, FAKE), (FAKE, FAKE, 0), (FAKE + 8, FAKE, FAKE), (FAKE, FAKE + 2, FAKE),
                    (FAKE, FAKE, FAKE + 1)):
        assert lib.mp_paged_init(ctypes.byref(c), k or None, v or None, e or None, ctypes.byref(out)) == L.MP_EINVAL
    assert lib.mp_paged_init(None, FAKE, FAKE, FAKE, ctypes.byref(out)) == L.MP_EINVAL


def cache(dtype=L.MP_BF16, **kw):
    h = L.MpPagedCache()
    h.cfg = L.MpPagedConfig(kv_heads=2, head_dim=64, num_pages=4, page_tokens=16, dtype=dtype, page_stride=2048,
                            head_stride=1024, token_stride=64)
    h.K = h.V = h.err = FAKE
    h.sms = 148
    return h


def attend_args(**kw):
    a = L.MpPagedAttendArgs(batch=2, q_heads=8, rows=4, max_new=2, table_pages=3, table_stride=3, table=FAKE, lens=FAKE,
                            cu=FAKE, Q=FAKE, O=FAKE, q_row_stride=512, q_head_stride=64, o_row_stride=512,
                            o_head_stride=64)
    for k, v in kw.items():
        setattr(a, k, v)
    return bytes(a)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), L.MP_EINVAL), (dict(rows=-1), L.MP_EINVAL), (dict(max_new=5), L.MP_EINVAL), (dict(max_new=-1), L.MP_EINVAL),
    (dict(q_heads=7), L.MP_EINVAL), (dict(q_heads=6), L.MP_EUNSUPPORTED), (dict(q_heads=32), L.MP_EUNSUPPORTED),
    (dict(table_stride=2), L.MP_EINVAL), (dict(table=None), L.MP_EINVAL), (dict(lens=None), L.MP_EINVAL),
    (dict(cu=None), L.MP_EINVAL), (dict(Q=None), L.MP_EINVAL), (dict(O=None), L.MP_EINVAL), (dict(Q=FAKE + 2), L.MP_EINVAL),
    (dict(O=FAKE + 8), L.MP_EINVAL), (dict(q_row_stride=-8), L.MP_EINVAL), (dict(q_head_stride=4), L.MP_EINVAL),
    (dict(o_row_stride=0), L.MP_EINVAL), (dict(o_head_stride=0), L.MP_EINVAL), (dict(scale=float("nan")), L.MP_EINVAL),
    (dict(softcap=-1.0), L.MP_EINVAL), (dict(softcap=float("inf")), L.MP_EINVAL), (dict(window=-1), L.MP_EINVAL),
    (dict(flags=2), L.MP_EINVAL), (dict(batch=1 << 17), L.MP_EUNSUPPORTED), (dict(rows=(1 << 24) + 1), L.MP_EUNSUPPORTED),
    (dict(table_pages=1 << 27, table_stride=1 << 27), L.MP_EUNSUPPORTED), (dict(), L.MP_OK),
])
def test_attend_refusals(lib, kw, status):
    h, need = cache(), ctypes.c_size_t()
    assert lib.mp_paged_attend_scratch(ctypes.byref(h), attend_args(**kw), ctypes.byref(need)) == status
    if status != L.MP_OK:
        assert lib.mp_paged_attend(ctypes.byref(h), attend_args(**kw), None, 0, None) == status


def test_scratch_is_asked_for_where_keys_are_shared_out(lib):
    def need(dtype=L.MP_BF16, **kw):
        n = ctypes.c_size_t()
        assert lib.mp_paged_attend_scratch(ctypes.byref(cache(dtype)), attend_args(**kw), ctypes.byref(n)) == L.MP_OK
        return n.value
    long = dict(table_pages=1 << 16, table_stride=1 << 16)
    assert need() == 0 and need(L.MP_F32) == 0 and need(rows=0, max_new=0) == 0 and need(batch=0) == 0
    for dtype in (L.MP_BF16, L.MP_F16, L.MP_F32):
        assert need(dtype, **long) > 0
    # 256 rows of 64 + 2 floats, two parts of each of 148 blocks
    assert need(rows=400, max_new=200) >= 2 * 148 * 256 * 66 * 4


@pytest.mark.parametrize("kw", [dict(batch=-1), dict(table_pages=-1), dict(table_stride=2), dict(rows=-1), dict(free_capacity=-1),
                                dict(reserved=1), dict(lens=None), dict(new_tokens=None), dict(table=None),
                                dict(free_pages=None), dict(free_count=None), dict(lens_out=None), dict(cu_out=None),
                                dict(slots_out=None), dict(positions_out=None), dict(free_count_out=None)])
def test_plan_refusals(lib, kw):
    a = L.MpPagedPlanArgs(batch=2, table_pages=3, table_stride=3, rows=4, free_capacity=5)
    for f, t in L.MpPagedPlanArgs._fields_:
        if t is ctypes.c_void_p:
            setattr(a, f, FAKE)
    for k, v in kw.items():
        setattr(a, k, v)
    assert lib.mp_paged_plan(ctypes.byref(cache()), bytes(a), None) == L.MP_EINVAL


def test_plan_of_too_many_requests(lib):
    a = L.MpPagedPlanArgs(batch=8193, table_pages=3, table_stride=3, rows=4, free_capacity=5)
    for f, t in L.MpPagedPlanArgs._fields_:
        if t is ctypes.c_void_p:
            setattr(a, f, FAKE)
    assert lib.mp_paged_plan(ctypes.byref(cache()), bytes(a), None) == L.MP_EUNSUPPORTED


def test_append_and_gather_refusals(lib):
    h = ctypes.byref(cache())                        # byref holds the cache, its bare address would not
    for args in ((FAKE, FAKE, 128, 64, FAKE, -1), (None, FAKE, 128, 64, FAKE, 2), (FAKE, None, 128, 64, FAKE, 2),
                 (FAKE, FAKE, 128, 64, None, 2), (FAKE + 2, FAKE, 128, 64, FAKE, 2), (FAKE, FAKE, 124, 64, FAKE, 2),
                 (FAKE, FAKE, 128, 4, FAKE, 2), (FAKE, FAKE, -128, 64, FAKE, 2)):
        assert lib.mp_paged_append(h, *args, None) == L.MP_EINVAL
    for args in ((-1, FAKE, 3, 3, FAKE, 5, FAKE, FAKE), (1, None, 3, 3, FAKE, 5, FAKE, FAKE), (1, FAKE, 3, 2, FAKE, 5, FAKE, FAKE),
                 (1, FAKE, 3, 3, None, 5, FAKE, FAKE), (1, FAKE, 3, 3, FAKE, 49, FAKE, FAKE), (1, FAKE, 3, 3, FAKE, -1, FAKE, FAKE),
                 (1, FAKE, 3, 3, FAKE, 5, None, FAKE), (1, FAKE, 3, 3, FAKE, 5, FAKE, FAKE + 4)):
        assert lib.mp_paged_gather(h, *args, None) == L.MP_EINVAL
    assert lib.mp_paged_append(None, FAKE, FAKE, 128, 64, FAKE, 2, None) == L.MP_EINVAL
