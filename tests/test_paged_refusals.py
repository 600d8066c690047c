"""Calls of the paged cache's C ABI that are refused before any device work (no GPU needed)."""
import ctypes
import random

import pytest

from clustered_sparse_decode_b200 import _lib as L
from test_paged_abi import FAKE, attend_args, cache, lib  # noqa: F401


def test_gather_whole_refusals(lib):                 # noqa: F811
    h = ctypes.byref(cache())
    for args in ((-1, FAKE, 3, 3, FAKE, 5, FAKE, FAKE), (1, None, 3, 3, FAKE, 5, FAKE, FAKE), (1, FAKE, 3, 2, FAKE, 5, FAKE, FAKE),
                 (1, FAKE, 3, 3, None, 5, FAKE, FAKE), (1, FAKE, 3, 3, FAKE, 49, FAKE, FAKE), (1, FAKE, 3, 3, FAKE, -1, FAKE, FAKE),
                 (1, FAKE, 3, 3, FAKE, 5, None, FAKE), (1, FAKE, 3, 3, FAKE, 5, FAKE, FAKE + 4)):
        assert lib.mp_paged_gather_whole(h, *args, None) == L.MP_EINVAL


Q, O = 1 << 30, 1 << 31
APART = dict(rows=4, q_heads=8, Q=Q, O=O)            # head dim 64, 2 bytes: a row of 8 heads has 512 elements


@pytest.mark.parametrize("kw,status", [
    (dict(o_row_stride=512, o_head_stride=64), L.MP_OK), (dict(o_row_stride=64, o_head_stride=256), L.MP_OK),
    (dict(o_row_stride=64, o_head_stride=64), L.MP_EINVAL),            # row 1's first head on row 0's second
    (dict(o_row_stride=128, o_head_stride=64), L.MP_EINVAL), (dict(o_row_stride=504, o_head_stride=64), L.MP_EINVAL),
    (dict(o_row_stride=64, o_head_stride=248), L.MP_EINVAL), (dict(o_row_stride=512, o_head_stride=56), L.MP_EINVAL),
    (dict(o_row_stride=56, o_head_stride=512), L.MP_EINVAL),
    (dict(o_row_stride=1024, o_head_stride=128), L.MP_OK), (dict(o_row_stride=192, o_head_stride=128, rows=2, q_heads=2), L.MP_OK),
    (dict(o_row_stride=192, o_head_stride=128, rows=3, q_heads=4), L.MP_EINVAL),     # 2 x 192 = 3 x 128
    (dict(o_row_stride=1 << 60, o_head_stride=1 << 60), L.MP_EINVAL), (dict(o_row_stride=8, o_head_stride=64, rows=1, max_new=1), L.MP_OK),
])
def test_output_rows_do_not_meet(lib, kw, status):   # noqa: F811
    need = ctypes.c_size_t()
    a = attend_args(**{**APART, **kw})
    assert lib.mp_paged_attend_scratch(ctypes.byref(cache()), a, ctypes.byref(need)) == status


@pytest.mark.parametrize("kw", [
    dict(O=Q), dict(O=Q + 4 * 512 * 2 - 16), dict(O=Q - 4 * 512 * 2 + 16),
    # slices of one buffer [4 rows, 24 heads, 64]: the first 8 heads in, others out
    dict(q_row_stride=1536, o_row_stride=1536, O=Q + 7 * 64 * 2), dict(q_row_stride=1536, o_row_stride=1536, O=Q + 17 * 64 * 2),
    dict(q_row_stride=1536, o_row_stride=512, O=Q + 8 * 64 * 2),       # unlike strides in Q's span
    dict(q_row_stride=0, q_head_stride=0, O=Q + 32 * 2),
])
def test_output_does_not_meet_the_queries(lib, kw):  # noqa: F811
    assert lib.mp_paged_attend(ctypes.byref(cache()), attend_args(**{**APART, **kw}), None, 0, None) == L.MP_EINVAL


@pytest.mark.parametrize("seed", range(40))
def test_overlap_by_brute_force(lib, seed):          # noqa: F811
    r = random.Random(seed)
    rows, heads = r.randint(1, 5), r.choice([2, 4, 8])
    a = dict(rows=rows, max_new=1, q_heads=heads, q_row_stride=8 * r.randint(0, 90), q_head_stride=8 * r.randint(1, 60))
    if r.random() < 0.5:
        a.update(o_row_stride=a["q_row_stride"], o_head_stride=a["q_head_stride"])
    else:
        a.update(o_row_stride=8 * r.randint(0, 90), o_head_stride=8 * r.randint(1, 60))
    shift = 8 * r.randint(-150, 150)

    def spots(kind):
        return [t * a[kind + "_row_stride"] * (rows > 1) + h * a[kind + "_head_stride"] for t in range(rows) for h in range(heads)]
    q, o = spots("q"), [x + shift for x in spots("o")]
    need = ctypes.c_size_t()
    args = attend_args(Q=Q, O=Q + 2 * shift, **a)
    meets = any(abs(x - y) < 64 for i, x in enumerate(o) for y in o[:i])
    assert lib.mp_paged_attend_scratch(ctypes.byref(cache()), args, ctypes.byref(need)) == (L.MP_EINVAL if meets else L.MP_OK)
    if meets or any(abs(x - y) < 64 for x in o for y in q):
        assert lib.mp_paged_attend(ctypes.byref(cache()), args, None, 0, None) == L.MP_EINVAL
