"""Calls of the paged cache's C ABI that are refused before any device work (no GPU needed)."""
import ctypes

from clustered_sparse_decode_b200 import _lib as L
from test_paged_abi import FAKE, cache, lib  # noqa: F401


def test_gather_whole_refusals(lib):                 # noqa: F811
    h = ctypes.byref(cache())
    for args in ((-1, FAKE, 3, 3, FAKE, 5, FAKE, FAKE), (1, None, 3, 3, FAKE, 5, FAKE, FAKE), (1, FAKE, 3, 2, FAKE, 5, FAKE, FAKE),
                 (1, FAKE, 3, 3, None, 5, FAKE, FAKE), (1, FAKE, 3, 3, FAKE, 49, FAKE, FAKE), (1, FAKE, 3, 3, FAKE, -1, FAKE, FAKE),
                 (1, FAKE, 3, 3, FAKE, 5, None, FAKE), (1, FAKE, 3, 3, FAKE, 5, FAKE, FAKE + 4)):
        assert lib.mp_paged_gather_whole(h, *args, None) == L.MP_EINVAL
