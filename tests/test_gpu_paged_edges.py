"""Paged-cache calls at the edges of what their documentation allows."""
import numpy as np
import pytest

from paged_cases import Case, bounds, cache_of, call

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 64)])
@pytest.mark.parametrize("n,new", [(300, 200), (5000, 600)])
def test_rows_done_again_are_the_ones_that_stay(dtype, d, n, new):
    """Every row shares a tile with an infinite value that it does not see: whole units and shared-out ones, many times."""
    c = Case([n], [new], H=1, G=4, d=d, P=32, dtype=dtype, seed=21)
    first = np.full(c.rows, n - new - 40)
    want = c.want(first_key=first)
    page, row = c.at(0, np.arange(n - new - 60, n - new - 40))
    c.V[page, :, row] = np.inf
    tol = bounds(c, want[2], want[0], want[1])[0]
    cache = cache_of(c)
    for _ in range(10):
        got = call(c, cache=cache, first_key=first)
        assert (np.abs(got[0] - want[0]) <= tol).all()
