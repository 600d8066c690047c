"""Paged attention where rounding could go wrong, against 64-bit results of the same inputs; tolerances count roundings."""
import numpy as np
import pytest

from paged_cases import Case, U, call, check

pytestmark = pytest.mark.gpu


def line_case(n, new, G, dtype, q, k):
    """Scores are single exact products: row r has q[r] in its first element, key j k[j]."""
    c = Case([n], [new], H=1, G=G, d=64, P=64, dtype=dtype, seed=1)
    c.Q[:] = 0.0
    c.Q[:, :, 0] = np.asarray(q)[:, None]
    j = np.arange(n)
    c.K[:] = 0.0
    page, row = c.at(0, j)
    c.K[page, 0, row, 0] = k
    return c


def line_lse_tol(n, info, lse):
    """A score: one exact product, then scaling, base 2 and the maximum's subtraction, 4 roundings of at most zmax.
    A weight's exponential: 2^-21.  A sum of n weights by at least 4 chains: n / 4 roundings.  The logarithm, its
    sum with the maximum and the change of base: 8 roundings of 1 + |lse|."""
    return 2.0 ** -22 * info["zmax"] + 2.0 ** -21 + n / 4 * 2.0 ** -24 + 8 * 2.0 ** -24 * (1 + np.abs(lse))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("G,new", [(1, 1), (4, 4), (8, 4), (1, 64), (4, 40)])
@pytest.mark.parametrize("kind", ["equal", "one_in_four", "spread"])
def test_lse_counts_every_weight_in_32_bits(dtype, G, new, kind):
    n = 256
    j = np.arange(n)
    k = {"equal": np.zeros(n), "one_in_four": np.where(j % 8 >= 6, 0.0, -2048.0), "spread": (j * 37 % 64) / 64.0 - 0.5}[kind]
    c = line_case(n, new, G, dtype, 1.0 + (np.arange(new) % 8) / 8, k)
    got = call(c, scale=1.0, full=True)
    O, lse, info = c.want(scale=1.0, full=True)
    # keys whose weight is 0 do not move the sum, whatever their score
    zmax = {k: (np.minimum(v, 1.0) if k == "zmax" else v) for k, v in info.items()}
    assert (np.abs(got[1] - lse) <= line_lse_tol(n, zmax, lse)).all(), np.abs(got[1] - lse).max()


@pytest.mark.parametrize("G,new", [(1, 1), (4, 3), (8, 3), (1, 20), (1, 64)])
def test_many_small_fp16_weights_add_up(G, new):
    """One key far above 60,000 others, each of whose weights is below half of fp16's smallest step.

    Requests of the same pages, so many that no request's keys are shared out: each keeps one maximum.  A weight's
    rounding is off by at most 2^-25 of 2^7 (the largest weight's place), so n of them by n 2^-32 of the values; the
    exponentials and sums add 2^-19, the output's rounding 2^-11 of it.  The sum beside the lone key is a chain in 32
    bits: a lane adds pairs of weights, a pair in 32 keys, each sum rounded to 2^-24 of it.
    """
    n, B = 60000, 296
    k = np.full(n, -17.5)
    k[123] = 0.0
    c = line_case(n, new, G, "f16", np.ones(new), k)
    c.V[:] = 1.0
    page, row = c.at(0, 123)
    c.V[page, :, row] = 0.0
    O, lse, _ = c.want(scale=1.0)
    assert O.min() > 1e-3
    c.table, c.Q = np.repeat(c.table, B, 0), np.tile(c.Q, (B, 1, 1))
    c.lens, c.new, c.cu, c.rows = [n] * B, [new] * B, np.arange(B + 1) * new, B * new
    got, gl = call(c, scale=1.0)
    off = np.abs(got.reshape(B, new, G, 64) - O)
    assert (off <= n * 2.0 ** -32 + 2.0 ** -19 * O + U["f16"] * O + 2.0 ** -25).all(), off.max()
    assert np.abs(gl.reshape(B, new, G) - lse).max() <= n / 32 * 2.0 ** -24 + 2.0 ** -22 * 17.5 + 2.0 ** -19


CAPS = [1e-40, 0.5, 30.0, 1e4, 1e6, 1e8, 1e20, 1e38, 3.4028234e38]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 64)])
@pytest.mark.parametrize("new", [1, 4, 8, 150])
@pytest.mark.parametrize("cap", CAPS)
def test_caps_of_any_size(dtype, d, new, cap):
    """A cap's error counts by the capped score, which is at most the cap and at most the score."""
    c = Case([500, 160], [new, min(new, 160)], H=2, G=4, d=d, P=32, dtype=dtype, seed=7, qscale=2.0)
    page, row = c.at(0, np.arange(0, 500, 9))
    c.K[page, :, row] = 0.0                                   # scores of 0
    cap = float(np.float32(cap))
    want = c.want(softcap=cap)
    check(c, call(c, softcap=cap), want, np.minimum(cap, want[2]["zmax"])[:int(c.cu[-1])])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [4, 8, 128])
def test_a_rows_cap_does_not_depend_on_its_neighbours(dtype, new):
    """Every other row's scores reach the cap, its neighbours' stay far below it."""
    c = Case([400], [new], H=1, G=4, d=64, P=32, dtype=dtype, seed=11)
    c.Q[1::2] *= 2.0 ** 17
    want = c.want(softcap=2e5)
    check(c, call(c, softcap=2e5), want, np.minimum(2e5, want[2]["zmax"]))
