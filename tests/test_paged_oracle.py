"""The paged-cache oracle against the framework's other oracle, closed forms and brute force (CPU)."""
import numpy as np
import pytest

from oracle import multipole as mp
from oracle import paged as op
from paged_cases import Case


def test_attention_of_single_tokens_is_the_dense_oracles():
    c = Case([37, 80], [1, 1], H=2, G=2, d=64, dtype="f32")
    K, V = (op.gather(x, c.table, [37, 37], 37, 16) for x in (c.K, c.V))
    O, _, _ = op.attend(c.Q, c.K, c.V, c.table, [37, 37], c.cu, 16)
    np.testing.assert_allclose(O, mp.dense_attention(c.Q, K, V, 37, 2), rtol=0, atol=1e-12)


def test_a_chunk_is_its_tokens_one_by_one():
    c = Case([21], [6], H=1, G=2, d=64, dtype="f32")
    O, lse, _ = c.want()
    for i in range(6):
        o, l, _ = op.attend(c.Q[i:i + 1], c.K, c.V, c.table, [16 + i], [0, 1], 16)
        np.testing.assert_allclose(o[0], O[i], atol=1e-12)
        np.testing.assert_allclose(l[0], lse[i], atol=1e-12)


def test_masks_by_hand():
    """Equal keys: the output is the mean of the values seen, the lse the log of their number plus the score."""
    c = Case([8], [8], H=1, G=1, d=64, dtype="f32")
    c.K[:] = 0.0
    v = op.rows_of(c.V, c.table[0], 8, 16)[0]
    for kw, spans in [({}, [(0, i + 1) for i in range(8)]), (dict(window=3), [(max(0, i - 2), i + 1) for i in range(8)]),
                      (dict(full=True), [(0, 8)] * 8), (dict(prefix=[4]), [(0, max(4, i + 1)) for i in range(8)]),
                      (dict(first_key=[0, 0, 2, 2, 2, 5, 5, 7]), list(zip([0, 0, 2, 2, 2, 5, 5, 7], range(1, 9)))),
                      (dict(first_key=[1] * 8), [(1, i + 1) for i in range(8)])]:
        O, lse, _ = c.want(**kw)
        for i, (lo, hi) in enumerate(spans):
            if hi <= lo:
                assert (O[i] == 0).all() and lse[i, 0] == -np.inf
            else:
                np.testing.assert_allclose(O[i, 0], v[lo:hi].mean(0), atol=1e-12)
                np.testing.assert_allclose(lse[i, 0], np.log(hi - lo), atol=1e-12)


def test_cap_and_bias_by_hand():
    c = Case([2], [1], H=1, G=1, d=64, dtype="f32")
    c.Q[:] = 0.0
    c.Q[0, 0, 0] = 8.0                                        # scale 1/8: the score is the key's first element
    k, v = op.rows_of(c.K, c.table[0], 2, 16)[0], op.rows_of(c.V, c.table[0], 2, 16)[0]
    z = 2.0 * np.tanh(k[:, 0] / 2.0) - 0.5 * np.array([1.0, 0.0])
    w = np.exp(z) / np.exp(z).sum()
    np.testing.assert_allclose(c.want(softcap=2.0, slopes=[0.5])[0][0, 0], w @ v, atol=1e-12)


def test_plan_by_hand():
    lens, cu, slots, pos, left, table = op.plan([3, 4, 0], [2, 1, 0], [[5, -1], [6, -1], [-1, -1]], [9, 8, 7], 3, 4, 4)
    assert lens.tolist() == [5, 5, 0] and cu.tolist() == [0, 2, 3, 3] and left == 1
    assert slots.tolist() == [23, 28, 32, -1] and pos.tolist() == [3, 4, 4, 0]
    assert table.tolist() == [[5, 7], [6, 8], [-1, -1]]


@pytest.mark.parametrize("kw", [dict(count=1), dict(rows=2), dict(lens=[-1, 4]), dict(new=[2, 9])])
def test_plan_refuses(kw):
    a = dict(lens=[3, 4], new=[2, 1], table=[[5, -1], [6, -1]], free=[9, 8, 7], count=3, P=4, rows=3)
    assert op.plan(**a) is not None
    assert op.plan(**{**a, **kw}) is None
