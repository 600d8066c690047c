"""Paged-cache calls at the edges of what their documentation allows."""
import threading

import numpy as np
import pytest
import torch

from clustered_sparse_decode_b200 import Config, MpError, MultipoleIndex, PagedCache
from clustered_sparse_decode_b200 import _lib as L
from oracle import paged as op
from paged_cases import TDT, Case, bounds, cache_of, call, check, dev

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


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 64)])
@pytest.mark.parametrize("new", [1, 6, 300])
@pytest.mark.parametrize("kind", ["one_value", "all_behind"])
@pytest.mark.parametrize("qscale", [1.0, 20.0])
def test_bad_values_of_one_request_stay_its_own(dtype, d, new, kind, qscale):
    """An early NaN and a late infinity among one long request's values: in its own rows where they belong, in the
    columns that hold them, and nowhere else, however small their weights; other requests' rows are written as without
    it."""
    c = Case([16400, 700], [new] * 2, H=1, G=4, d=d, P=64, dtype=dtype, seed=31, qscale=qscale)
    want = c.want()
    tol, ltol = bounds(c, want[2], want[0], want[1])
    late = 16400 - min(50, new // 2 + 1)
    for j, col, bad in ((5, 3, np.nan), (late, 7, np.inf)):
        j = np.arange(j, 16400 if kind == "all_behind" and bad == np.inf else j + 1)
        page, row = c.at(0, j)
        c.V[page, 0, row, col] = bad
    O = want[0].copy()
    pos = np.arange(16400 - new, 16400)
    O[:new, :, 3] = np.nan
    O[np.arange(new)[pos >= late], :, 7] = np.inf
    got = call(c)
    odd = ~np.isfinite(O)
    assert np.array_equal(got[0][odd], O[odd], equal_nan=True)
    assert (np.abs(got[0][~odd] - O[~odd]) <= tol[~odd]).all()
    assert (np.abs(got[1] - want[1]) <= ltol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("new", [1, 6, 100])
def test_values_near_the_types_largest(dtype, new):
    """Weights of up to 2^8 times the largest finite value pass fp32's range; the average of the values does not."""
    c = Case([900], [new], H=1, G=4, d=64, P=32, dtype=dtype, seed=13)
    top = torch.finfo(TDT[dtype]).max
    for j, col in ((3, 1), (500, 5), (700, 9), (810, 60)):
        page, row = c.at(0, j)
        c.V[page, 0, row, col] = top if j % 2 else -top
    want = c.want()
    got = call(c)
    tol = bounds(c, want[2], want[0], want[1])[0]
    assert np.isfinite(got[0]).all()
    assert (np.abs(got[0] - want[0]) <= tol).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("new", [1, 4, 40, 300])
def test_a_bad_page_is_nobody_elses(dtype, P, new):
    """What a request with a bad table entry gets comes from no other page, and other requests' rows stay."""
    c = Case([700, 700, 350], [new] * 3, H=2, G=4, d=64, P=P, dtype=dtype, seed=5)
    want = c.want()
    tol = bounds(c, want[2], want[0], want[1])[0]
    table = c.table.copy()
    table[0, 1], table[1, 0] = c.pages, -1
    mine = set(table[:2].ravel()) | set(c.table[2].ravel())
    for p in range(c.pages):
        if p not in mine:
            c.K[p], c.V[p] = 1.0, 1000.0
    # whatever page stands first in the pool is one of these
    z = next(p for p in range(c.pages) if p not in mine)
    order = np.arange(c.pages)
    order[[0, z]] = z, 0
    c.K, c.V = c.K[order], c.V[order]
    moved = np.where(table == 0, z, np.where(table == z, 0, table))
    cache = cache_of(c)
    out = cache.attend(dev(c.Q, dtype), dev(moved), dev(c.lens), dev(c.cu), max_new=new).double().cpu().numpy()
    assert cache.check_device_error() == 1
    assert np.abs(out[:2 * new]).max() < 10
    assert (np.abs(out[2 * new:] - want[0][2 * new:]) <= tol[2 * new:]).all()


@pytest.mark.parametrize("lens", [[-1, 40], [20, 65], [20, 1 << 30]])
def test_gather_flags_lengths_outside_the_table(lens):
    c = Case([20, 64], [0, 0], H=1, G=1, d=64)
    cache = cache_of(c)
    n = 30
    K, _ = cache.gather(dev(c.table), dev(lens), n)
    held = [min(max(m, 0), 64) for m in lens]
    assert np.array_equal(K.double().cpu().numpy(), op.gather(c.K, c.table, held, n, 16))
    assert cache.check_device_error() == 1


def test_build_paged_flags_requests_shorter_than_n():
    c = Case([64, 50], [0, 0], H=1, G=1, d=64)
    cfg = Config(batch=2, kv_heads=1, q_heads=1, head_dim=64, max_tokens=64, block_tokens=64, kmeans_iters=1)
    cache, idx = cache_of(c), MultipoleIndex(cfg)
    idx.build_paged(cache, dev(c.table), dev(c.lens), 50)
    assert cache.check_device_error() == 0
    idx.build_paged(cache, dev(c.table), dev(c.lens), 51)
    assert cache.check_device_error() == 1
    assert idx.check_device_error() == 0


@pytest.mark.parametrize("new", [1, 4, 60])
def test_queries_and_output_in_one_buffer(new):
    """Slices of a joined projection that do not overlap are taken, the queries' own place is refused."""
    c = Case([300, 90], [new, new], H=2, G=2, d=64, P=32, dtype="bf16", seed=17)
    cache = cache_of(c)
    buf = torch.zeros(c.rows, 12, 64, dtype=torch.bfloat16, device="cuda")
    O, lse, info = c.want()
    tol = bounds(c, info, O, lse)[0]
    for at in (0, 4, 8):
        q, out = buf[:, 4:8], buf[:, at:at + 4]
        q.copy_(dev(c.Q, "bf16"))
        args = dict(max_new=new, out=out)
        if at == 4:
            with pytest.raises(MpError) as e:
                cache.attend(q, dev(c.table), dev(c.lens), dev(c.cu), **args)
            assert e.value.status == L.MP_EINVAL
            continue
        cache.attend(q, dev(c.table), dev(c.lens), dev(c.cu), **args)
        assert (np.abs(out.double().cpu().numpy() - O) <= tol).all()
        assert torch.equal(q, dev(c.Q, "bf16"))
    assert cache.check_device_error() == 0


def many_requests(B, P=16):
    """A step of B requests on its own cache: the call, and what it has to give."""
    r = np.random.default_rng(B)
    lens, new = r.integers(0, 40, B), r.integers(0, 3, B)
    need = int((-(-(lens + new) // P)).sum())
    table = np.full((B, 4), -3)
    ids, at = r.permutation(need + 5), 0
    for b, n in enumerate(lens):
        h = -(-int(n) // P)
        table[b, :h] = ids[at:at + h]
        at += h
    free, rows = ids[at:], int(new.sum()) + 3
    cache = PagedCache(1, 64, need + 5, P)
    args = dev(lens), dev(new), dev(table), dev(free), dev([len(free)])
    want = op.plan(lens, new, table, free, len(free), P, rows)

    def check(p):
        for got, w in zip((p.lens, p.cu, p.slots, p.positions, p.free_count, args[2]), want):
            assert np.array_equal(got.cpu().numpy().reshape(np.shape(w)), w)
        assert cache.check_device_error() == 0
    return cache, args, rows, check


@pytest.mark.parametrize("B", [3000, 4000, 8192])
def test_plan_of_thousands_of_requests(B):
    cache, args, rows, check = many_requests(B)
    check(cache.plan(*args, rows=rows))


def test_plans_of_unlike_sizes_from_two_threads():
    """A kernel's shared memory is set for the device's context, whoever else is about to launch it."""
    steps = [many_requests(B) for B in (3500, 8192)]
    plans, errors = [None, None], []

    def work(k):
        cache, args, rows, _ = steps[k]
        out = cache.new_plan(args[0].numel(), rows)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.default_stream())
        try:
            for _ in range(2000):
                plans[k] = cache.plan(*args, out=out, stream=s)
        except Exception as e:                               # noqa: BLE001
            errors.append(e)
    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    [t.start() for t in threads]
    [t.join() for t in threads]
    torch.cuda.synchronize()
    assert not errors
    for (_, _, _, check), p in zip(steps, plans):
        check(p)


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new", [1, 4, 60, 300])
@pytest.mark.parametrize("axis", ["rows", "heads", "both"])
def test_expanded_queries(dtype, new, axis):
    """Queries whose rows or heads stand on one another, whichever kernel the number of rows leads to."""
    c = Case([400, 333], [new, min(new, 333)], H=2, G=4, d=64, P=32, dtype=dtype, seed=19, poison=np.nan)
    q = dev(c.Q, dtype)
    q = q[:1] if axis != "heads" else q
    q = (q[:, :1] if axis != "rows" else q).expand(c.rows, c.H * c.G, 64)
    assert 0 in q.stride()
    c.Q = q.double().cpu().numpy()
    check(c, call(c, q=q), c.want())
    cache, out = cache_of(c), torch.empty(c.rows, c.H * c.G, 64, dtype=TDT[dtype], device="cuda")
    g = torch.cuda.CUDAGraph()
    args = q, dev(c.table), dev(c.lens), dev(c.cu)
    ref = cache.attend(*args, max_new=new)
    with torch.cuda.graph(g):
        cache.attend(*args, max_new=new, out=out)
    g.replay()
    assert torch.equal(out, ref) and cache.check_device_error() == 0


def test_append_of_a_single_row_from_unlike_views():
    """The strides of an axis of length 1 mean nothing, so K_new's and V_new's may differ there."""
    cache = PagedCache(2, 64, 4, 16)
    cache.K.zero_(), cache.V.zero_()
    kv = torch.randn(1, 4, 64, device="cuda").bfloat16()
    k, v = kv[:, :2], kv[:, 2:].clone(memory_format=torch.contiguous_format)
    assert k.stride() != v.stride()
    cache.append(k, v, torch.tensor([17], device="cuda"))
    assert torch.equal(cache.K[1, :, 1], k[0]) and torch.equal(cache.V[1, :, 1], v[0])
    one = PagedCache(1, 64, 4, 16)
    x = torch.randn(3, 2, 64, device="cuda").bfloat16()
    k, v = x[:, :1], x.transpose(0, 1).contiguous().transpose(0, 1)[:, 1:]
    one.append(x[:, :1], x.as_strided((3, 1, 64), (128, 64, 1), 64), torch.tensor([1, 2, 3], device="cuda"))
    one.append(k.as_strided((3, 1, 64), (128, 8, 1)), k, torch.tensor([5, 6, 7], device="cuda"))
    assert torch.equal(one.K[0, 0, 5:8], k[:, 0]) and torch.equal(one.V[0, 0, 5:8], k[:, 0])


def test_pool_of_a_single_page_or_head_from_unlike_views():
    """The same for the pool's own K and V."""
    kv = torch.zeros(2, 1, 3, 16, 64, dtype=torch.bfloat16, device="cuda")
    K, V = kv[0], torch.zeros(1, 6, 16, 64, dtype=torch.bfloat16, device="cuda")[:, :3]
    assert K.stride() != V.stride()
    cache = PagedCache(3, 64, 1, 16, K=K, V=V)
    x = torch.randn(2, 3, 64, device="cuda").bfloat16()
    cache.append(x, x, torch.tensor([0, 15], device="cuda"))
    for X in (K, V):
        assert torch.equal(X[0, :, 0], x[0]) and torch.equal(X[0, :, 15], x[1])
    one = torch.zeros(16 * 64, dtype=torch.bfloat16, device="cuda").as_strided((1, 1, 16, 64), (7, 12345, 64, 1))
    cache = PagedCache(1, 64, 1, 16, K=one, V=torch.zeros_like(one))
    cache.append(x[:, :1], x[:, :1], torch.tensor([0, 15], device="cuda"))
    assert torch.equal(one[0, 0, 15], x[1, 0])
    with pytest.raises(ValueError):
        PagedCache(3, 64, 1, 16, K=K, V=torch.zeros(1, 16, 3, 64, dtype=torch.bfloat16, device="cuda").transpose(1, 2))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("G,new", [(1, 1), (8, 4), (1, 64)])
@pytest.mark.parametrize("n", [600, 30000])
def test_infinities_and_nan_outlast_any_factor(dtype, G, new, n):
    """Keys whose weights beside the others' underflow, in a part of the keys that others finish: what is not finite among
    them is still seen, what is finite has no weight."""
    c = Case([n], [new], H=1, G=G, d=64, P=32, dtype=dtype, seed=23)
    page, row = c.at(0, np.arange(n))
    c.Q[:], c.K[:] = 0.0, 0.0
    c.Q[:, :, 0] = 1.0
    c.K[page, 0, row, 0] = np.where(np.arange(n) < n // 2, -1000.0, 0.0)
    want = c.want(scale=1.0)
    tol = bounds(c, want[2], want[0], want[1])[0]
    O = want[0].copy()
    for j, col, bad in ((3, 7, np.inf), (40, 9, np.nan), (n // 2 - 300, 11, -np.inf), (3, 13, np.inf), (n // 2 - 1, 13, -np.inf)):
        page, row = c.at(0, j)
        c.V[page, 0, row, col] = bad
        O[..., col] = np.nan if np.isinf(O[0, 0, col]) else bad
    got = call(c, scale=1.0)[0]
    odd = ~np.isfinite(O)
    assert np.array_equal(got[odd], O[odd], equal_nan=True)
    assert (np.abs(got[~odd] - O[~odd]) <= tol[~odd]).all()


@pytest.mark.parametrize("dtype,d", [("bf16", 64), ("bf16", 128), ("f16", 64), ("f32", 64)])
@pytest.mark.parametrize("new", [1, 3, 60, 300])
@pytest.mark.parametrize("kw", [{}, dict(softcap=2.0), dict(window=90)], ids=["plain", "cap", "window"])
def test_results_are_the_same_bits_after_other_calls(dtype, d, new, kw):
    """What earlier calls leave in an SM's memories, and what lies behind a request's tokens, moves no bit of the result."""
    c = Case([400, 333, 70], [new, new, min(new, 70)], H=2, G=4, d=d, P=32, dtype=dtype, seed=19, poison=0.0)
    first = call(c, **kw)
    others = []
    for k, fill in enumerate((np.nan, 30.0, -50.0)):
        o = Case([900, 500], [61, 300], H=2, G=4, d=d, P=32, dtype=dtype, seed=50 + k, poison=fill, qscale=10.0 ** k)
        o.K *= 5.0
        others.append((o, cache_of(o)))
    caches = [cache_of(c)]
    for fill in (np.nan, 100.0):
        x = Case(c.lens, c.new, H=2, G=4, d=d, P=32, dtype=dtype, seed=19, poison=fill)
        caches.append(cache_of(x))
    for turn in range(30):
        o, cache = others[turn % 3]
        cache.attend(dev(o.Q, dtype), dev(o.table), dev(o.lens), dev(o.cu), max_new=300)
        got = call(c, cache=caches[turn % len(caches)], **kw)
        assert np.array_equal(got[0], first[0]) and np.array_equal(got[1], first[1]), turn
