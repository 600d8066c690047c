"""The paged-cache calls against their 64-bit oracle: addresses, appending, attention, gathering, and a run of them together.

Error bounds are derived in paged_cases.bounds; copies and addresses are exact.
"""
import numpy as np
import pytest
import torch

import helpers as H
from clustered_sparse_decode_b200 import Config, MpError, MultipoleIndex, PagedCache
from clustered_sparse_decode_b200 import _lib as L
from oracle import paged as op
from paged_cases import Case, TDT, bounds, cache_of, call, check, dev

pytestmark = pytest.mark.gpu


def small_cache(P=16, pages=64, **kw):
    return PagedCache(kv_heads=kw.pop("H", 2), head_dim=64, num_pages=pages, page_tokens=P, dtype="bf16", **kw)


# ---------------------------------------------------------------------------
# Step addresses
# ---------------------------------------------------------------------------
def plan_inputs(lens, new, P, W, pages, seed=0):
    r = np.random.default_rng(seed)
    ids, at = r.permutation(pages), 0
    table = np.full((len(lens), W), -3)
    for b, n in enumerate(lens):
        h = -(-n // P)
        table[b, :h] = ids[at:at + h]
        at += h
    free = np.concatenate([ids[at:], np.full(at, -9)])
    return table, free, pages - at


def run_plan(c, lens, new, table, free, count, rows, **kw):
    t = dev(table)
    p = c.plan(dev(lens), dev(new), t, dev(free), dev([count]), rows=rows, **kw)
    return p, t


@pytest.mark.parametrize("P", [16, 64, 256])
@pytest.mark.parametrize("lens,new", [
    ([0], [1]), ([15, 16, 17], [1, 1, 1]), ([0, 0, 5], [33, 0, 16]), ([100] * 5, [0] * 5), ([], []),
    ([31] * 300, [1] * 300), ([0, 700, 3], [1500, 2, 0]), ([7] * 1100, list(range(1100))),
])
def test_plan(P, lens, new):
    rows = sum(new) + (5 if len(lens) != 3 else 0)
    W = max([-(-(a + b) // P) for a, b in zip(lens, new)], default=0) + 1
    pages = sum(-(-(a + b) // P) for a, b in zip(lens, new)) + 2
    table, free, count = plan_inputs(lens, new, P, W, pages)
    c = small_cache(P, pages)
    p, t = run_plan(c, lens, new, table, free, count, rows)
    want = op.plan(lens, new, table, free, count, P, rows)
    for got, w in zip((p.lens, p.cu, p.slots, p.positions, p.free_count, t), want):
        assert np.array_equal(got.cpu().numpy().reshape(np.shape(w)), w)
    assert c.check_device_error() == 0


def test_plan_in_place_and_replayed():
    """Lengths and count advanced in place by a captured step, replayed: 40 steps of the oracle."""
    P, B, W, pages = 16, 5, 8, 40
    lens, new = [0, 3, 15, 16, 40], [1, 1, 0, 2, 1]
    table, free, count = plan_inputs(lens, new, P, W, pages)
    c = small_cache(P, pages)
    dl, dn, dt, df, dc = dev(lens), dev(new), dev(table), dev(free), dev([count])
    p = c.new_plan(B, 8)
    p.lens, p.free_count = dl, dc
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.plan(dl, dn, dt, df, dc, out=p)
    for _ in range(12):
        lens, cu, slots, pos, count, table = op.plan(lens, new, table, free, count, P, 8)
        g.replay()
        torch.cuda.synchronize()
        for got, w in ((dl, lens), (p.cu, cu), (p.slots, slots), (p.positions, pos), (dc, [count]), (dt, table)):
            assert np.array_equal(got.cpu().numpy(), w)


def test_plan_wide_in_place():
    """More rows than one pass of the blocks of an in-place step takes."""
    P, lens, new = 32, [5, 0, 77], [30000, 1, 20011]
    pages = sum(-(-(a + b) // P) for a, b in zip(lens, new))
    W = -(-30005 // P)
    table, free, count = plan_inputs(lens, new, P, W, pages)
    want = op.plan(lens, new, table, free, count, P, sum(new))
    for in_place in (False, True):
        c = small_cache(P, pages)
        dl, dc, dt = dev(lens), dev([count]), dev(table)
        p = c.new_plan(3, sum(new))
        if in_place:
            p.lens, p.free_count = dl, dc
        c.plan(dl, dev(new), dt, dev(free), dc, out=p)
        for got, w in zip((p.lens, p.cu, p.slots, p.positions, p.free_count, dt), want):
            assert np.array_equal(got.cpu().numpy().reshape(np.shape(w)), w)


@pytest.mark.parametrize("kw", [dict(count=2), dict(rows=20), dict(lens=[-1, 16]), dict(new=[-2, 20]), dict(new=[3, 200]),
                                dict(count=-1), dict(count=1000), dict(lens=[2 ** 31 - 5, 3])])
def test_plan_that_does_not_fit_changes_nothing(kw):
    P, W = 16, 4
    a = dict(lens=[5, 16], new=[20, 20], count=10, rows=45)
    table, free, _ = plan_inputs([5, 16], [20, 20], P, W, 16)
    a.update(kw)
    c = small_cache(P, 16)
    p, t = run_plan(c, a["lens"], a["new"], table, free, a["count"], a["rows"])
    assert np.array_equal(t.cpu().numpy(), table)
    assert p.lens.tolist() == a["lens"] and p.free_count.tolist() == [a["count"]]
    assert (p.slots == -1).all() and (p.positions == 0).all() and (p.cu == 0).all()
    assert c.check_device_error() == 8
    assert c.check_device_error() == 0


def test_plan_bad_page_ids_give_no_slot():
    c = small_cache(16, 8)
    p, t = run_plan(c, [3, 0], [1, 2], np.array([[99, -1], [-1, -1]]), [1, 2, -5], 3, 3)
    assert p.slots.tolist() == [-1, -1, -1] and t.tolist() == [[99, -1], [-1, -1]]
    assert c.check_device_error() == 1


# ---------------------------------------------------------------------------
# Appending and gathering
# ---------------------------------------------------------------------------
LAYOUTS = ["hptd", "token_major", "joined", "head_major"]


@pytest.mark.parametrize("dtype,d,heads,P,rows", [("bf16", 128, 8, 16, 1), ("f16", 64, 3, 32, 77), ("f32", 64, 1, 16, 500),
                                                  ("bf16", 128, 2, 256, 4099), ("f32", 128, 2, 64, 0)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_append(dtype, d, heads, P, rows, layout):
    r = np.random.default_rng(rows)
    c = Case([rows + 9], [1], H=heads, G=1, d=d, P=P, dtype=dtype, seed=rows)
    cache = cache_of(c, layout)
    slots = r.permutation(c.pages * P)[:rows].astype(np.int64)
    skip = r.random(rows) < 0.2
    kv = torch.randn(rows, 3, heads, d, device="cuda").to(TDT[dtype])     # slices of a joined projection
    k, v = kv[:, 1], kv[:, 2]
    K, V = cache.K.clone(), cache.V.clone()
    s = torch.from_numpy(np.where(skip, -1 - (slots % 3), slots)).cuda()
    cache.append(k, v, s)
    for t in range(rows):
        if not skip[t]:
            K[slots[t] // P, :, slots[t] % P] = k[t]
            V[slots[t] // P, :, slots[t] % P] = v[t]
    assert torch.equal(cache.K, K) and torch.equal(cache.V, V)
    assert cache.check_device_error() == 0


def test_append_slot_past_the_pool_is_skipped():
    cache = small_cache(16, 4)
    cache.K.zero_(), cache.V.zero_()
    x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    cache.append(x, x, torch.tensor([64, 2 ** 40, 5], device="cuda"))
    assert cache.K.sum().item() == 2 * 64 and cache.check_device_error() == 1


@pytest.mark.parametrize("dtype,d,heads,P", [("bf16", 128, 8, 16), ("f16", 64, 3, 128), ("f32", 64, 1, 32)])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("lens,n", [([1], 1), ([130, 0, 300], 129), ([700, 64, 65], 700)])
def test_gather(dtype, d, heads, P, layout, lens, n):
    c = Case(lens, [0] * len(lens), H=heads, G=1, d=d, P=P, dtype=dtype, seed=n, width=-(-n // P) + 1)
    cache = cache_of(c, layout)
    K, V = cache.gather(dev(c.table), dev(lens), n)
    assert np.array_equal(K.double().cpu().numpy(), op.gather(c.K, c.table, lens, n, P))
    assert np.array_equal(V.double().cpu().numpy(), op.gather(c.V, c.table, lens, n, P))
    assert cache.check_device_error() == 0


def test_gather_bad_pages_read_as_zero():
    c = Case([40], [0], H=1, G=1, d=64)
    cache = cache_of(c)
    table = c.table.copy()
    table[0, 1] = c.pages
    K, _ = cache.gather(dev(table), dev([40]), 40)
    want = op.gather(c.K, c.table, [40], 40, 16)
    want[:, :, 16:32] = 0
    assert np.array_equal(K.double().cpu().numpy(), want)
    assert cache.check_device_error() == 1


# ---------------------------------------------------------------------------
# Attention
# ---------------------------------------------------------------------------
DECODE = [([1], [1]), ([16, 17, 15, 300], [1, 1, 1, 1]), ([2049], [1]), ([5, 0, 900], [1, 0, 1])]
FEW = [([40, 7], [2, 4]), ([513], [3]), ([4, 129, 130], [4, 3, 2])]
CHUNKS = [([70], [70]), ([130, 1, 260, 64], [130, 1, 5, 64]), ([700], [33]), ([300, 0, 1000], [257, 0, 40])]


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("bf16", 64), ("f16", 128), ("f16", 64), ("f32", 128), ("f32", 64)])
@pytest.mark.parametrize("G,P", [(1, 16), (2, 128), (4, 16), (8, 32), (4, 256)])
@pytest.mark.parametrize("lens,new", DECODE + FEW + CHUNKS)
def test_attend(dtype, d, G, P, lens, new):
    c = Case(lens, new, H=2, G=G, d=d, P=P, dtype=dtype, seed=len(lens) + G, poison=np.nan, pad_rows=2)
    got = call(c, pad_value=3.25)
    check(c, got, c.want())
    assert (got[0][int(c.cu[-1]):] == 3.25).all() and (got[1][int(c.cu[-1]):] == 7.0).all()


MASKS = [
    dict(window=1), dict(window=20), dict(full=True), dict(full=True, window=50), dict(prefix="half"),
    dict(first_key="documents"), dict(first_key="nothing"), dict(softcap=15.0), dict(slopes="usual"),
    dict(slopes="usual", prefix="half", softcap=30.0), dict(window=40, first_key="documents", prefix="half"),
    dict(scale=0.02), dict(scale=-0.3, softcap=2.0), dict(softcap=1e-3), dict(softcap=1e4, slopes="usual"),
]


def masked(c, m):
    m = dict(m)
    r = np.random.default_rng(5)
    pos = np.concatenate([np.arange(n - q, n) for n, q in zip(c.lens, c.new)] + [np.zeros(c.rows - int(c.cu[-1]))])
    if m.get("prefix"):
        m["prefix"] = [n // 2 for n in c.lens]
    kind = m.get("first_key")
    if kind == "documents":
        m["first_key"] = (pos // 37 * 37).astype(int)
    elif kind == "nothing":                                   # a third of the rows see no key at all
        m["first_key"] = np.where(r.random(c.rows) < 0.33, pos + 1, np.maximum(pos - 9, 0)).astype(int)
    if m.get("slopes"):
        m["slopes"] = 2.0 ** (-8.0 * (np.arange(c.H * c.G) + 1) / (c.H * c.G))
    return m


@pytest.mark.parametrize("dtype,d", [("bf16", 128), ("f16", 64), ("f32", 64)])
@pytest.mark.parametrize("G,P", [(1, 32), (4, 16), (8, 128)])
@pytest.mark.parametrize("lens,new", [([300, 16, 1], [1, 1, 1]), ([200, 40], [3, 4]), ([400, 150, 20], [150, 150, 1])])
@pytest.mark.parametrize("m", MASKS, ids=lambda m: "-".join(m))
def test_masks(dtype, d, G, P, lens, new, m):
    c = Case(lens, new, H=2, G=G, d=d, P=P, dtype=dtype, seed=3, poison=np.inf)
    m = masked(c, m)
    check(c, call(c, **m), c.want(**m), m.get("softcap", 0.0))


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("lens,new", [([300], [1]), ([300], [4]), ([300], [200])])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf, "lowest"])
def test_masked_keys_may_hold_anything(dtype, lens, new, bad):
    """Keys that some rows see and others do not: the rows that do not are exact, whatever the keys hold."""
    c = Case(lens, new, H=2, G=4, d=64, P=16, dtype=dtype, seed=8)
    bad = torch.finfo(TDT[dtype]).min if bad == "lowest" else bad
    hidden = list(range(120, 140)) + [299]                    # 299: the last row's own key
    first = np.where(np.arange(c.rows) < c.rows - 1, 140, 141)
    want = c.want(first_key=first)
    for j in hidden:
        page, row = c.at(0, j)
        c.K[page, :, row] = bad
        c.V[page, :, row] = bad
    got = call(c, first_key=first)
    T = c.rows - 1                                            # all but the row that sees the last key
    if T == 0:
        return
    tol, _ = bounds(c, want[2], want[0], want[1])
    pos = np.arange(300 - c.rows, 300)
    rows = [i for i in range(T) if pos[i] >= 140 or pos[i] < 120]
    assert (np.abs(got[0][rows] - want[0][rows]) <= tol[rows]).all()
    none = [i for i in range(T) if pos[i] < 140]
    assert (got[0][none] == 0).all() and (got[1][none] == -np.inf).all()


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("new", [1, 4, 100])
@pytest.mark.parametrize("qscale", [4.0, 100.0])
def test_sharp_softmax(dtype, new, qscale):
    c = Case([600], [new], H=1, G=4, d=128, dtype=dtype, seed=4, qscale=qscale)
    check(c, call(c), c.want())


@pytest.mark.parametrize("new", [1, 3, 90])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_layouts_and_strided_queries(layout, dtype, new):
    c = Case([333, 90], [new, min(new, 90)], H=3, G=2, d=64, P=64, dtype=dtype, seed=6)
    wide = torch.randn(c.rows, 2 * c.H * c.G, c.d + 64, device="cuda").to(TDT[dtype])
    q = wide[:, ::2, :c.d]
    q.copy_(dev(c.Q, dtype))
    check(c, call(c, cache=cache_of(c, layout), q=q), c.want())


@pytest.mark.parametrize("B,Hkv,G,n,new", [(9, 2, 4, 4100, 1), (1, 1, 8, 20000, 1), (3, 2, 4, 6000, 2), (2, 1, 4, 9000, 65),
                                           (1, 1, 1, 3000, 1500), (70, 1, 2, 130, 1)])
def test_long_and_split(B, Hkv, G, n, new):
    """Lengths and batches at which the keys of a row are shared out and joined, ragged."""
    r = np.random.default_rng(n)
    lens = [int(x) for x in r.integers(max(n // 4, new), n + 1, B)]
    c = Case(lens, [new] * B, H=Hkv, G=G, d=128, P=32, dtype="bf16", seed=n)
    check(c, call(c), c.want())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,most", [(700, 1), (1500, 1), (1500, 40), (600, 3)])
def test_many_requests(B, most, dtype):
    """More requests than a block lists itself, and than one round of the list takes; some without rows."""
    r = np.random.default_rng(B + most)
    lens = [int(x) for x in r.integers(0, 60, B)]
    new = [int(min(n, x)) for n, x in zip(lens, r.integers(0, most + 1, B))]
    c = Case(lens, new, H=1, G=1, d=64, P=16, dtype=dtype, seed=B, width=600)
    check(c, call(c), c.want())


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("P", [16, 32, 128])
@pytest.mark.parametrize("window,lens,new", [(20, [700, 333], [1, 1]), (50, [900, 161], [6, 4]), (37, [1500, 700], [40, 90]),
                                             (300, [1500, 700], [1, 200])])
def test_pages_before_the_window_may_be_given_away(dtype, P, window, lens, new):
    c = Case(lens, new, H=2, G=4, d=64, P=P, dtype=dtype, seed=window, poison=np.nan)
    want = c.want(window=window)
    for b, (n, q) in enumerate(zip(lens, new)):
        gone = max(0, n - q - window + 1) // P               # pages that no row sees a key of
        c.table[b, :gone] = -9
    check(c, call(c, window=window), want)


def test_strides_of_single_rows_and_heads_mean_nothing():
    c = Case([100], [1], H=1, G=1, d=64, P=16, dtype="bf16", seed=3)
    cache = cache_of(c)
    q = dev(c.Q, "bf16").as_strided((1, 1, 64), (3, 5, 1))
    out = torch.empty(64, dtype=torch.bfloat16, device="cuda").as_strided((1, 1, 64), (1, 7, 1))
    cache.attend(q, dev(c.table), dev(c.lens), dev(c.cu), out=out)
    O, lse, info = c.want()
    assert (np.abs(out.double().cpu().numpy() - O) <= bounds(c, info, O, lse)[0]).all()
    cache.append(q, q, torch.tensor([5], device="cuda"))
    assert torch.equal(cache.K[0, 0, 5], q[0, 0]) and cache.check_device_error() == 0


def test_shared_pages():
    """Two requests whose tables begin with the same pages."""
    c = Case([64, 80], [1, 20], H=2, G=2, d=64, dtype="bf16", seed=12)
    c.table[1, :3] = c.table[0, :3]
    check(c, call(c), c.want())


def test_bad_tables_lengths_and_offsets_set_the_error_word():
    c = Case([50, 50], [1, 1], H=1, G=1, d=64)
    cache = cache_of(c)
    q, t, lens, cu = dev(c.Q, "bf16"), dev(c.table), dev(c.lens), dev(c.cu)
    for kw in (dict(t=[[0, 1, c.pages, 2], [0, -1, 1, 2]]), dict(lens=[50, 1 << 20]), dict(lens=[-3, 50]),
               dict(cu=[0, 1, 99]), dict(cu=[-1, 1, 2]), dict(cu=[0, 2, 1])):
        cache.attend(q, dev(kw["t"]) if "t" in kw else t, dev(kw.get("lens", c.lens)), dev(kw.get("cu", c.cu)))
        assert cache.check_device_error() & 1, kw
    cache.attend(q, t, lens, dev([0, 2, 2]), max_new=1)
    assert cache.check_device_error() == 8
    cache.attend(q, t, lens, cu)
    assert cache.check_device_error() == 0


@pytest.mark.parametrize("new", [1, 40])
def test_streams_graphs_and_two_calls_at_once(new):
    """On a side stream, captured and replayed with other lengths, and two calls of one cache side by side."""
    c = Case([900, 640], [new, new], H=2, G=4, d=128, dtype="bf16", seed=2)
    cache = cache_of(c)
    q, t, lens, cu = dev(c.Q, "bf16"), dev(c.table), dev(c.lens), dev(c.cu)
    ref = cache.attend(q, t, lens, cu, max_new=new)
    torch.cuda.synchronize()
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [cache.attend(q, t, lens, cu, max_new=new, stream=s) for s in (a, b) for _ in range(10)]
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) for o in outs)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            o = cache.attend(q, t, lens, cu, max_new=new)
        graphs.append((g, o))
    for shorter in (0, 333):
        lens.copy_(dev([900 - shorter, 640 - shorter]))
        want = cache.attend(q, t, lens, cu, max_new=new)
        torch.cuda.synchronize()
        for s, (g, _) in zip((a, b), graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for _, o in graphs)
    assert cache.check_device_error() == 0


def test_refusals():
    c = Case([50], [2], H=2, G=2, d=64)
    cache = cache_of(c)
    q, t, lens, cu = dev(c.Q, "bf16"), dev(c.table), dev(c.lens), dev(c.cu)
    for bad in (dict(Q=q.float()), dict(Q=q[:, :3]), dict(Q=q[..., :32]), dict(Q=q.cpu()), dict(table=t.long()), dict(lens=lens.long()),
                dict(cu=cu[:1]), dict(table=t.cpu()), dict(slopes=torch.ones(3, device="cuda")),
                dict(prefix=torch.ones(2, dtype=torch.int32, device="cuda")),
                dict(first_key=torch.ones(3, dtype=torch.int32, device="cuda")), dict(out=q[:1]),
                dict(table=t.expand(3, t.shape[1]), lens=lens.expand(3).contiguous(), cu=dev([0, 0, 1, 2])),
                dict(lse=torch.ones(2, 4, dtype=torch.float16, device="cuda")), dict(Q=q.transpose(1, 2).contiguous().transpose(1, 2))):
        with pytest.raises(ValueError):
            cache.attend(**{**dict(Q=q, table=t, lens=lens, cu=cu), **bad})
    for bad in (dict(scale=float("nan")), dict(softcap=-1.0), dict(window=-1), dict(softcap=float("inf"))):
        with pytest.raises(MpError) as e:
            cache.attend(q, t, lens, cu, **bad)
        assert e.value.status == L.MP_EINVAL
    with pytest.raises(MpError) as e:                         # rows of the output on one another
        cache.attend(q, t, lens, cu, out=q[:1].expand(2, 4, 64))
    assert e.value.status == L.MP_EINVAL
    with pytest.raises(MpError) as e:                         # 3 query heads per KV head
        cache.attend(torch.zeros(2, 6, 64, dtype=torch.bfloat16, device="cuda"), t, lens, cu)
    assert e.value.status == L.MP_EUNSUPPORTED
    off = torch.zeros(2 * 4 * 64 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(2, 4, 64)
    with pytest.raises(MpError) as e:                         # rows that do not start on 16 bytes
        cache.attend(off, t, lens, cu)
    assert e.value.status == L.MP_EINVAL
    with pytest.raises(MpError) as e:
        cache.gather(t, lens, t.shape[1] * 16 + 1)
    assert e.value.status == L.MP_EINVAL
    with pytest.raises(ValueError):
        cache.append(q[:, :2], q[:, :2], torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        cache.plan(lens, lens, t, t[0], lens)                 # neither rows nor out
    for kw, status in ((dict(head_dim=96), L.MP_EUNSUPPORTED), (dict(page_tokens=8), L.MP_EUNSUPPORTED),
                       (dict(page_tokens=48), L.MP_EUNSUPPORTED), (dict(page_tokens=512), L.MP_EUNSUPPORTED)):
        with pytest.raises(MpError) as e:
            PagedCache(**{**dict(kv_heads=1, head_dim=64, num_pages=2, page_tokens=16), **kw})
        assert e.value.status == status


def test_empty_calls():
    c = Case([20], [1], H=1, G=1, d=64)
    cache = cache_of(c)
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")
    q = dev(c.Q, "bf16")
    assert cache.attend(q[:0], i32(1, 2), i32(1), i32(2)).shape == (0, 1, 64)
    out = torch.full_like(q, 2.0)
    cache.attend(q, i32(0, 2), i32(0), i32(1), out=out)
    assert (out == 2.0).all()
    out = cache.attend(q, i32(1, 0), i32(1), dev([0, 1]))      # a table without columns: nothing is cached
    assert (out == 0).all()
    assert cache.gather(i32(0, 2), i32(0), 5)[0].shape == (0, 1, 5, 64)
    assert cache.gather(i32(2, 2), i32(2), 0)[0].shape == (2, 1, 0, 64)
    cache.append(q[:0], q[:0], torch.zeros(0, dtype=torch.int64, device="cuda"))
    assert cache.check_device_error() == 0


# ---------------------------------------------------------------------------
# Together: prompts in chunks, decode steps, then the clustering
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype,d,P", [("bf16", 128, 16), ("f32", 64, 32)])
def test_prompts_in_chunks_decode_steps_and_clustering(dtype, d, P):
    Hkv, G, B, pages = 2, 4, 2, 60
    r = torch.Generator(device="cuda").manual_seed(9)
    cache = PagedCache(Hkv, d, pages, P, dtype)
    cache.K.fill_(float("nan")), cache.V.fill_(float("nan"))
    lens, count = dev([0, 0]), dev([pages])
    table, free = dev(np.full((B, 24), -1)), dev(np.random.default_rng(1).permutation(pages))
    draw = lambda n, h: torch.randn(n, h, d, generator=r, device="cuda").to(TDT[dtype])
    kept = [[], []]
    for new in ([100, 30], [90, 0], [1, 170], [1, 1], [8, 0]) + ([1, 1],) * 3:
        T = sum(new)
        plan = cache.plan(lens, dev(new), table, free, count, rows=T)
        lens, count = plan.lens, plan.free_count
        q, k, v = draw(T, Hkv * G), draw(T, Hkv), draw(T, Hkv)
        cache.append(k, v, plan.slots)
        out = cache.attend(q, table, lens, plan.cu, max_new=max(new))
        at = 0
        for b, n in enumerate(new):
            kept[b].append((k[at:at + n], v[at:at + n]))
            K, V = (torch.cat(x).double().cpu().numpy() for x in zip(*kept[b]))
            for i in range(n):
                m = len(K) - n + i + 1
                for h in range(Hkv * G):
                    z = K[:m, h // G] @ q[at + i, h].double().cpu().numpy() / d ** 0.5
                    w = np.exp(z - z.max())
                    o = w @ V[:m, h // G] / w.sum()
                    assert np.abs(out[at + i, h].double().cpu().numpy() - o).max() <= H.TOL[dtype]
            at += n
    assert lens.tolist() == [203, 204] and cache.check_device_error() == 0
    # the first 203 tokens of both, clustered; with the whole budget the decode is the dense attention of single tokens
    cfg = Config(batch=B, kv_heads=Hkv, q_heads=Hkv * G, head_dim=d, max_tokens=256, block_tokens=256, kmeans_iters=2,
                 dtype=dtype)
    idx = MultipoleIndex(cfg)
    idx.build_paged(cache, table, lens, 203)
    q = draw(B, Hkv * G)
    O = idx.decode(q, budget=1000)
    paged = cache.attend(q, table, dev([203, 203]), dev([0, 1, 2]), max_new=1)
    assert (O.float() - paged.float()).abs().max().item() <= 2 * H.TOL[dtype]
    assert idx.check_device_error() == 0 and cache.check_device_error() == 0
    with pytest.raises(MpError) as e:
        idx.build_paged(cache, table, lens, 257)
    assert e.value.status == L.MP_ENOSPC
    with pytest.raises(ValueError):
        idx.build_paged(cache, table[:1], lens[:1], 10)


def test_offsets_past_32_bits():
    """A pool whose pages lie more than 2^32 elements apart from its first."""
    P, d, pages = 256, 128, 33000                             # times 4 heads: 4.3e9 elements in K and in V
    K = torch.zeros(pages, 4, P, d, dtype=torch.bfloat16, device="cuda")
    cache = PagedCache(4, d, pages, P, "bf16", K=K, V=torch.zeros_like(K))
    c = Case([300, 300], [1, 40], H=4, G=4, d=d, P=P, dtype="bf16", seed=1, spare=0)
    far = np.array([pages - 1, pages - 2, pages - 3, pages - 5])
    K[torch.from_numpy(far).cuda()] = dev(c.K, "bf16")
    cache.V[torch.from_numpy(far).cuda()] = dev(c.V, "bf16")
    table = dev(far[c.table])
    out = cache.attend(dev(c.Q, "bf16"), table, dev(c.lens), dev(c.cu), max_new=40)
    O, lse, info = c.want()
    tol, _ = bounds(c, info, O, lse)
    assert (np.abs(out.double().cpu().numpy() - O) <= tol).all()
    one = cache.attend(dev(c.Q, "bf16")[:1], table[:1], dev([300]), dev([0, 1]), max_new=1)
    assert (np.abs(one.double().cpu().numpy() - O[:1]) <= tol[:1]).all()
    x = torch.ones(1, 4, d, dtype=torch.bfloat16, device="cuda")
    cache.append(x, x, torch.tensor([(pages - 3) * P - 2], device="cuda"))   # a page of neither request
    assert (K[pages - 4, :, P - 2] == 1).all()
    got, _ = cache.gather(table, dev([300, 300]), 300)
    assert np.array_equal(got.double().cpu().numpy(), op.gather(c.K, c.table, [300, 300], 300, P))
