"""Inputs, marshalling and error bounds of the paged-cache tests."""
import numpy as np
import torch

from oracle import paged as op

TDT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
U = {k: torch.finfo(v).eps / 2 for k, v in TDT.items()}     # half a step: the most that one rounding is off


def rounded(x, dtype):
    """float64 values of x rounded to dtype."""
    return torch.from_numpy(np.ascontiguousarray(x)).to(TDT[dtype]).double().numpy()


class Case:
    """A paged cache with requests of `lens` tokens whose last `new` are the step's rows, on the host in 64 bits."""

    def __init__(self, lens, new, H=2, G=4, d=128, P=16, dtype="bf16", seed=0, spare=3, width=None, poison=None,
                 pad_rows=0, qscale=1.0):
        r = np.random.default_rng(seed)
        self.lens, self.new, self.H, self.G, self.d, self.P, self.dtype = lens, new, H, G, d, P, dtype
        need = [-(-n // P) for n in lens]
        self.pages = sum(need) + spare
        ids = r.permutation(self.pages)
        W = max([width or 1] + need)
        self.table = np.full((len(lens), W), -7)             # entries that no call may follow
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = ids[at:at + m]
            at += m
        self.cu = np.concatenate([[0], np.cumsum(new)]).astype(int)
        self.rows = int(self.cu[-1]) + pad_rows
        self.Q = rounded(qscale * r.standard_normal((self.rows, H * G, d)), dtype)
        self.K = rounded(r.standard_normal((self.pages, H, P, d)), dtype)
        self.V = rounded(r.standard_normal((self.pages, H, P, d)), dtype)
        if poison is not None:                               # every row that no request holds
            held = np.zeros((self.pages, P), bool)
            for b, m in enumerate(lens):
                j = np.arange(m)
                held[self.table[b, j // P], j % P] = True
            for X in (self.K, self.V):
                X.transpose(0, 2, 1, 3)[~held] = poison

    def at(self, b, j):
        """Page and row of token j of request b."""
        return self.table[b, j // self.P], j % self.P

    def want(self, **kw):
        return op.attend(self.Q, self.K, self.V, self.table, self.lens, self.cu, self.P, **kw)


def dev(x, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(x))
    return (t.to(TDT[dtype]) if dtype else t.int()).cuda()


def cache_of(c, layout="hptd"):
    """A PagedCache with the case's K and V, in one of several memory layouts."""
    from clustered_sparse_decode_b200 import PagedCache
    K, V = dev(c.K, c.dtype), dev(c.V, c.dtype)
    if layout == "token_major":                              # [pages, P, H, d] in memory
        K, V = (x.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3) for x in (K, V))
    elif layout == "joined":                                 # [pages, 2, H, P, d] in memory
        KV = torch.stack([K, V], 1).contiguous()
        K, V = KV[:, 0], KV[:, 1]
    elif layout == "head_major":                             # [H, pages, P, d] in memory
        K, V = (x.permute(1, 0, 2, 3).contiguous().permute(1, 0, 2, 3) for x in (K, V))
    return PagedCache(c.H, c.d, c.pages, c.P, c.dtype, K=K, V=V)


def call(c, cache=None, pad_value=None, max_new=None, lse=True, q=None, **kw):
    """(O, lse) of attend() on the case, as 64-bit arrays; rows behind the last hold pad_value before the call."""
    cache = cache or cache_of(c)
    q = dev(c.Q, c.dtype) if q is None else q
    out = torch.full((c.rows, c.H * c.G, c.d), float("nan") if pad_value is None else pad_value, dtype=TDT[c.dtype],
                     device="cuda")
    ls = torch.full((c.rows, c.H * c.G), 7.0, device="cuda") if lse else None
    for k, f in (("slopes", "f32"), ("prefix", None), ("first_key", None)):
        if kw.get(k) is not None:
            kw[k] = dev(np.asarray(kw[k]), f)
    cache.attend(q, dev(c.table), dev(c.lens), dev(c.cu), max_new=max(c.new) if max_new is None else max_new, out=out,
                 lse=ls, **kw)
    torch.cuda.synchronize()
    assert cache.check_device_error() == 0
    return out.double().cpu().numpy(), ls.double().cpu().numpy() if lse else None


def bounds(c, info, O, lse, softcap=0.0):
    """Largest deviation of O and of lse by arithmetic.

    A score: products exact in fp32's double width, d additions of at most 2^-22
    of the sum of magnitudes each (tensor cores may truncate), a few roundings of
    z itself (scaling, cap, bias, base 2), the cap's tanh to some 2^-21 of the cap.
    A weight e^(z - m): the score's deviation, the exponential's 2^-21, and the
    rounding u of the weights to the values' type.  Sums over the keys add at most
    2^-22 of the sum of magnitudes per 8 keys and per joined part.  The result is
    rounded once more.
    """
    u, n = U[c.dtype], max(max(c.lens, default=0), 1)
    dz = 2.0 ** -22 * (c.d * info["zabs"] + 8 * info["zmax"] + 8 * softcap) + 2.0 ** -21
    acc = 2.0 ** -22 * (n / 8 + 256)
    rel = 2 * dz + acc + (2 * u if c.dtype != "f32" else 0.0)
    small = 2.0 ** -24 if c.dtype == "f16" else 0.0          # f16's own smallest steps, once for the weights, once for O
    tol = rel[..., None] * info["amp"] * 1.01 + u * np.abs(O) + small * (1 + info["amp"]) + 1e-30
    return tol, dz + acc + 2.0 ** -22 * np.abs(np.where(np.isfinite(lse), lse, 0.0))


def check(c, got, want, softcap=0.0):
    O, lse, info = want
    tol, ltol = bounds(c, info, O, lse, softcap)
    T = int(c.cu[-1])
    g, gl = got
    assert np.isfinite(g[:T]).all()
    off = np.abs(g[:T] - O[:T]) / tol[:T]
    assert off.size == 0 or off.max() <= 1, f"{off.max():.3g} of the bound at {np.unravel_index(off.argmax(), off.shape)}"
    if gl is not None:
        none = np.isinf(lse[:T])
        assert (gl[:T][none] == -np.inf).all()
        assert (np.abs(gl[:T][~none] - lse[:T][~none]) <= ltol[:T][~none]).all()
