"""Python binding of the paged cache: step addresses, appending, attention, gathering.

Marshalling only, as in api.py: torch allocates the memory and supplies the
stream, the library's CUDA kernels do the rest.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib as L

_DT = {"bf16": (L.MP_BF16, torch.bfloat16), "f16": (L.MP_F16, torch.float16), "f32": (L.MP_F32, torch.float32)}


@dataclass
class PagedPlan:
    """A step's addresses (mp_paged_plan): device tensors, reusable as the next call's `out`."""
    lens: torch.Tensor          # int32 [B]: tokens of each request, the new ones among them
    cu: torch.Tensor            # int32 [B + 1]: first row of each request
    slots: torch.Tensor         # int64 [rows]: slot of each row, -1 behind the last
    positions: torch.Tensor     # int32 [rows]: position of each row, 0 behind the last
    free_count: torch.Tensor    # int32 [1]: free pages left


class PagedCache:
    """Keys and values of many requests in pages of one pool (one attention layer).

    K, V: [num_pages, kv_heads, page_tokens, head_dim] on the device, allocated
    when absent.  Views with any order of the first three axes are taken as they
    are (equal strides for both, the last axis contiguous, 16-byte multiples),
    so that a pool of another layout is passed as its permuted view.  The error
    word is cleared on the current stream: calls on another one come after it.
    """

    def __init__(self, kv_heads, head_dim, num_pages, page_tokens, dtype="bf16", K=None, V=None, device=None):
        self.lib = L.load()
        code, self.torch_dtype = _DT[dtype]
        want = (num_pages, kv_heads, page_tokens, head_dim)
        if (K is None) != (V is None):
            raise ValueError("K and V come together")
        if K is None:
            device = torch.device(device) if device is not None else torch.device("cuda", torch.cuda.current_device())
            K, V = (torch.empty(want, dtype=self.torch_dtype, device=device) for _ in range(2))
        for t in (K, V):
            if tuple(t.shape) != want or t.dtype != self.torch_dtype or t.device.type != "cuda" or t.device != K.device:
                raise ValueError(f"K and V must be {self.torch_dtype} device tensors of shape {want}")
            if t.stride(3) != 1 or any(n > 1 and a != b for n, a, b in zip(want, t.stride(), K.stride())):
                raise ValueError("K and V need equal strides and contiguous rows")
        if device is not None and torch.device(device) not in (K.device, torch.device("cuda")):
            raise ValueError(f"K and V are on {K.device}")
        self.K, self.V, self.device = K, V, K.device
        self.kv_heads, self.head_dim, self.num_pages, self.page_tokens = kv_heads, head_dim, num_pages, page_tokens
        c = L.MpPagedConfig(kv_heads=kv_heads, head_dim=head_dim, num_pages=num_pages, page_tokens=page_tokens,
                            dtype=code)
        # the stride of an axis of length 1 is torch's to choose: the contiguous one then
        row = head_dim
        c.token_stride = K.stride(2) if page_tokens > 1 else row
        c.head_stride = K.stride(1) if kv_heads > 1 else max(row, K.stride(2) * page_tokens)
        c.page_stride = K.stride(0) if num_pages > 1 else max(row, K.stride(2) * page_tokens, c.head_stride * kv_heads)
        with torch.cuda.device(self.device):
            self._err = torch.zeros(1, dtype=torch.int32, device=self.device)
            self.h = L.MpPagedCache()
            L.check(self.lib.mp_paged_init(ctypes.byref(c), K.data_ptr(), V.data_ptr(), self._err.data_ptr(),
                                           ctypes.byref(self.h)), "mp_paged_init")
        self._h = ctypes.addressof(self.h)
        self._index = self.device.index

    # ------------------------------------------------------------------ helpers
    # A decode step's calls take a few microseconds each, most of them here: the
    # checks read each attribute once and compare plain integers.
    def _run(self, stream, name, f, *args):
        """The call on `stream` (default: the current one) with the cache's device current."""
        if stream is None and torch._C._cuda_getDevice() == self._index:
            st = f(*args, torch._C._cuda_getCurrentRawStream(self._index))
        else:
            if stream is not None and stream.device != self.device:
                raise ValueError(f"the stream belongs to {stream.device}, the cache to {self.device}")
            with torch.cuda.device(self.device):
                s = stream if stream is not None else torch.cuda.current_stream()
                st = f(*args, s.cuda_stream)
        if st != L.MP_OK:
            L.check(st, name)

    def _empty(self, stream, shape, dtype):
        """Device memory for a call on `stream`."""
        if stream is None:
            return torch.empty(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            return torch.empty(shape, dtype=dtype, device=self.device)

    def _ints(self, t, n, what, dtype=torch.int32):
        """The address of a contiguous vector of n integers."""
        if t.dtype is not dtype or t.numel() != n or t.dim() != 1 or t.get_device() != self._index or not t.is_contiguous():
            raise ValueError(f"{what} must be a contiguous {dtype} tensor of shape {(n,)} on {self.device}")
        return t.data_ptr()

    def _table(self, t):
        if t.dtype is not torch.int32 or t.dim() != 2 or t.get_device() != self._index:
            raise ValueError(f"the table must be an int32 tensor [requests, pages] on {self.device}")
        B, W = t.shape
        row, col = t.stride()
        if (W > 1 and col != 1) or (B > 1 and row < W):
            raise ValueError("the table's rows must be contiguous and apart from one another")
        return B, W, row if B > 1 else W

    def _rows(self, t, shape, what):
        """Address and strides of [rows, heads, head_dim] whose head rows are contiguous."""
        s = t.stride()
        if t.dtype is not self.torch_dtype or t.shape != shape or t.get_device() != self._index or s[2] != 1:
            raise ValueError(f"{what} must be a {self.torch_dtype} tensor of shape {tuple(shape)} on {self.device} "
                             "with contiguous head rows")
        return t.data_ptr(), s

    # ------------------------------------------------------------------ calls
    def new_plan(self, batch, rows):
        """Buffers of plan(out=...) for `batch` requests and `rows` rows."""
        i32 = dict(dtype=torch.int32, device=self.device)
        return PagedPlan(torch.empty(batch, **i32), torch.empty(batch + 1, **i32),
                         torch.empty(rows, dtype=torch.int64, device=self.device), torch.empty(rows, **i32),
                         torch.empty(1, **i32))

    def plan(self, lens, new_tokens, table, free_pages, free_count, rows=None, out=None, stream=None):
        """The addresses of a step (mp_paged_plan): pages for new_tokens[b] tokens of request b behind lens[b].

        lens, new_tokens: int32 [B]; table: int32 [B, W], new pages are written to
        it; free_pages: int32, a stack of free ids of which free_count (int32 [1])
        are valid.  rows: rows of the step, at least the new tokens' sum (or
        out's).  out's lens and free_count may be the given ones: a captured step
        then advances them at each replay.
        """
        B, W, stride = self._table(table)
        if out is None:
            if rows is None:
                raise ValueError("plan needs rows or out")
            if stream is None:
                out = self.new_plan(B, rows)
            else:
                with torch.cuda.stream(stream):
                    out = self.new_plan(B, rows)
        T, F = out.slots.numel(), free_pages.numel()
        args = L.PLAN_ARGS.pack(
            B, W, stride, T, F, 0, self._ints(lens, B, "lens"), self._ints(new_tokens, B, "new_tokens"), table.data_ptr(),
            self._ints(free_pages, F, "free_pages"), self._ints(free_count, 1, "free_count"),
            self._ints(out.lens, B, "out.lens"), self._ints(out.cu, B + 1, "out.cu"),
            self._ints(out.slots, T, "out.slots", torch.int64), self._ints(out.positions, T, "out.positions"),
            self._ints(out.free_count, 1, "out.free_count"))
        self._run(stream, "mp_paged_plan", self.lib.mp_paged_plan, self._h, args)
        return out

    def append(self, K_new, V_new, slots, stream=None):
        """Write rows K_new, V_new [rows, kv_heads, head_dim] to their slots (mp_paged_append); slot -1 is skipped."""
        T = slots.numel()
        shape = (T, self.kv_heads, self.head_dim)
        k, ks = self._rows(K_new, shape, "K_new")
        v, vs = self._rows(V_new, shape, "V_new")
        if ks != vs and ((T > 1 and ks[0] != vs[0]) or (self.kv_heads > 1 and ks[1] != vs[1])):
            raise ValueError("K_new and V_new need equal strides")     # (an axis of length 1 has none that counts)
        self._run(stream, "mp_paged_append", self.lib.mp_paged_append, self._h, k, v, ks[0], ks[1],
                  self._ints(slots, T, "slots", torch.int64), T)

    def attend(self, Q, table, lens, cu, max_new=None, scale=0.0, softcap=0.0, window=0, full=False, slopes=None,
               prefix=None, first_key=None, out=None, lse=None, scratch=None, stream=None):
        """Attention of the rows Q [rows, Hq, d] over their requests' cached keys (mp_paged_attend).

        Request b's rows are cu[b] .. cu[b + 1] and hold its last tokens of the
        lens[b] that the cache has (append before attending).  A row sees the keys
        up to its own position, or up to prefix[b] where that is further (all with
        full=True); of these only the last `window` positions (0: all) and none
        before first_key[row].  Scores are scale * q.k, capped by softcap *
        tanh(z / softcap), minus slopes[head] * |position - key|.  max_new: most
        rows that a request has (a bound known to the host; it chooses the
        kernel).  Returns O [rows, Hq, d]; rows behind cu[B] are left as they are;
        out must not overlap Q.  lse: float32 [rows, Hq] that receives the log of
        each row's sum, -inf where it sees nothing.
        """
        if Q.dim() != 3:
            raise ValueError("Q must be [rows, heads, head_dim]")
        T, Hq, _ = Q.shape
        B, W, stride = self._table(table)
        q, qs = self._rows(Q, (T, Hq, self.head_dim), "Q")
        if Hq % self.kv_heads:
            raise ValueError(f"{Hq} query heads over {self.kv_heads} KV heads")
        if out is None:
            if stream is None:
                out = torch.empty_like(Q)
            else:
                out = self._empty(stream, Q.shape, self.torch_dtype)
            o, os = out.data_ptr(), out.stride()
        else:
            o, os = self._rows(out, Q.shape, "out")
        if lse is not None and (lse.dtype is not torch.float32 or lse.shape != (T, Hq) or not lse.is_contiguous()
                                or lse.get_device() != self._index):
            raise ValueError(f"lse must be a contiguous float32 tensor of shape {(T, Hq)} on {self.device}")
        args = L.ATTEND_ARGS.pack(
            B, Hq, T, 0 if max_new is None else min(max_new, T), W, stride, table.data_ptr(),
            self._ints(lens, B, "lens"), self._ints(cu, B + 1, "cu"), q, o, qs[0], qs[1], os[0], os[1],
            scale, softcap, window, L.MP_ATTEND_FULL if full else 0,
            self._ints(slopes, Hq, "slopes", torch.float32) if slopes is not None else 0,
            self._ints(prefix, B, "prefix") if prefix is not None else 0,
            self._ints(first_key, T, "first_key") if first_key is not None else 0,
            lse.data_ptr() if lse is not None else 0)
        need = ctypes.c_size_t()
        L.check(self.lib.mp_paged_attend_scratch(self._h, args, ctypes.byref(need)), "mp_paged_attend_scratch")
        need = need.value
        if scratch is not None:
            s, n = self._ints(scratch, scratch.numel(), "scratch", torch.uint8), scratch.numel()
        elif need:
            scratch = self._empty(stream, (need,), torch.uint8)
            s, n = scratch.data_ptr(), need
        else:
            s = n = 0
        self._run(stream, "mp_paged_attend", self.lib.mp_paged_attend, self._h, args, s, n)
        return out

    def gather(self, table, lens, n, out=None, stream=None, whole=False):
        """The first n tokens of every request as K, V [B, kv_heads, n, head_dim] (mp_paged_gather).

        The layout that MultipoleIndex.build and dense_decode take; rows from
        lens[b] on are zero.  whole: every request has to hold n tokens, a
        shorter one sets the cache's error word (mp_paged_gather_whole).  out:
        (K, V) to write to.
        """
        B, W, stride = self._table(table)
        shape = (B, self.kv_heads, n, self.head_dim)
        if out is None:
            K = self._empty(stream, shape, self.torch_dtype)
            V = torch.empty_like(K) if stream is None else self._empty(stream, shape, self.torch_dtype)
        else:
            K, V = out
            for t in (K, V):
                if t.shape != shape or t.dtype is not self.torch_dtype or t.device != self.device or not t.is_contiguous():
                    raise ValueError(f"out must be contiguous {self.torch_dtype} tensors of shape {shape} on {self.device}")
        f = self.lib.mp_paged_gather_whole if whole else self.lib.mp_paged_gather
        self._run(stream, f.__name__, f, self._h, B, table.data_ptr(), W, stride,
                  self._ints(lens, B, "lens"), n, K.data_ptr(), V.data_ptr())
        return K, V

    def check_device_error(self, stream=None):
        """Synchronise and return the cache's error word (0 = none); clears it."""
        code = ctypes.c_int32(0)
        with torch.cuda.device(self.device):
            s = stream if stream is not None else torch.cuda.current_stream()
            st = self.lib.mp_paged_check_error(self._h, ctypes.byref(code), s.cuda_stream)
        if st not in (L.MP_OK, L.MP_EDEVICE):
            L.check(st, "mp_paged_check_error")
        return code.value
