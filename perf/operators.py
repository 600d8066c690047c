"""The paged-cache operators' cases: what is timed, on which inputs, and what they compute.

A paged key-value cache holds the keys and values of many requests in pages of
`page` tokens, [pages, kv heads, page, head_dim] each; a request's tokens lie in
the pages that its row of the block table lists.  Four operators work on it:

  plan     block tables, slot maps and offsets of a step, from the requests' lengths
  append   new keys and values written to their slots
  attend   the new tokens' attention over their requests' cached tokens
  gather   requests' tokens copied out into [batch, kv heads, n, head_dim]

`run` computes each in elementary torch operations; where `own` is true it makes
the framework's calls instead.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}


def attend_case(name=None, **kw):
    c = dict(op="attend", dtype="bf16", batch=1, kv_heads=8, group=4, d=128, page=16, past_lo=0, past_hi=0, new_lo=1,
             new_hi=1, ones=0.0, softcap=0.0, window=0, slopes=False, doc=0, prefix=0, mix=1)
    c.update(kw)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one decode step of 16 running requests: each gets one token, now and then a page
        dict(name="plan_decode_16", op="plan", batch=16, page=16, past_lo=16384, past_hi=32767, new_lo=1, new_hi=1, mix=11),
        # 256 prompts of ragged lengths admitted at once, some requests waiting with no token
        dict(name="plan_prompts_256", op="plan", batch=256, page=16, past_lo=0, past_hi=2000, new_lo=0, new_hi=2000,
             mix=12),
        # the decode step's 16 tokens written to their pages
        dict(name="append_decode_16", op="append", dtype="bf16", rows=16, kv_heads=8, d=128, page=16, mix=13),
        # a prompt chunk of 16K tokens written to scattered pages
        dict(name="append_prompt_16k", op="append", dtype="bf16", rows=16384, kv_heads=8, d=128, page=16, mix=14),
        # the tiny fp32 cache handed to the clustering
        dict(name="gather_tiny_f32", op="gather", dtype="f32", batch=1, kv_heads=1, d=64, page=16, n=2048, mix=15),
        # 16 requests of 32K tokens handed to the clustering
        dict(name="gather_16x32k", op="gather", dtype="bf16", batch=16, kv_heads=8, d=128, page=16, n=32768, mix=16),
        # the tiny fp32 configuration's single query over 2048 tokens: the latency of a call
        attend_case("attend_tiny_f32", dtype="f32", kv_heads=1, d=64, past_lo=2047, past_hi=2047, mix=17),
        # a decode step of 16 requests of 16K to 32K tokens
        attend_case("attend_decode_16x32k", batch=16, past_lo=16384, past_hi=32767, mix=18),
        # one long request's decode step, 64K tokens in larger pages
        attend_case("attend_decode_64k", dtype="f16", page=64, past_lo=65535, past_hi=65535, mix=19),
        # a prompt's chunk of 4K tokens over the 12K before it
        attend_case("attend_chunk_4k_16k", page=64, past_lo=12288, past_hi=12288, new_lo=4096, new_hi=4096, mix=20),
        # decode tokens and odd chunks of prompts in one batch, scores capped, a sliding window
        attend_case("attend_mixed", dtype="f16", batch=6, past_lo=1, past_hi=15000, new_lo=2, new_hi=600, ones=0.3,
                    softcap=30.0, window=4096, mix=21),
        # packed documents without shared heads, distance bias, a short prefix that all tokens see
        attend_case("attend_documents", batch=4, group=1, d=64, page=32, new_lo=1000, new_hi=4000, slopes=True, doc=500,
                    prefix=128, mix=22),
    ]


# What one drawn case may cost at most: the largest listed case's bytes and operations; the plain
# form's padded scores stay in memory; fp32 has no fast matrix product.
MOST_BYTES, MOST_FLOPS, MOST_FLOPS_F32, MOST_SCORES = 2.2e9, 9.5e11, 4e10, 2.0e9


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "gather", "attend", "attend", "attend"])
    mix = rng.randrange(1 << 30)
    page = rng.choice([16, 16, 32, 64, 128])
    if op == "plan":
        hi = _log(rng, 1, 2000)
        return dict(op=op, batch=_log(rng, 1, 256), page=page, past_lo=0, past_hi=_log(rng, 1, 32767),
                    new_lo=rng.choice([0, 1]), new_hi=hi, mix=mix)
    dtype, d = rng.choice(["bf16", "bf16", "f16", "f32"]), rng.choice([64, 128, 128])
    heads = rng.choice([1, 2, 3, 4, 8, 8])
    while True:
        if op == "append":
            c = dict(op=op, dtype=dtype, rows=_log(rng, 1, 16384), kv_heads=heads, d=d, page=page, mix=mix)
        elif op == "gather":
            c = dict(op=op, dtype=dtype, batch=_log(rng, 1, 16), kv_heads=heads, d=d, page=page, n=_log(rng, 1, 32768),
                     mix=mix)
        else:
            past = _log(rng, 1, 65536) - 1
            new = rng.choice([1, 1, rng.randint(2, 8), _log(rng, 2, 4096), _log(rng, 2, 4096)])
            c = attend_case(dtype=dtype, batch=_log(rng, 1, 32), kv_heads=heads, group=rng.choice([1, 2, 4, 4, 8]), d=d,
                            page=page, past_lo=rng.choice([0, past // 2, past]), past_hi=past,
                            new_lo=rng.choice([0, 1, new]), new_hi=new, ones=rng.choice([0.0, 0.0, 0.3]),
                            softcap=rng.choice([0.0, 0.0, 20.0, 50.0]),
                            window=rng.choice([0, 0, 0, _log(rng, 1, 8192)]), slopes=rng.random() < 0.25,
                            doc=rng.choice([0, 0, 0, _log(rng, 8, 4096)]),
                            prefix=rng.choice([0, 0, 0, _log(rng, 1, 2048)]), mix=mix)
            p, q = lengths(c)
            if not sum(q):
                continue
            cells = c["batch"] * c["kv_heads"] * max(a + b for a, b in zip(p, q))
            if cells * c["group"] * max(q) > MOST_SCORES or 2 * cells * d * BYTES[dtype] > MOST_BYTES:
                continue
            if work(c)["flops"] > (MOST_FLOPS_F32 if dtype == "f32" else MOST_FLOPS):
                continue
        if work(c)["bytes"] <= MOST_BYTES:
            return c


# ---------------------------------------------------------------------------
# A case's lengths and masks: of the case alone, not of the seed
# ---------------------------------------------------------------------------
def lengths(c):
    """(cached tokens, new tokens) of each request."""
    r = random.Random(c["mix"])
    past = [r.randint(c["past_lo"], c["past_hi"]) for _ in range(c["batch"])]
    new = [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["batch"])]
    if c.get("ones"):
        new = [1 if r.random() < c["ones"] else n for n in new]
    if c["op"] == "plan" and c["new_hi"] > 1:
        new = [0 if r.random() < 0.1 else n for n in new]
    return past, new


def masks(c):
    """Positions of all new tokens' rows, the first key each may see (documents), the requests' prefixes, as arrays."""
    past, new = lengths(c)
    r = random.Random(c["mix"] + 1)
    pos, first, prefix = [], [], []
    for p, n in zip(past, new):
        at = np.arange(p, p + n)
        pos.append(at)
        if c["doc"]:
            edges = [0]
            while edges[-1] < p + n:
                edges.append(edges[-1] + r.randint(1, 2 * c["doc"]))
            edges = np.array(edges)
            first.append(edges[np.searchsorted(edges, at, side="right") - 1])
        else:
            first.append(np.zeros(n, np.int64))
        prefix.append(min(p + n, r.randint(0, c["prefix"])) if c["prefix"] else 0)
    return np.concatenate(pos), np.concatenate(first), np.array(prefix)


def intervals(c):
    """The keys [lo, hi) that each new token's row sees, and the row's request."""
    _, new = lengths(c)
    pos, first, prefix = masks(c)
    req = np.repeat(np.arange(len(new)), new)
    hi = np.maximum(pos + 1, prefix[req])
    lo = np.maximum(first, pos - c["window"] + 1) if c["window"] else first
    return lo, hi, req


def work(c):
    if c["op"] == "plan":
        past, new = lengths(c)
        B, T = c["batch"], sum(new)
        pages = sum(-(-(p + n) // c["page"]) - -(-p // c["page"]) for p, n in zip(past, new))
        # lengths in and out, offsets, a slot and a position for each token, each new page's id from the pool to its table
        return {"bytes": 4 * (3 * B + 1) + 12 * T + 8 * pages + 8 + 4 * B, "flops": 0}
    row = c["kv_heads"] * c["d"] * BYTES[c["dtype"]]
    if c["op"] == "append":
        return {"bytes": 4 * c["rows"] * row + 8 * c["rows"], "flops": 0}
    if c["op"] == "gather":
        return {"bytes": 4 * c["batch"] * c["n"] * row + 4 * c["batch"] * -(-c["n"] // c["page"]), "flops": 0}
    past, new = lengths(c)
    lo, hi, req = intervals(c)
    seen = 0
    for b in range(c["batch"]):
        at = req == b
        if at.any():
            # the union of its rows' intervals: ends are sorted with the rows
            ends = np.maximum.accumulate(np.concatenate([[0], hi[at][:-1]]))
            seen += int(np.maximum(hi[at] - np.maximum(lo[at], ends), 0).sum())
    T, pairs = sum(new), int(np.maximum(hi - lo, 0).sum())
    return {"bytes": 2 * seen * row + 2 * T * c["group"] * row + 4 * (-(-seen // c["page"])) + 8 * c["batch"],
            "flops": 4.0 * pairs * c["kv_heads"] * c["group"] * c["d"]}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _keys(shape, g, dtype):
    """Keys near the means of a mixture of 512 components of norms 1 to 4, as attention's keys cluster: [..., tokens, d]."""
    d = shape[-1]
    mu = torch.randn(512, d, generator=g, device="cuda")
    mu *= (1 + 3 * torch.rand(512, 1, generator=g, device="cuda")) / mu.norm(dim=1, keepdim=True)
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(-1, d).split(1 << 22):
        at = torch.randint(512, (part.shape[0],), generator=g, device="cuda")
        part.copy_(mu[at] + 0.25 * torch.randn(part.shape, generator=g, device="cuda"))
    return out


def _normal(shape, g, dtype):
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for part in out.view(-1, shape[-1]).split(1 << 22):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return out


def _int(x, dtype=torch.int32):
    return torch.as_tensor(np.asarray(x), dtype=dtype).cuda()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * (seed % 1000003) + c["mix"] % 1000003)
    rnd = random.Random(seed * 7919 + c["mix"])
    s = {"case": c}
    P = c["page"]
    if c["op"] == "plan":
        past, new = lengths(c)
        held = [-(-p // P) for p in past]
        width = max(-(-(p + n) // P) for p, n in zip(past, new)) + 1
        total = sum(-(-(p + n) // P) for p, n in zip(past, new))
        pages = total + 64
        ids = list(range(pages))
        rnd.shuffle(ids)
        table = np.full((c["batch"], width), -1)
        at = 0
        for b, h in enumerate(held):
            table[b, :h] = ids[at:at + h]
            at += h
        free = np.array(ids[at:] + [-1] * at)
        s.update(lens=_int(past), new=_int(new), table=_int(table), free=_int(free), count=_int([pages - at]),
                 rows=sum(new), pages=pages)
        if own:
            from clustered_sparse_decode_b200 import PagedCache
            s["cache"] = PagedCache(kv_heads=1, head_dim=64, num_pages=pages, page_tokens=P)
            s["plan"] = s["cache"].new_plan(c["batch"], s["rows"])
        return s

    dt, H, d = DTYPES[c["dtype"]], c["kv_heads"], c["d"]
    if c["op"] == "append":
        T = c["rows"]
        pages = -(-T // P) + 3
        # tokens lie in runs inside scattered pages, the first run starting inside a page
        ids = list(range(pages))
        rnd.shuffle(ids)
        off = rnd.randrange(P)
        slots = np.array(ids)[(off + np.arange(T)) // P] * P + (off + np.arange(T)) % P
        s.update(slots=_int(slots, torch.int64), k=_keys((T, H, d), g, dt), v=_normal((T, H, d), g, dt),
                 K=_normal((pages, H, P, d), g, dt), V=_normal((pages, H, P, d), g, dt))
    else:
        if c["op"] == "gather":
            past, new = [c["n"]] * c["batch"], [0] * c["batch"]
        else:
            past, new = lengths(c)
        lens = [p + n for p, n in zip(past, new)]
        need = [-(-n // P) for n in lens]
        pages = sum(need) + 8
        ids = np.array(rnd.sample(range(pages), pages))
        table = np.full((c["batch"], max(max(need), 1)), -1)
        at = 0
        for b, h in enumerate(need):
            table[b, :h] = ids[at:at + h]
            at += h
        s.update(table=_int(table), lens=_int(lens), K=_keys((pages, H, P, d), g, dt), V=_normal((pages, H, P, d), g, dt))
        if c["op"] == "attend":
            Hq, T = H * c["group"], sum(new)
            _, first, prefix = masks(c)
            s.update(q=_normal((T, Hq, d), g, dt), cu=_int(np.concatenate([[0], np.cumsum(new)])), most=max(new),
                     longest=max(lens), first=_int(first) if c["doc"] else None,
                     prefix=_int(prefix) if c["prefix"] else None, slopes=None, new=_int(new))
            if c["slopes"]:
                s["slopes"] = torch.as_tensor([2.0 ** (-8.0 * (h + 1) / Hq) for h in range(Hq)]).float().cuda()
    if own:
        from clustered_sparse_decode_b200 import PagedCache
        s["cache"] = PagedCache(kv_heads=H, head_dim=d, num_pages=s["K"].shape[0], page_tokens=P, dtype=c["dtype"],
                                K=s["K"], V=s["V"])
    return s


# ---------------------------------------------------------------------------
# The operators
# ---------------------------------------------------------------------------
def run(s):
    return globals()["_" + s["case"]["op"]](s)


def _plan(s):
    if own:
        p = s["cache"].plan(s["lens"], s["new"], s["table"], s["free"], s["count"], out=s["plan"])
        return p.lens, p.cu, p.slots, p.positions, p.free_count, s["table"]
    P, T, width = s["case"]["page"], s["rows"], s["table"].shape[1]
    lens, new = s["lens"].long(), s["new"].long()
    after = lens + new
    cu = torch.nn.functional.pad(new.cumsum(0), (1, 0))
    held, need = (lens + P - 1) // P, (after + P - 1) // P
    got = (need - held).cumsum(0)
    # request b's k-th new page is the pool's (got before b + k)-th from its end
    col = torch.arange(width, device="cuda")[None]
    kth = got[:, None] - need[:, None] + col
    fresh = (col >= held[:, None]) & (col < need[:, None])
    ids = s["free"].long()[(s["count"].long() - 1 - kth).clamp(0, s["free"].numel() - 1)]
    s["table"].copy_(torch.where(fresh, ids, s["table"].long()))
    row = torch.arange(T, device="cuda")
    req = torch.searchsorted(cu[1:], row, right=True)
    pos = lens[req] + row - cu[req]
    slots = s["table"].long()[req, pos // P] * P + pos % P
    return after.int(), cu.int(), slots, pos.int(), (s["count"] - got[-1]).int(), s["table"]


def _append(s):
    if own:
        s["cache"].append(s["k"], s["v"], s["slots"])
        return s["K"], s["V"]
    P = s["case"]["page"]
    page, off = s["slots"] // P, s["slots"] % P
    s["K"][page, :, off] = s["k"]
    s["V"][page, :, off] = s["v"]
    return s["K"], s["V"]


def _gather(s):
    c = s["case"]
    if own:
        return s["cache"].gather(s["table"], s["lens"], c["n"])
    at = s["table"][:, : -(-c["n"] // c["page"])].long()
    return tuple(x[at].transpose(1, 2).reshape(c["batch"], c["kv_heads"], -1, c["d"])[:, :, : c["n"]].contiguous()
                 for x in (s["K"], s["V"]))


def _attend(s):
    c = s["case"]
    if own:
        return s["cache"].attend(s["q"], s["table"], s["lens"], s["cu"], max_new=s["most"], softcap=c["softcap"],
                                 window=c["window"], slopes=s["slopes"], prefix=s["prefix"], first_key=s["first"])
    B, H, G, d, N, n = c["batch"], c["kv_heads"], c["group"], c["d"], s["longest"], s["most"]
    at = s["table"].clamp(min=0).long()
    K, V = (x[at].transpose(1, 2).reshape(B, H, 1, -1, d)[:, :, :, :N].float() for x in (s["K"], s["V"]))
    i = torch.arange(n, device="cuda")[None]
    row = (s["cu"][:-1, None] + i).clamp(max=s["q"].shape[0] - 1).long()                         # [B, n]
    pos = s["lens"][:, None] - s["new"][:, None] + i
    q = s["q"][row].float().view(B, n, H, G, d).permute(0, 2, 3, 1, 4)                           # [B, H, G, n, d]
    z = torch.matmul(q.reshape(B, H, 1, G * n, d) / math.sqrt(d), K.transpose(-1, -2)).view(B, H, G, n, N)
    if c["softcap"]:
        z = c["softcap"] * torch.tanh(z / c["softcap"])
    j = torch.arange(N, device="cuda")[None, None]
    if s["slopes"] is not None:
        z = z - s["slopes"].view(1, H, G, 1, 1) * (pos[:, :, None] - j).abs()[:, None, None].float()
    hi = pos + 1
    if s["prefix"] is not None:
        hi = torch.maximum(hi, s["prefix"][:, None])
    seen = j < hi[:, :, None]
    if c["window"]:
        seen = seen & (j > pos[:, :, None] - c["window"])
    if s["first"] is not None:
        seen = seen & (j >= s["first"][row][:, :, None])
    seen = (seen & (i < s["new"][:, None])[:, :, None])[:, None, None]
    z = z.masked_fill(~seen, -math.inf)
    m = z.amax(-1, keepdim=True).clamp(min=-1e30)
    w = torch.exp(z - m)
    o = torch.matmul(w.view(B, H, 1, G * n, N), V).view(B, H, G, n, d) / w.sum(-1, keepdim=True).clamp(min=1e-30)
    o = o.permute(0, 3, 1, 2, 4).reshape(B * n, H * G, d)
    return o[(i < s["new"][:, None]).reshape(-1)].to(s["q"].dtype)


# ---------------------------------------------------------------------------
# The definition in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    if c["op"] in ("append", "gather"):
        return None                                                # copies: no computed number
    s = prepare(c, seed)
    if c["op"] == "plan":
        past, new = lengths(c)
        table, free = s["table"].cpu().tolist(), s["free"].cpu().tolist()
        left, cu, slots, pos = int(s["count"][0]), [0], [], []
        for b, (p, n) in enumerate(zip(past, new)):
            for t in range(p, p + n):
                if t % c["page"] == 0:
                    left -= 1
                    table[b][t // c["page"]] = free[left]
                slots.append(table[b][t // c["page"]] * c["page"] + t % c["page"])
                pos.append(t)
            cu.append(cu[-1] + n)
        i32 = lambda x: torch.tensor(x, dtype=torch.int32)
        return (i32([p + n for p, n in zip(past, new)]), i32(cu), torch.tensor(slots, dtype=torch.int64), i32(pos),
                i32([left]), i32(table))
    past, new = lengths(c)
    lo, hi, _ = intervals(c)
    H, G, d, P = c["kv_heads"], c["group"], c["d"], c["page"]
    out = torch.zeros(sum(new), H * G, d, dtype=torch.float64, device="cuda")
    lo, hi, start = torch.as_tensor(lo).cuda(), torch.as_tensor(hi).cuda(), 0
    for b in range(c["batch"]):
        p, n = past[b], new[b]
        t = torch.arange(p + n, device="cuda")
        page = s["table"][b].long()[t // P]
        for h in range(H):
            K, V = s["K"][page, h, t % P].double(), s["V"][page, h, t % P].double()
            for r in range(0, n, 1024):
                e = min(n, r + 1024)
                rows = slice(start + r, start + e)
                q = s["q"][rows, h * G:(h + 1) * G].double()                                    # [rows, G, d]
                z = torch.einsum("rgd,kd->rgk", q, K) * d ** -0.5
                if c["softcap"]:
                    z = torch.tanh(z / c["softcap"]) * c["softcap"]
                if c["slopes"]:
                    away = (torch.arange(p + r, p + e, device="cuda")[:, None] - t[None]).abs().double()
                    z = z - s["slopes"][h * G:(h + 1) * G].double()[None, :, None] * away[:, None]
                hide = (t[None] < lo[rows, None]) | (t[None] >= hi[rows, None])
                z = z.masked_fill(hide[:, None], -math.inf)
                w = torch.where(hide.all(-1)[:, None, None], torch.zeros_like(z), torch.softmax(z, -1))
                out[rows, h * G:(h + 1) * G] = torch.einsum("rgk,kd->rgd", w, V)
        start += n
    return out
