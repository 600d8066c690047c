"""The oracle of the paged-cache calls: plain numpy, 64 bits.

Shares no code with the CUDA path.  Arrays: K, V [pages, H, P, d]; table
[B, W]; a request's token at position p lies in page table[b][p // P], row p % P.
"""
import numpy as np


def plan(lens, new, table, free, count, P, rows):
    """(lens, cu, slots, positions, count, table) after a step, or None where it does not fit."""
    table = np.array(table)
    slots, pos, cu = [], [], [0]
    left = int(count)
    for b, (p, n) in enumerate(zip(lens, new)):
        if p < 0 or n < 0 or p + n > table.shape[1] * P:
            return None
        for t in range(p, p + n):
            if t % P == 0:
                left -= 1
                if left < 0:
                    return None
                table[b, t // P] = free[left]
            slots.append(int(table[b, t // P]) * P + t % P)
            pos.append(t)
        cu.append(cu[-1] + n)
    if len(slots) > rows:
        return None
    slots += [-1] * (rows - len(slots))
    pos += [0] * (rows - len(pos))
    return np.asarray(lens) + np.asarray(new), np.array(cu), np.array(slots), np.array(pos), left, table


def rows_of(X, table_row, n, P):
    """The first n tokens [H, n, d] of a request."""
    j = np.arange(n)
    return np.asarray(X, dtype=np.float64)[np.asarray(table_row)[j // P], :, j % P].transpose(1, 0, 2) if n else \
        np.zeros((X.shape[1], 0, X.shape[3]))


def gather(X, table, lens, n, P):
    out = np.zeros((len(lens), X.shape[1], n, X.shape[3]))
    for b, m in enumerate(lens):
        m = min(m, n)
        out[b, :, :m] = rows_of(X, table[b], m, P)
    return out


def attend(Q, K, V, table, lens, cu, P, scale=None, softcap=0.0, window=0, full=False, slopes=None, prefix=None,
           first_key=None):
    """O [rows, Hq, d], lse [rows, Hq], and what the error bounds need.

    Per row and head: the weighted sum of |v| (amp [rows, Hq, d]), the largest
    sum of |q_e k_e| * scale over the keys seen (zabs) and the largest |z| (zmax).
    Only the keys that a row sees enter any of its sums.
    """
    Q = np.asarray(Q, dtype=np.float64)
    T, Hq, d = Q.shape
    H = K.shape[1]
    G = Hq // H
    scale = d ** -0.5 if scale is None else scale
    O, amp = np.zeros((T, Hq, d)), np.zeros((T, Hq, d))
    lse, zabs, zmax = np.full((T, Hq), -np.inf), np.zeros((T, Hq)), np.zeros((T, Hq))
    for b in range(len(lens)):
        n, m = int(cu[b + 1] - cu[b]), int(lens[b])
        Kb, Vb = rows_of(K, table[b], m, P), rows_of(V, table[b], m, P)
        for i in range(n):
            t, p = int(cu[b]) + i, m - n + i
            hi = m if full else max(p + 1, min(int(prefix[b]), m) if prefix is not None else 0)
            lo = max(0, p - window + 1) if window else 0
            if first_key is not None:
                lo = max(lo, int(first_key[t]))
            if hi <= lo:
                continue
            j = np.arange(lo, hi)
            for hq in range(Hq):
                k, v = Kb[hq // G, lo:hi], Vb[hq // G, lo:hi]
                z = scale * (k @ Q[t, hq])
                if softcap:
                    z = softcap * np.tanh(z / softcap)
                if slopes is not None:
                    z = z - float(slopes[hq]) * np.abs(p - j)
                top = z.max()
                w = np.exp(z - top)
                s = w.sum()
                O[t, hq] = w @ v / s
                amp[t, hq] = w @ np.abs(v) / s
                lse[t, hq] = top + np.log(s)
                zabs[t, hq] = abs(scale) * (np.abs(k) @ np.abs(Q[t, hq])).max()
                zmax[t, hq] = np.abs(z).max()
    return O, lse, dict(amp=amp, zabs=zabs, zmax=zmax)
