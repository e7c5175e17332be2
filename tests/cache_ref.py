"""Plain definitions of the cache operators and the norm, in numpy, 64 bits.

Where a definition states a rounding to fp32, the 64-bit result of that one
operation is rounded to fp32 (for a product or quotient of fp32 numbers this
is the correctly rounded fp32 operation)."""
import numpy as np
import scipy.linalg
import torch


def f32(x):
    return np.asarray(x, dtype=np.float64).astype(np.float32).astype(np.float64)


def e4m3_bits(v):
    """Nearest OCP E4M3 code of |v| <= 448 (ties to even), as uint8."""
    t = torch.from_numpy(np.ascontiguousarray(v, dtype=np.float32)).to(torch.float8_e4m3fn)
    return t.view(torch.uint8).numpy()


def e4m3_value(b):
    return torch.from_numpy(np.ascontiguousarray(b)).view(torch.float8_e4m3fn).float().numpy().astype(np.float64)


def place(page, D, value):
    """[page, D] byte offsets of a block."""
    t, d = np.meshgrid(np.arange(page), np.arange(D), indexing="ij")
    if value:
        return ((t // 32) * 32 * D + (d // 32) * 1024 + (t % 16 // 4) * 256 + (d % 16) * 16
                + (d // 16 % 2) * 8 + (t // 16 % 2) * 4 + t % 4)
    return (t // 16) * 16 * D + (d // 16) * 256 + (t % 16) * 16 + d % 16


def to_rows(blocks, value):
    """Cache bytes [..., page, D] in the block order -> row-major."""
    page, D = blocks.shape[-2:]
    flat = blocks.reshape(*blocks.shape[:-2], page * D)
    return flat[..., place(page, D, value)]


def to_blocks(rows, value):
    page, D = rows.shape[-2:]
    out = np.empty(rows.shape[:-2] + (page * D,), rows.dtype)
    out[..., place(page, D, value)] = rows
    return out.reshape(rows.shape)


class Tables:
    """The bookkeeping with lists."""

    def __init__(self, page, lens, table, free):
        self.page, self.lens, self.free = page, [int(x) for x in lens], [int(x) for x in free]
        self.table = np.array(table)

    def step(self, add, keep=None, max_tokens=1 << 30, pages=1 << 30):
        page, R, nb = self.page, len(self.lens), self.table.shape[1]
        kept = [min(max(int(keep[r]), 0), self.lens[r]) if keep is not None else self.lens[r] for r in range(R)]
        add = [max(int(a), 0) for a in add]
        new = [k + a for k, a in zip(kept, add)]
        up = lambda n: -(-n // page)  # noqa: E731
        have, want = [up(n) for n in self.lens], [up(n) for n in new]
        released = [(r, b) for r in range(R) for b in range(want[r], have[r])]
        wanted = [(r, b) for r in range(R) for b in range(have[r], want[r])]
        status = (1 if len(wanted) > len(self.free) + len(released) else 0) | \
                 (2 if max(want + have) > nb else 0) | (4 if sum(add) > max_tokens else 0)
        n = min(max_tokens, 1 << 20)
        slots, pos = np.full(n, -1, np.int64), np.zeros(n, np.int64)
        if status:
            return status, np.zeros(R + 1, np.int64), slots, pos
        ids = [int(self.table[r, b]) for r, b in released]
        # the first released is the next to be taken
        stack = self.free + ids[::-1]
        table = self.table.copy()
        for r, b in released:
            table[r, b] = -1
        for r, b in wanted:
            table[r, b] = stack.pop()
        self.table, self.free, self.lens = table, stack, new
        q_start = np.concatenate([[0], np.cumsum(add)])
        i = 0
        for r in range(R):
            for p in range(kept[r], new[r]):
                slots[i], pos[i] = table[r, p // page] * page + p % page, p
                i += 1
        return status, q_start, slots, pos


def append(codes, scales, x, slots, value, e4m3):
    """New codes (uint8 [pages, H, page, D]) and scales after the append."""
    pages, H, page, D = codes.shape
    top = 448.0 if e4m3 else 127.0
    rows, scales = to_rows(codes, value).copy(), scales.astype(np.float64).copy()

    def dec(b):
        return e4m3_value(b) if e4m3 else b.view(np.int8).astype(np.float64)

    def enc(z):
        z = np.clip(np.where(np.isnan(z), 0.0, z), -top, top)
        return e4m3_bits(z) if e4m3 else np.rint(z).astype(np.int8).view(np.uint8)

    runs = []
    for m, s in enumerate(slots):
        s = int(s)
        if s < 0 or s >= pages * page:
            continue
        if runs and runs[-1][0] + runs[-1][2] == m and s == runs[-1][1] + runs[-1][2] and s % page:
            runs[-1][2] += 1
        else:
            runs.append([m, s, 1])
    for m, s, n in runs:
        p, o = s // page, s % page
        v = x[m:m + n]                                   # [n, H, D]
        for h in range(H):
            a = np.abs(v[:, h])
            a = np.where(np.isfinite(a), a, 0.0)
            amax = a.max() if a.max() >= 2.0 ** -100 else 0.0
            old = scales[p, h] if o else 0.0
            new = max(old, float(f32(amax * float(f32(1.0 / top)))))
            inv = float(f32(1.0 / new)) if new > 0 else 0.0
            if o and new > old:
                rows[p, h] = enc(f32(dec(rows[p, h]) * float(f32(old / new))))
            with np.errstate(invalid="ignore", over="ignore"):
                rows[p, h, o:o + n] = enc(f32(v[:, h] * inv))
            scales[p, h] = new
    return to_blocks(rows, value), scales


def attention(k, v, ks, vs, e4m3, q, q_start, lens, table, tree=None, window=0, scale=None):
    """(out [M, Hq, D], sum of p |v| / l [M, Hq, D], largest |v|, largest error-relevant
    score sum [M, Hq]) in 64 bits; rows of no request are NaN.  k, v: row-major
    values' codes [pages, H, page, D] (uint8)."""
    pages, H, page, D = k.shape
    M, Hq = q.shape[:2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    dec = e4m3_value if e4m3 else (lambda b: b.view(np.int8).astype(np.float64))
    out = np.full((M, Hq, D), np.nan)
    A, S = np.zeros((M, Hq, D)), np.zeros((M, Hq))
    for r in range(len(lens)):
        T, n = int(q_start[r + 1] - q_start[r]), int(lens[r])
        ids = [int(i) for i in table[r][: -(-n // page)]]
        there = np.repeat([0 <= i < pages for i in ids], page)[:n] if ids else np.zeros(0, bool)
        safe = [i if 0 <= i < pages else 0 for i in ids]
        for h in range(H):
            if n:
                K = (dec(np.ascontiguousarray(k[safe, h])) * ks[safe, h][:, None, None]).reshape(-1, D)[:n]
                V = (dec(np.ascontiguousarray(v[safe, h])) * vs[safe, h][:, None, None]).reshape(-1, D)[:n]
            for j in range(T):
                row, pos = int(q_start[r]) + j, n - T + j
                t = np.arange(n)
                see = t <= pos
                if tree is not None:
                    rel = t - (n - T)
                    see = (rel < 0) | (((int(tree[row]) >> np.clip(rel, 0, 31)) & 1) > 0)
                if window:
                    see &= t > pos - window
                see &= there
                for i in range(h * G, (h + 1) * G):
                    if not see.any():
                        out[row, i] = 0
                        continue
                    qq = q[row, i]
                    s = scale * (K[see] @ qq)
                    S[row, i] = (abs(scale) * (np.abs(K[see]) @ np.abs(qq))).max()
                    p = np.exp(s - s.max())
                    out[row, i] = p @ V[see] / p.sum()
                    A[row, i] = p @ np.abs(V[see]) / p.sum()
    return out, A, S


def norm(x, w, eps, res=None, signs=None):
    """(r, y, codes, scales) in 64 bits."""
    r = x if res is None else x + res
    rs = 1.0 / np.sqrt((r * r).mean(1) + eps)
    z = r * w
    K = x.shape[1]
    if signs is not None:
        z = ((z * signs).reshape(-1, 32) @ scipy.linalg.hadamard(32).astype(np.float64)).reshape(-1, K)
    amax = np.abs(z).max(1)
    safe = np.where(amax > 0, amax, 1.0)[:, None]
    codes = np.rint(z * 127.0 / safe).astype(np.int8)
    return r, r * rs[:, None] * w, codes, amax * rs / (127.0 * (np.sqrt(32.0) if signs is not None else 1.0))
