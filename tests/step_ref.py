"""Plain definitions, in numpy and 64 bits, of the operators between the
projections, the cache and the next token: head norm with rotation, sampling,
attention behind a shared prefix."""
import numpy as np

from cache_ref import e4m3_value


def rope(x, w, eps, positions, axis, inv_freq, interleaved):
    """(z, |a| + |b| of each element's pair, largest angle) of x [M, H, D]."""
    M, H, D = x.shape
    half = len(inv_freq)
    y = x.copy()
    if w is not None:
        y = y / np.sqrt((x * x).mean(2, keepdims=True) + eps) * w
    positions = np.asarray(positions, np.int64).reshape(-1, M)
    z, size, far = y.copy(), np.abs(y), 0.0
    for i in range(half):
        ax = 0 if axis is None else int(axis[i])
        # (extended precision, so that the reference's own angle is not the limit)
        t = (positions[ax].astype(np.longdouble) if ax < len(positions) else np.zeros(M, np.longdouble)) * np.longdouble(inv_freq[i])
        far = max(far, float(np.abs(t).max()) if M else 0.0)
        c, s = (f(t).astype(np.float64)[:, None] for f in (np.cos, np.sin))
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + half)
        z[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        z[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
        size[:, :, a] = size[:, :, b] = np.abs(y[:, :, a]) + np.abs(y[:, :, b])
    return z, size, far


def sample(x, u, T=None, k=None, p=None, minp=None):
    """(tokens, logprobs, kept) of logits [M, V]: by sorting."""
    M, V = x.shape
    tokens, logp, keeps = np.full(M, -1), np.full(M, np.nan), []
    for m in range(M):
        row = np.where(np.isnan(x[m]), -np.inf, x[m])
        top = row.max()
        keep = np.zeros(V, bool)
        keeps.append(keep)
        if top == -np.inf:
            continue
        t = 1.0 if T is None else float(T[m])
        kk = 0 if k is None else int(k[m])
        if not t > 0:
            t, kk = 1.0, 1
        with np.errstate(invalid="ignore", over="ignore"):
            w = np.exp(np.where(row == top, 0.0, (row - top) / t if np.isfinite(t) else np.where(row == -np.inf, -np.inf, 0.0)))
        order = np.argsort(-row, kind="stable")
        n = V if kk <= 0 or kk > V else kk
        ws = w[order[:n]]
        before = np.concatenate([[0.0], np.cumsum(ws)[:-1]])
        pp, mp = 1.0 if p is None else float(p[m]), 0.0 if minp is None else float(minp[m])
        ok = np.ones(n, bool)
        if pp < 1:
            ok &= before < pp * ws.sum()
        if mp > 0:
            ok &= ws >= min(mp, 1.0)
        ok[0] = True
        keep[order[:n][ok]] = True
        c = np.cumsum(np.where(keep, w, 0.0))
        uu = min(max(float(u[m]), 0.0), 1.0) if not np.isnan(u[m]) else 0.0
        i = int(np.searchsorted(c, uu * c[-1], side="right"))
        i = min(i, int(np.searchsorted(c, c[-1])))
        tokens[m], logp[m] = i, np.log(w[i] / c[-1])
    return tokens, logp, keeps


def prefix_attention(k, v, ks, vs, e4m3, q, q_start, lens, table, prefix, prefix_len, tree=None, scale=None):
    """(out, sum of p |v| / l, largest sum |q k| scale) as cache_ref.attention's,
    with the `prefix_len` tokens of the pages `prefix` before each request's
    own; rows of no request are NaN.  k, v: row-major codes (uint8)."""
    pages, H, page, D = k.shape
    M, Hq = q.shape[:2]
    G = Hq // H
    scale = D ** -0.5 if scale is None else scale
    dec = e4m3_value if e4m3 else (lambda b: b.view(np.int8).astype(np.float64))
    out, A, S = np.full((M, Hq, D), np.nan), np.zeros((M, Hq, D)), np.zeros((M, Hq))

    def tokens(ids, n, h):
        ids = [int(i) for i in ids[: -(-n // page)]]
        if not ids:
            return np.zeros((0, D)), np.zeros((0, D)), np.zeros(0, bool)
        safe = [i if 0 <= i < pages else 0 for i in ids]
        there = np.repeat([0 <= i < pages for i in ids], page)[:n]
        return tuple((dec(np.ascontiguousarray(c[safe, h])) * sc[safe, h][:, None, None]).reshape(-1, D)[:n] for c, sc in ((k, ks), (v, vs))) + (there,)

    for h in range(H):
        pk, pv, pt = tokens(prefix, prefix_len, h)
        for r in range(len(lens)):
            a, b, n = int(q_start[r]), int(q_start[r + 1]), int(lens[r])
            T = b - a
            if T <= 0:
                continue
            ok, ov, ot = tokens(table[r], n, h)
            K, V, there = np.concatenate([pk, ok]), np.concatenate([pv, ov]), np.concatenate([pt, ot])
            new = np.arange(-len(pk), n) - (n - T)
            see = np.zeros((T, len(new)), bool)
            for j in range(T):
                see[j] = new <= j if tree is None else (new < 0) | (((int(tree[a + j]) >> np.clip(new, 0, 31)) & 1) > 0)
            see &= there
            for i in range(h * G, (h + 1) * G):
                with np.errstate(invalid="ignore"):
                    s = np.where(see, scale * (q[a:b, i] @ K.T), -np.inf)
                    big = np.where(see, abs(scale) * (np.abs(q[a:b, i]) @ np.abs(K).T), 0.0)
                top = s.max(1, keepdims=True) if s.shape[1] else np.full((T, 1), -np.inf)
                p = np.where(see, np.exp(s - np.where(top == -np.inf, 0.0, top)), 0.0)
                l = p.sum(1, keepdims=True)
                some = l > 0
                Vz = np.where(there[:, None], V, 0.0)
                out[a:b, i] = np.where(some, p @ Vz / np.where(some, l, 1.0), 0.0)
                A[a:b, i] = np.where(some, p @ np.abs(Vz) / np.where(some, l, 1.0), 0.0)
                S[a:b, i] = big.max(1) if big.shape[1] else 0.0
    return out, A, S
