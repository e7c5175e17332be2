"""GPU: attention over the paged 8-bit cache, against its definition in 64
bits.

Tolerance of one output o = sum p v / l, with A = sum p |v| / l:
 * rounding of the output, half a step: 2^-8 |o| (bf16), 2^-24 |o| (fp32);
 * p rounded to f16: 2^-11 A, and below f16's normal range half its smallest
   step, 2^-25, for each of the n tokens, in units of the largest |v| and
   the power of two above the largest value scale (2 at most);
 * the scores: D products summed in fp32 (2^-23 each, whatever the order),
   d = (D + 4) 2^-23 sum |q k| scale, twice that in p / l;
 * the sums over n tokens in fp32: 2 n 2^-24 A; exp2 and the scales: 2^-20 A."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import quantized_weight_decode_dequant_amd as pkg
from helpers import note, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Case:
    def __init__(self, seed, lens, T, H=2, G=4, D=128, page=64, fmt=pkg.KV_INT8, tree=False, spare=3, qscale=1.0, pages=None):
        g = np.random.default_rng(seed)
        self.g, self.fmt, self.page, self.H, self.G, self.D = g, fmt, page, H, G, D
        R = len(lens)
        self.lens, self.T = np.array(lens), np.array(T)
        nb = -(-self.lens // page)
        self.cols = max(int(nb.max()), 1)
        self.pages = int(nb.sum()) + spare if pages is None else pages
        perm = g.permutation(self.pages)
        self.table = np.full((R, self.cols), -1)
        at = 0
        for r in range(R):
            self.table[r, : nb[r]] = perm[at: at + nb[r]]
            at += nb[r]
        self.q_start = np.concatenate([[0], np.cumsum(self.T)])
        self.M = int(self.q_start[-1])
        shape = (self.pages, H, page, D)
        if fmt == pkg.KV_INT8:
            self.k, self.v = (np.clip(np.rint(40 * g.standard_normal(shape)), -127, 127).astype(np.int8).view(np.uint8) for _ in range(2))
            unit = 0.025
        else:
            self.k, self.v = (ref.e4m3_bits(np.clip(140 * g.standard_normal(shape), -448, 448)) for _ in range(2))
            unit = 0.007
        self.ks, self.vs = (((0.3 + g.random(shape[:2])) * unit).astype(np.float32) for _ in range(2))
        self.q = to_np(torch.from_numpy(qscale * g.standard_normal((max(self.M, 1), H * G, D))).to(torch.bfloat16))[: self.M]
        self.tree = None
        if tree:
            masks = []
            for n in self.T:
                seen = []
                for j in range(n):
                    p = int(g.integers(-1, j)) if j else -1
                    seen.append((seen[p] if p >= 0 else 0) | (1 << j))
                masks += seen
            self.tree = np.array(masks, dtype=np.uint32)

    def cache(self):
        dt = torch.int8 if self.fmt == pkg.KV_INT8 else torch.float8_e4m3fn
        dev = [torch.from_numpy(ref.to_blocks(c, i)).to(DEV).view(dt) for i, c in ((False, self.k), (True, self.v))]
        return pkg.KVCache(*dev, torch.from_numpy(self.ks).to(DEV), torch.from_numpy(self.vs).to(DEV))

    def args(self):
        t = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
        d = dict(q=torch.from_numpy(self.q).to(torch.bfloat16).to(DEV), q_start=t(self.q_start), lens=t(self.lens),
                 table=t(self.table), max_q=max(int(self.T.max()), 1))
        if self.tree is not None:
            d["tree_mask"] = torch.from_numpy(self.tree.view(np.int32)).to(DEV)
        return d

    def want(self, window=0, scale=None):
        return ref.attention(self.k, self.v, self.ks.astype(np.float64), self.vs.astype(np.float64), self.fmt == pkg.KV_E4M3,
                             self.q, self.q_start, self.lens, self.table, self.tree, window, scale)

    def check(self, got, window=0, scale=None, f32=False):
        o, A, S = self.want(window, scale)
        n = int(self.lens.max())
        vmax = float(self.vs.max()) * (127 if self.fmt == pkg.KV_INT8 else 448)
        d = (self.D + 4) * 2.0 ** -23 * S[:, :, None]
        tol = ((2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(o) + (2.0 ** -11 + 2 * d + 2 * n * 2.0 ** -24 + 2.0 ** -20) * A
               + n * 2.0 ** -25 * 2 * vmax)
        got = to_np(got)
        ok = ~np.isnan(o)
        assert np.all(np.isfinite(got[ok]))
        err = np.abs(got - o)[ok] / tol[ok].clip(1e-30)
        zero = ok & (A == 0)
        assert not got[zero].any()
        assert err.size == 0 or err.max() <= 1, err.max()
        return float(err.max()) if err.size else 0.0

    def run_rows(self, requests):
        """Runs all, checks the rows of some requests."""
        got = pkg.kv_attention_run(self.cache(), **self.args())
        torch.cuda.synchronize()
        sub = object.__new__(Case)
        sub.__dict__.update(self.__dict__)
        sub.lens, sub.table, sub.T = self.lens[requests], self.table[requests], self.T[requests]
        sub.q_start = np.concatenate([[0], np.cumsum(sub.T)])
        rows = np.concatenate([np.arange(self.q_start[r], self.q_start[r + 1]) for r in requests])
        sub.q, sub.M = self.q[rows], len(rows)
        sub.check(got[torch.from_numpy(rows).to(DEV)])
        return got

    def run(self, window=0, scale=None, out_dtype=None, **kw):
        a = self.args()
        a.update(kw)
        for dt in (pkg.OUT_BF16, pkg.OUT_F32) if out_dtype is None else (out_dtype,):
            got = pkg.kv_attention_run(self.cache(), window=window, scale=scale, out_dtype=dt, **a)
            torch.cuda.synchronize()
            self.check(got, window, scale, dt == pkg.OUT_F32)
        return got


FMTS = [pkg.KV_INT8, pkg.KV_E4M3]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
def test_types_heads_pages(fmt, D, page):
    note("attention fmt=%d D=%d page=%d" % (fmt, D, page))
    Case(D + page, [1, page, page + 1, 700, 31, 33], [1] * 6, D=D, page=page, fmt=fmt).run()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (2, 3), (1, 7), (2, 16), (1, 17), (1, 71)])
@pytest.mark.parametrize("T", [1, 2, 5, 16, 32])
def test_groups_and_tiles(fmt, H, G, T):
    note("attention H=%d G=%d T=%d" % (H, G, T))
    Case(H * 100 + G + T, [T, 47, 300 + T], [T, min(T, 3), T], H=H, G=G, D=64, fmt=fmt).run()


@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1000, 5003])
def test_lengths(n):
    note("attention length", n)
    Case(n, [n], [1], H=1, G=4, D=64, page=32).run()
    Case(n, [n], [min(n, 7)], H=1, G=4, D=64, page=64, fmt=pkg.KV_E4M3).run()


@pytest.mark.parametrize("R,H", [(1, 1), (1, 8), (40, 2), (160, 8)])
def test_splits(R, H):
    """One long request and a ragged batch: many chunks and few."""
    note("attention splits R=%d H=%d" % (R, H))
    lens = [9001] + [int(x) for x in np.random.default_rng(R).integers(1, 3000 // R + 40, R - 1)]
    Case(R, lens, [1] * R, H=H, G=4, D=64, page=32).run(out_dtype=pkg.OUT_F32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T", [1, 2, 8, 16, 31, 32])
def test_trees(fmt, T):
    note("attention tree T=%d" % T)
    c = Case(T, [T, T + 1, 200 + T, 64 * 3], [T, min(T, 2), T, T], D=128, tree=True, fmt=fmt)
    c.run()
    c.tree[:] = 0                        # a draft token that does not see itself: context only, or nothing
    c.run()
    c.tree[:] = 0xFFFFFFFF               # bits behind the last new token mean nothing
    c.run()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 512, 5000, 1 << 30])
@pytest.mark.parametrize("T", [1, 6])
def test_windows(fmt, window, T):
    note("attention window=%d T=%d" % (window, T))
    Case(window % 977, [T, 40, 1200, 4099], [T] * 4, H=2, G=2, D=64, page=32, fmt=fmt).run(window=window)


def test_empty_requests_and_rows_left_alone():
    """Requests without tokens, without query rows, longer than their rows
    say; the rows of no request and the padding keep what they held."""
    c = Case(3, [0, 5, 0, 100, 64, 2], [1, 0, 2, 3, 1, 4], D=64)
    a = c.args()
    M = c.M + 5
    for dt in (torch.bfloat16, torch.float32):
        wide = torch.full((M, c.H * c.G + 2, c.D), 7.0, dtype=dt, device=DEV)
        out = wide[:, : c.H * c.G]
        q = torch.cat([a["q"], torch.full((5, c.H * c.G, c.D), float("nan"), dtype=torch.bfloat16, device=DEV)])
        got = pkg.kv_attention_run(c.cache(), **dict(a, q=q, out=out))
        torch.cuda.synchronize()
        c.check(got[: c.M], f32=dt == torch.float32)
        assert bool((wide[c.M:] == 7).all()) and bool((wide[:, c.H * c.G:] == 7).all())


def test_strided_q():
    c = Case(8, [70, 300], [3, 1], D=128, H=2, G=3)
    a = c.args()
    joint = torch.full((c.M, (c.H * c.G + 2 * c.H) * c.D), float("nan"), dtype=torch.bfloat16, device=DEV)
    q = joint[:, : c.H * c.G * c.D].view(c.M, c.H * c.G, c.D)
    q.copy_(a["q"])
    assert not q.is_contiguous()
    c.check(pkg.kv_attention_run(c.cache(), **dict(a, q=q)))


@pytest.mark.parametrize("fmt", FMTS)
def test_garbage_behind_the_last_token(fmt):
    """Slots behind a request's last token, unused pages and the scales of
    unused pages may hold anything, NaN codes and NaN scales among it."""
    c = Case(5, [37, 65, 1], [1, 2, 1], D=64, page=64, fmt=fmt)
    ref_out = c.run(out_dtype=pkg.OUT_BF16)
    used = {int(p) for p in c.table.reshape(-1) if p >= 0}
    for p in range(c.pages):
        if p not in used:
            c.k[p] = c.v[p] = 0x7F
            c.ks[p] = c.vs[p] = np.nan
    for r, n in enumerate(c.lens):
        c.k[c.table[r, (n - 1) // 64], :, (n - 1) % 64 + 1:] = 0x7F
        c.v[c.table[r, (n - 1) // 64], :, (n - 1) % 64 + 1:] = 0xFF
    got = pkg.kv_attention_run(c.cache(), **c.args())
    assert torch.equal(got, ref_out)


def test_pages_that_are_not_there():
    c = Case(6, [200, 130, 64], [1, 2, 1], D=64, page=32)
    c.table[0, 2] = -1
    c.table[1, 0] = c.pages
    c.table[2, :2] = 2 ** 31 - 1
    c.run()


def test_zero_scales_and_wide_ones():
    """Value blocks of zeros (scale 0), and neighbours whose scales differ by
    2^40: the small ones still count where they are all that is seen."""
    c = Case(7, [640, 64, 96], [1, 1, 1], D=64, page=32)
    for i, p in enumerate(c.table[0]):
        c.vs[p] = [0.0, 1e-3, 2.0 ** -40, 1e4, 0.25][i % 5]
    c.vs[c.table[1, :2]] = 0.0
    c.vs[c.table[2, :3]] = 2.0 ** -60
    c.ks[c.table[1, 0]] = 0.0
    c.run()
    one = Case(7, [96], [1], D=64, page=32)
    one.vs[:] = 2.0 ** -60
    one.run()                            # its tolerance scales with its own values


def test_scores_far_apart():
    """Large queries: the softmax is one token; scores far below zero; a scale
    of zero (the mean of the values)."""
    Case(11, [300, 33], [2, 1], D=128, qscale=100.0).run()
    Case(12, [300, 33], [2, 1], D=128, qscale=1e30).run(scale=1e-30)
    Case(13, [700], [1], D=64).run(scale=0.0)
    Case(14, [700], [1], D=64).run(scale=-0.2)


def test_rising_scores():
    """Keys ordered so that each step's scores pass the running maximum."""
    c = Case(15, [2000], [1], H=1, G=2, D=64, page=64)
    q = c.q[0, 0]
    ids = c.table[0]
    rows = np.concatenate([c.k[p, 0] for p in ids]).view(np.int8).astype(np.float64)[:2000]
    order = np.argsort(rows @ q)
    flat = np.zeros((len(ids) * 64, 64), np.uint8)
    flat[:2000] = rows[order].astype(np.int8).view(np.uint8)
    for i, p in enumerate(ids):
        c.k[p, 0] = flat[i * 64:(i + 1) * 64]
        c.ks[p] = 0.05
    c.run()


def test_query_rows_that_are_not_finite_stay_alone():
    c = Case(16, [500, 90], [4, 2], D=64)
    a = c.args()
    cache = c.cache()
    clean = pkg.kv_attention_run(cache, **a)
    a["q"] = a["q"].clone()
    a["q"][1, 3, 5] = float("nan")
    a["q"][4, 0, 0] = float("inf")
    got = pkg.kv_attention_run(cache, **a)
    bad = torch.zeros(c.M, c.H * c.G, dtype=torch.bool, device=DEV)
    bad[1, 3] = bad[4, 0] = True
    assert torch.equal(got[~bad], clean[~bad]) and torch.isnan(got[bad]).all()


def test_longer_than_max_len_is_seen():
    c = Case(17, [3000, 40], [1, 1], D=64, page=32)
    got = pkg.kv_attention_run(c.cache(), **c.args(), max_len=64)
    torch.cuda.synchronize()
    assert torch.isnan(got[0]).all() and torch.isfinite(got[1]).all()


def test_more_rows_than_max_q_are_left_alone():
    c = Case(18, [100], [6], D=64)
    a = dict(c.args(), max_q=4)
    out = torch.full((c.M, c.H * c.G, c.D), 3.0, dtype=torch.bfloat16, device=DEV)
    pkg.kv_attention_run(c.cache(), **a, out=out)
    assert bool((out[4:] == 3).all())


@pytest.mark.parametrize("lens", [[100, 90], [3000, 2500]])
def test_more_rows_than_max_q_are_seen(lens):
    c = Case(34, lens, [6, 3], D=64)
    a = dict(c.args(), max_q=4)
    want = pkg.kv_attention_run(c.cache(), **c.args())
    out = torch.full((c.M, c.H * c.G, c.D), 3.0, dtype=torch.bfloat16, device=DEV)
    pkg.kv_attention_run(c.cache(), **a, out=out)
    torch.cuda.synchronize()
    assert torch.isnan(out[:4]).all() and bool((out[4:6] == 3).all())
    out[:6] = want[:6]
    c.check(out)


def test_q_start_past_all_rows():
    """Offsets near the end of 32 bits: not computed, and nothing else is."""
    c = Case(35, [100, 70, 50], [2, 2, 2], D=64)
    a = c.args()
    a["q_start"] = torch.tensor([0, 2, 2 ** 31 - 1, -2 ** 31 + 4], dtype=torch.int32, device=DEV)
    out = torch.full((c.M, c.H * c.G, c.D), 3.0, dtype=torch.bfloat16, device=DEV)
    got = pkg.kv_attention_run(c.cache(), **dict(a, max_q=32), out=out)
    torch.cuda.synchronize()
    assert torch.isfinite(got[:2]).all() and bool((got[2:] == 3).all())


def test_q_start_that_cannot_be():
    """Offsets past the rows of q: those requests are not computed."""
    c = Case(19, [100, 70], [2, 2], D=64)
    a = c.args()
    a["q_start"] = torch.tensor([0, 2, 99], dtype=torch.int32, device=DEV)
    out = torch.full((c.M, c.H * c.G, c.D), 3.0, dtype=torch.bfloat16, device=DEV)
    got = pkg.kv_attention_run(c.cache(), **dict(a, max_q=32), out=out)
    torch.cuda.synchronize()
    assert bool((got[2:] == 3).all()) and torch.isfinite(got[:2]).all()


@pytest.mark.parametrize("fmt", FMTS)
def test_past_32_bits(fmt):
    """A pool of more than 4 GiB a side, the request on its last pages."""
    page, H, D = 128, 8, 256
    pages = (1 << 32) // (page * H * D) + 40
    note("attention pool of %.1f GiB" % (pages * page * H * D / 2 ** 30))
    c = Case(20, [3 * page + 5], [2], H=H, G=2, D=D, page=page, fmt=fmt, spare=4)
    dt = torch.int8 if fmt == pkg.KV_INT8 else torch.float8_e4m3fn
    small = c.cache()
    big = []
    for x in (small.k, small.v):
        b = torch.zeros(pages, H, page, D, dtype=torch.uint8, device=DEV)
        b[-c.pages:] = x.view(torch.uint8)
        big.append(b.view(dt))
    sc = []
    for x in (small.k_scales, small.v_scales):
        s = torch.zeros(pages, H, device=DEV)
        s[-c.pages:] = x
        sc.append(s)
    a = c.args()
    a["table"] = torch.where(a["table"] >= 0, a["table"] + pages - c.pages, a["table"])
    c.check(pkg.kv_attention_run(pkg.KVCache(*big, *sc), **a))


def test_same_result_every_time_and_alone():
    """Bit-equal in repeated runs, on another stream, beside another call, and
    for a request alone in the batch with the same split."""
    c = Case(21, [2500, 300], [5, 5], D=128)
    a, cache = c.args(), c.cache()
    first = pkg.kv_attention_run(cache, **a)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    outs = []
    for _ in range(3):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(pkg.kv_attention_run(cache, **a))
    torch.cuda.synchronize()
    assert all(torch.equal(first, o) for o in outs)


@pytest.mark.parametrize("lens,H", [([200003] * 4, 8), ([150001, 1, 0, 90000] + [70000] * 20, 16)])
def test_long_runs_over_shared_pages(lens, H):
    """Workgroups whose run is longer than the 64 pages whose entries a wave
    holds at once; requests that share pages with each other, and a table
    that names a page many times; value scales that grow along the way."""
    note("attention long runs R=%d" % len(lens))
    page, pages = 32, 97
    c = Case(30, [min(n, 3000) for n in lens], [1 if n else 0 for n in lens], H=H, G=1, D=64, page=page, pages=4096)
    c.lens = np.array(lens)
    c.pages = pages
    c.k, c.v, c.ks, c.vs = c.k[:pages], c.v[:pages], c.ks[:pages], c.vs[:pages]
    c.vs *= np.linspace(0.01, 1, pages, dtype=np.float32)[:, None]
    cols = -(-max(lens) // page)
    c.table = np.stack([np.sort(c.g.integers(0, pages, cols)) if r % 2 else c.g.integers(0, pages, cols) for r in range(len(lens))])
    # the reference for some of the requests (the rows of the others are checked against each other's split)
    got = c.run_rows([0, len(lens) - 1])
    assert torch.isfinite(got).all()


def test_many_requests():
    """More requests than a wave has lanes, most of them without new tokens."""
    g = np.random.default_rng(31)
    R = 1500
    T = (g.random(R) < 0.1).astype(int)
    T[-1] = 3
    lens = np.where(T > 0, g.integers(3, 200, R), 5)
    lens[700], T[700] = 2100, 2
    Case(32, lens.tolist(), T.tolist(), H=2, G=2, D=64, page=32).run(out_dtype=pkg.OUT_BF16)


@pytest.mark.parametrize("as_int", [False, True])
def test_given_stream_takes_its_own_memory(as_int):
    """Output and workspace of a call on a given stream are not memory that
    the current stream freed but has work left to do on."""
    c = Case(33, [5000], [5])
    a, cache = c.args(), c.cache()
    first = pkg.kv_attention_run(cache, **a)
    side = torch.cuda.Stream()
    mats = [torch.ones(4096, 4096, device=DEV) for _ in range(2)]
    ws = pkg.kv_attention_workspace_bytes(1, c.M, 8, 2, 128, c.page, 5, c.cols * c.page)
    torch.cuda.synchronize()
    for _ in range(3):
        left = [torch.empty(n, dtype=torch.uint8, device=DEV) for n in (ws, first.numel() * 2)]
        for _ in range(20):
            mats[1] = torch.mm(mats[0], mats[0])
        for t in left:
            t.fill_(255)
        del left, t
        got = pkg.kv_attention_run(cache, stream=side.cuda_stream if as_int else side, **a)
        torch.cuda.synchronize()
        assert torch.equal(got, first)


def reference(c, r, window=0, scale=None):
    """Request r of a case in 64 bits, with what its tolerance needs: output,
    sum of p |v| / l, largest sum of |scale q k|, l (p relative to the largest)
    [T, Hq, ...] and the request's largest value scale that is attended to."""
    page, D, G, H = c.page, c.D, c.G, c.H
    e4m3 = c.fmt == pkg.KV_E4M3
    dec = ref.e4m3_value if e4m3 else (lambda b: b.view(np.int8).astype(np.float64))
    T, n, scale = int(c.T[r]), int(c.lens[r]), c.D ** -0.5 if scale is None else scale
    rows = np.arange(c.q_start[r], c.q_start[r] + T)
    ids = np.asarray(c.table[r][: -(-n // page)])
    there = (ids >= 0) & (ids < len(c.k))
    safe = np.where(there, ids, 0)
    t, pos = np.arange(n), n - T + np.arange(T)
    see = (t[None, :] <= pos[:, None]) & np.repeat(there, page)[None, :n]
    if window:
        see &= t[None, :] > pos[:, None] - window
    out, A, S, L = np.zeros((T, H * G, D)), np.zeros((T, H * G, D)), np.zeros((T, H * G)), np.ones((T, H * G))
    for h in range(H):
        K = (dec(np.ascontiguousarray(c.k[safe, h])) * c.ks[safe, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:n]
        V = (dec(np.ascontiguousarray(c.v[safe, h])) * c.vs[safe, h].astype(np.float64)[:, None, None]).reshape(-1, D)[:n]
        for i in range(h * G, (h + 1) * G):
            s = np.where(see, scale * (c.q[rows, i] @ K.T), -np.inf)
            top = s.max(1, keepdims=True)
            p = np.exp(s - np.where(np.isinf(top), 0.0, top))
            l = np.maximum(p.sum(1), 1e-300)
            out[:, i], A[:, i] = p @ V / l[:, None], p @ np.abs(V) / l[:, None]
            S[:, i] = np.where(see, abs(scale) * (np.abs(c.q[rows, i]) @ np.abs(K).T), 0.0).max(1)
            L[:, i] = l
    seen = ids[there]
    return out, A, S, L, float(c.vs[seen].max()) if len(seen) else 0.0


def check_requests(c, got, requests, f32=False, window=0, scale=None, teeth=4.0):
    """The requests' rows against the tolerance of this file's head, with what
    a probability may lose below f16's normal range counted against the row's
    own sum l and the request's own scales; the outputs' size has to be `teeth`
    times it in the median, so that a wrong one is seen."""
    got = to_np(got)
    for r in requests:
        o, A, S, L, vs = reference(c, r, window, scale)
        n = int(c.lens[r])
        vmax = vs * (127 if c.fmt == pkg.KV_INT8 else 448)
        d = (c.D + 4) * 2.0 ** -23 * S[:, :, None]
        tol = ((2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(o) + (2.0 ** -11 + 2 * d + 2 * n * 2.0 ** -24 + 2.0 ** -20) * A
               + n * 2.0 ** -25 * 2 * vmax / L[:, :, None])
        mine = got[c.q_start[r]: c.q_start[r + 1]]
        assert np.all(np.isfinite(mine)), r
        err = np.abs(mine - o) / tol.clip(1e-300)
        assert err.max() <= 1, (r, err.max(), np.argwhere(err > 1)[:3])
        assert teeth == 0 or np.median(np.abs(o) / tol.clip(1e-300)) >= teeth, (r, np.median(np.abs(o) / tol))


def long_case(seed, R, n, T, H, G, D, fmt, pool=700, order=1):
    """R requests of about n tokens on shuffled pages of a shared pool of 32
    token pages, value scales over a factor of 100 and rising along each
    request (order 1), falling (-1) or mixed (0); the softmax of a row lies on
    few tokens."""
    c = Case(seed, [32 * pool], [T], H=H, G=G, D=D, page=32, fmt=fmt, pages=pool)
    g = c.g
    c.vs *= np.exp(g.uniform(np.log(0.01), 0, pool)).astype(np.float32)[:, None]
    c.lens = n - g.integers(0, 90, R)
    cols = -(-n // 32)
    rank = np.argsort(c.vs[:, 0])
    if order:
        c.table = np.stack([rank[np.sort(g.permutation(pool)[:cols])][::order] for _ in range(R)])
    else:
        c.table = np.stack([g.permutation(pool)[:cols] for _ in range(R)])
    c.T = np.full(R, T)
    c.q_start = np.concatenate([[0], np.cumsum(c.T)])
    c.M = R * T
    c.q = to_np(torch.from_numpy(3 * g.standard_normal((c.M, H * G, D))).to(torch.bfloat16))
    return c


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("order", [-1, 0, 1])
@pytest.mark.parametrize("R,n,T,H,G,D", [(64, 10240, 1, 16, 1, 64), (60, 8000, 3, 10, 5, 128), (40, 20480, 1, 8, 8, 256),
                                         (40, 20480, 8, 4, 4, 64), (40, 20480, 8, 4, 8, 128), (40, 20480, 16, 4, 8, 64),
                                         (40, 20480, 8, 4, 4, 256), (40, 20480, 16, 4, 4, 256)])
def test_runs_past_64_pages(R, n, T, H, G, D, order, fmt):
    """Workgroups whose run passes the 64 pages whose entries a wave holds at
    once, for each number of rows."""
    note("attention runs past 64 pages fmt=%d order=%d T=%d G=%d D=%d" % (fmt, order, T, G, D))
    c = long_case(40 + T + D, R, n, T, H, G, D, fmt, order=order)
    got = pkg.kv_attention_run(c.cache(), **c.args())
    torch.cuda.synchronize()
    assert torch.isfinite(got).all()
    check_requests(c, got, [0, R - 1])


@pytest.mark.parametrize("n,T", [(5003, 1), (5003, 9), (9001, 1)])
def test_cut_contexts_against_their_own_sums(n, T):
    c = Case(50 + n, [n, 700, 33], [T, 1, 2], H=2, G=4, D=64, page=32, qscale=3.0)
    for dt in (pkg.OUT_BF16, pkg.OUT_F32):
        got = pkg.kv_attention_run(c.cache(), **c.args(), out_dtype=dt)
        torch.cuda.synchronize()
        check_requests(c, got, range(3), f32=dt == pkg.OUT_F32)


def test_scales_of_other_requests_do_not_count():
    """Value scales 2^80 apart between the requests of a call, each request
    checked against its own; one has blocks of zeros among small ones."""
    c = Case(51, [640, 64, 96, 3000, 1500], [1, 1, 3, 2, 1], D=64, page=32, qscale=3.0)
    nb = lambda r: -(-c.lens[r] // 32)  # noqa: E731
    for r, s in enumerate([2.0 ** 20, 0.0, 2.0 ** -60, 1e-9, 2.0 ** -30]):
        c.vs[c.table[r, : nb(r)]] *= np.float32(s)
    c.vs[c.table[4, : nb(4): 3]] = 0.0
    for fmt_out in (pkg.OUT_BF16, pkg.OUT_F32):
        got = pkg.kv_attention_run(c.cache(), **c.args(), out_dtype=fmt_out)
        torch.cuda.synchronize()
        check_requests(c, got, [0, 2, 3, 4], f32=fmt_out == pkg.OUT_F32)
        assert not got[1].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,H,G,R,n", [(1, 16, 1, 64, 10240), (8, 4, 8, 40, 20480)])
def test_first_pages_without_values(T, H, G, R, n, fmt):
    """The first 130 pages of a request are not there, or hold only zeros, and
    the others' scales are small: those others decide all the bits."""
    note("attention first pages without values fmt=%d T=%d" % (fmt, T))
    c = long_case(60 + T, R, n, T, H, G, 64, fmt, order=0)
    c.vs = ((0.3 + c.g.random(c.vs.shape)) * 2.0 ** -20).astype(np.float32)
    zero = 5
    c.vs[zero] = 0.0
    c.table[c.table == zero] = 6
    c.table[::2, :130] = -1
    c.table[1::2, :130] = zero
    got = pkg.kv_attention_run(c.cache(), **c.args())
    torch.cuda.synchronize()
    check_requests(c, got, [0, 1, 2, R - 1])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("T,G", [(1, 4), (8, 4), (16, 8)])
def test_weight_on_pages_of_small_scale(T, G, fmt):
    """All of a row's weight lies on a page whose value scale is 1.3 * 2^-20
    beside a page of scale 1 that every row scores far below it.  The equal
    probabilities p vs / vref 2^7 = 1.3 * 2^-13 are normal in f16: half a step
    is 2^-11 of each, so of the output."""
    c = Case(70, [64], [T], H=1, G=G, D=64, page=32, fmt=fmt)
    far, near = (int(p) for p in c.table[0, :2])
    low = np.full(64, 100 if fmt == pkg.KV_INT8 else 448.0)
    c.q = np.abs(c.q) + 1.0
    c.q = to_np(torch.from_numpy(c.q).to(torch.bfloat16))
    c.k[far, 0] = (-low).astype(np.int8).view(np.uint8) if fmt == pkg.KV_INT8 else ref.e4m3_bits(low) | 0x80
    c.k[near] = 0
    c.ks[:] = 0.1
    c.vs[far], c.vs[near] = 1.0, 1.3 * 2.0 ** -20
    got = pkg.kv_attention_run(c.cache(), **c.args(), out_dtype=pkg.OUT_F32)
    torch.cuda.synchronize()
    o, A = reference(c, 0)[:2]
    # half a step of f16, and fp32 sums of 32 products, the scales and exp2
    assert np.all(np.abs(to_np(got) - o) <= (2.0 ** -11 + 64 * 2.0 ** -24 + 2.0 ** -20) * A)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("qexp,scale,kexp", [(122, None, -104), (120, -1.0, -100), (0, 2.0 ** 118, -104), (-100, 2.0 ** 126, -20)])
@pytest.mark.parametrize("n", [96, 3000])
def test_large_queries_and_scales(n, qexp, scale, kexp, fmt):
    """Queries near bf16's end, and large scales, with scores inside fp32: the
    token of the largest score is all of the softmax."""
    c = Case(80, [n], [2], H=1, G=2, D=64, page=32, fmt=fmt)
    best = [n - 3, 17]                      # for either sign of the scale
    c.q = np.full(c.q.shape, 2.0 ** qexp)
    code = np.zeros(n, np.int64)
    code[best[0]], code[best[1]] = 2, -2
    for t in range(n):
        p, o = int(c.table[0, t // 32]), t % 32
        v = np.full(64, float(code[t]))
        c.k[p, 0, o] = v.astype(np.int8).view(np.uint8) if fmt == pkg.KV_INT8 else ref.e4m3_bits(v)
    c.ks[:] = 2.0 ** kexp
    got = pkg.kv_attention_run(c.cache(), **c.args(), scale=scale)
    torch.cuda.synchronize()
    t = best[1] if scale is not None and scale < 0 else best[0]
    p, o = int(c.table[0, t // 32]), t % 32
    dec = ref.e4m3_value if fmt == pkg.KV_E4M3 else (lambda b: b.view(np.int8).astype(np.float64))
    want = dec(np.ascontiguousarray(c.v[p, 0, o])) * float(c.vs[p, 0])
    # the other tokens are 2^-1000 of it; f16's and bf16's half steps
    assert np.all(np.abs(to_np(got) - want) <= (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -20) * np.abs(want) + 64 * 2.0 ** -24 * 448 * float(c.vs.max()))


@pytest.mark.parametrize("lens,T", [([300, 500, 31], [5, 1, 3]), ([2500, 9000, 40], [5, 1, 16])])
def test_rows_depend_on_no_other_rows_values(lens, T):
    """Bit-equal whatever other requests' queries, pages and scales hold, NaN
    among it, for the same lengths; uncut contexts also for a request alone."""
    c = Case(90, lens, T, D=128)
    a = c.args()
    first = pkg.kv_attention_run(c.cache(), **a)
    whole = max(lens) <= 512
    for r in range(3):
        own = {int(p) for p in c.table[r] if p >= 0}
        others = np.array([p not in own for p in range(c.pages)])
        b = object.__new__(Case)
        b.__dict__.update(c.__dict__)
        b.k, b.v, b.ks, b.vs = c.k.copy(), c.v.copy(), c.ks.copy(), c.vs.copy()
        b.k[others] = c.g.integers(0, 127, b.k[others].shape)
        b.vs[others] *= 1000
        b.ks[others] = np.nan
        mine = slice(int(c.q_start[r]), int(c.q_start[r + 1]))
        q = torch.full_like(a["q"], float("nan"))
        q[mine] = a["q"][mine]
        got = pkg.kv_attention_run(b.cache(), **dict(a, q=q))
        torch.cuda.synchronize()
        assert torch.equal(got[mine], first[mine]), r
        if whole:
            one = dict(a, q=a["q"][mine].clone(), q_start=torch.tensor([0, T[r]], dtype=torch.int32, device=DEV),
                       lens=a["lens"][r:r + 1].clone(), table=a["table"][r:r + 1].clone())
            alone = pkg.kv_attention_run(c.cache(), **one)
            torch.cuda.synchronize()
            assert torch.equal(alone, first[mine]), r


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("exp", [118, 100, -107])
@pytest.mark.parametrize("n,T,G", [(96, 1, 2), (5003, 1, 2), (5003, 8, 8)])
def test_values_near_the_ends_of_fp32(n, T, G, exp, fmt):
    """Value scales so large that unnormalised sums of the values pass fp32's
    range, and the smallest that kv_append_run writes: the mean of all tokens
    (scores of 0)."""
    c = Case(85, [n, 40], [T, 1], H=1, G=G, D=64, page=32, fmt=fmt)
    c.q[:] = 0.0
    v = 60 + c.g.integers(0, 60, c.v.shape)
    c.v = v.astype(np.uint8) if fmt == pkg.KV_INT8 else ref.e4m3_bits(v)
    c.vs = ((0.5 + 0.5 * c.g.random(c.vs.shape)) * 2.0 ** exp).astype(np.float32)
    for dt in (pkg.OUT_BF16, pkg.OUT_F32):
        got = pkg.kv_attention_run(c.cache(), **c.args(), out_dtype=dt)
        torch.cuda.synchronize()
        check_requests(c, got, [0, 1], f32=dt == pkg.OUT_F32)
