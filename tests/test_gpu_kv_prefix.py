"""GPU: attention behind a shared prefix, against its definition in 64 bits.

Tolerance of one output o = sum p v / l over the prefix and the request's own
n tokens, with A = sum p |v| / l, as for the attention of requests alone:
 * rounding of the output, half a step: 2^-8 |o| (bf16), 2^-24 |o| (fp32);
 * p rounded to f16: 2^-11 A, and below f16's normal range half its smallest
   step, 2^-25, for each of the n tokens, in units of the largest |v| and
   the power of two above the largest value scale (2 at most);
 * the scores: D products summed in fp32, d = (D + 4) 2^-23 sum |q k| scale,
   twice that in p / l;
 * the sums over n tokens in fp32: 2 n 2^-24 A; exp2, the scales and the joins
   of up to 4096 segments: 2^-20 A + 2^-12 2^-8 A = 2^-19 A."""
import numpy as np
import pytest
import torch

import cache_ref
import step_ref as ref
import quantized_weight_decode_dequant_amd as pkg
from helpers import note, to_np
from quantized_weight_decode_dequant_amd import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = [pkg.KV_INT8, pkg.KV_E4M3]


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


class Case:
    def __init__(self, seed, P, lens, T, H=2, G=4, D=128, page=64, fmt=pkg.KV_INT8, tree=False, spare=3):
        g = self.g = np.random.default_rng(seed)
        self.fmt, self.page, self.H, self.G, self.D, self.P = fmt, page, H, G, D, P
        R = len(lens)
        self.lens, self.T = np.array(lens), np.array(T)
        nb, pb = -(-self.lens // page), -(-P // page)
        self.cols = max(int(nb.max()), 1)
        self.pages = int(nb.sum()) + pb + spare
        perm = g.permutation(self.pages)
        self.table = np.full((R, self.cols), -1)
        at = 0
        for r in range(R):
            self.table[r, : nb[r]] = perm[at: at + nb[r]]
            at += nb[r]
        self.prefix = np.concatenate([perm[at: at + pb], [-1]])  # one column more than it needs
        self.q_start = np.concatenate([[0], np.cumsum(self.T)])
        self.M = int(self.q_start[-1])
        shape = (self.pages, H, page, D)
        if fmt == pkg.KV_INT8:
            self.k, self.v = (np.clip(np.rint(40 * g.standard_normal(shape)), -127, 127).astype(np.int8).view(np.uint8) for _ in range(2))
            unit = 0.025
        else:
            self.k, self.v = (cache_ref.e4m3_bits(np.clip(140 * g.standard_normal(shape), -448, 448)) for _ in range(2))
            unit = 0.007
        self.ks, self.vs = (((0.3 + g.random(shape[:2])) * unit).astype(np.float32) for _ in range(2))
        self.q = to_np(torch.from_numpy(g.standard_normal((self.M, H * G, D))).to(torch.bfloat16))
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
        dev = [torch.from_numpy(cache_ref.to_blocks(c, i)).to(DEV).view(dt) for i, c in ((False, self.k), (True, self.v))]
        return pkg.KVCache(*dev, torch.from_numpy(self.ks).to(DEV), torch.from_numpy(self.vs).to(DEV))

    def args(self):
        d = dict(q=torch.from_numpy(self.q).to(torch.bfloat16).to(DEV), q_start=i32(self.q_start), lens=i32(self.lens),
                 table=i32(self.table), prefix_table=i32(self.prefix), prefix_len=i32([self.P]), max_q=max(int(self.T.max()), 1))
        if self.tree is not None:
            d["tree_mask"] = torch.from_numpy(self.tree.view(np.int32)).to(DEV)
        return d

    def check(self, got, scale=None, f32=False):
        o, A, S = ref.prefix_attention(self.k, self.v, self.ks.astype(np.float64), self.vs.astype(np.float64), self.fmt == pkg.KV_E4M3,
                                       self.q, self.q_start, self.lens, self.table, self.prefix, self.P, self.tree, scale)
        n = int(self.lens.max()) + self.P
        vmax = float(self.vs.max()) * (127 if self.fmt == pkg.KV_INT8 else 448)
        d = (self.D + 4) * 2.0 ** -23 * S[:, :, None]
        tol = ((2.0 ** -24 if f32 else 2.0 ** -8) * np.abs(o) + (2.0 ** -11 + 2 * d + 2 * n * 2.0 ** -24 + 2.0 ** -19) * A
               + n * 2.0 ** -25 * 2 * vmax)
        got, ok = to_np(got), ~np.isnan(o)
        assert np.all(np.isfinite(got[ok]))
        assert not got[ok & (A == 0)].any()
        err = np.abs(got - o)[ok] / tol[ok].clip(1e-30)
        assert err.size == 0 or err.max() <= 1, err.max()

    def run(self, scale=None, **kw):
        a = self.args()
        a.update(kw)
        for dt in (pkg.OUT_BF16, pkg.OUT_F32):
            got = pkg.kv_prefix_attention_run(self.cache(), scale=scale, out_dtype=dt, **a)
            torch.cuda.synchronize()
            self.check(got, scale, dt == pkg.OUT_F32)
        return got


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
def test_types_heads_pages(fmt, D, page):
    note("prefix fmt=%d D=%d page=%d" % (fmt, D, page))
    Case(D + page, 3 * page + 7, [1, page, page + 1, 300], [1] * 4, D=D, page=page, fmt=fmt).run()
    Case(D + page + 1, page - 1, [1, page, 17] * 5, [1] * 15, D=D, page=page, fmt=fmt).run()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows", [1, 4, 15, 16, 17, 32, 33, 48, 64, 65, 100, 128, 129, 200, 256, 257, 600])
def test_rows(fmt, D, rows):
    """All variants by the number of rows to a KV head, on both sides of their limits."""
    note("prefix rows=%d D=%d fmt=%d" % (rows, D, fmt))
    Case(rows, 777, [1 + i % 37 for i in range(rows)], [1] * rows, H=1, G=1, D=D, page=32, fmt=fmt).run()


@pytest.mark.parametrize("P", [0, 1, 15, 31, 32, 33, 63, 64, 65, 127, 129, 256, 1000, 5003])
@pytest.mark.parametrize("R", [2, 40])
def test_prefix_lengths(P, R):
    note("prefix length", P, R)
    Case(P, P, [1 + 7 * i for i in range(R)], [1] * R, H=1, G=4, D=64, page=32).run()
    Case(P + 1, P, [9 + i for i in range(R)], [1 + i % 7 for i in range(R)], H=2, G=2, D=128, page=64, fmt=pkg.KV_E4M3).run()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("H,G", [(1, 1), (3, 1), (2, 3), (1, 7), (2, 16), (1, 71)])
@pytest.mark.parametrize("T", [1, 5, 32])
def test_groups_and_drafts(fmt, H, G, T):
    note("prefix H=%d G=%d T=%d" % (H, G, T))
    Case(H * 100 + G + T, 450, [T, 47, 100 + T], [T, min(T, 3), T], H=H, G=G, D=64, fmt=fmt).run()


@pytest.mark.parametrize("R,T", [(1, 3), (3, 16), (12, 32)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_trees(R, T, D):
    Case(R + T, 290, [T + 20 * i for i in range(R)], [T - i % 3 for i in range(R)], D=D, tree=True).run()


@pytest.mark.parametrize("rows", [4, 150])
def test_idle_requests_and_rows_of_none(rows):
    """Requests without new tokens; rows behind the last request stay as they are."""
    lens, T = [5, 0, 40, 3] * (rows // 4), [1, 0, 0, 2] * (rows // 4)
    c = Case(rows, 200, lens, T, H=1, G=2)
    c.run()
    a = c.args()
    a["q"] = torch.cat([a["q"], torch.full((5, 2, 128), float("nan"), dtype=torch.bfloat16, device=DEV)])
    out = torch.full(a["q"].shape, 9.0, dtype=torch.bfloat16, device=DEV)
    pkg.kv_prefix_attention_run(c.cache(), out=out, **a)
    c.check(out[: c.M])
    assert bool((out[c.M:] == 9).all())


@pytest.mark.parametrize("R", [2, 30, 80])
def test_nothing_to_see_and_pages_that_are_not_there(R):
    c = Case(R, 190, [30 + i for i in range(R)], [1] * R, H=1, G=4)
    c.prefix[1] = c.pages + 5          # no such page: not attended to
    c.table[0, 0] = -7
    c.run()
    c.prefix[:] = -1
    c.run()
    c.table[:] = 1 << 30
    got = c.run()
    assert not got.any()


@pytest.mark.parametrize("R", [3, 50])
def test_calls_that_are_told_too_little(R):
    """A prefix longer than max_prefix: NaN everywhere; a request longer than
    max_len, or with more tokens than max_q: NaN in its rows."""
    c = Case(R, 300, [10] * (R - 1) + [70], [2] + [1] * (R - 1), H=1, G=4)
    a = c.args()
    got = pkg.kv_prefix_attention_run(c.cache(), max_prefix=299, **a)
    assert bool(got.isnan().all())
    got = pkg.kv_prefix_attention_run(c.cache(), max_prefix=300, max_len=69, **a)
    assert bool(got[-1].isnan().all()) and bool(got[:-1].isfinite().all())
    out = torch.full(got.shape, 9.0, dtype=torch.bfloat16, device=DEV)
    pkg.kv_prefix_attention_run(c.cache(), out=out, **dict(a, max_q=1))
    assert bool(out[0].isnan().all()) and bool((out[1] == 9).all()) and bool(out[2:].isfinite().all())


@pytest.mark.parametrize("R", [3, 70])
def test_slots_behind_the_last_token_may_hold_anything(R):
    c = Case(R, 77, [9] * R, [1] * R, H=2, G=2, D=64, page=64, fmt=pkg.KV_E4M3)
    want = c.run()
    for side in (c.k, c.v):
        side[c.prefix[1], :, 13:] = 0x7F  # NaN
        side[c.table[:, 0], :, 9:] = 0xFF
    assert torch.equal(c.run(), want)


@pytest.mark.parametrize("R", [3, 70])
@pytest.mark.parametrize("fmt", FMTS)
def test_value_scales_far_apart(R, fmt):
    c = Case(R, 64 * 5, [40] * R, [1] * R, H=1, G=4, fmt=fmt)
    c.vs[c.prefix[:5], 0] *= np.array([1, 2.0 ** -7, 0, 2.0 ** -3, 1], np.float32)
    c.ks[c.prefix[3], 0] = 0
    c.run()
    c.vs[:] = 0
    assert not c.run().any()


def test_a_prefix_of_more_pages_than_a_wave_has_lanes():
    for R in (2, 20, 70):
        Case(R, 32 * 131 + 5, [3] * R, [1] * R, H=1, G=4, D=64, page=32).run()


def test_scales_of_the_scores():
    for R in (2, 40):
        c = Case(R, 100, [12] * R, [1] * R)
        for s in (0.0, -0.3, 1.7):
            c.run(scale=s)


@pytest.mark.parametrize("R,T", [(4, 1), (40, 1), (20, 8)])
def test_strided_rows(R, T):
    c = Case(R, 333, [T + 9] * R, [T] * R, H=2, G=4, D=64)
    a = c.args()
    joint = torch.randn(c.M, 12, 64, device=DEV).to(torch.bfloat16)
    joint[:, 2:10] = a["q"]
    out = torch.full((c.M, 16, 64), 5.0, device=DEV)
    pkg.kv_prefix_attention_run(c.cache(), **dict(a, q=joint[:, 2:10], out=out[:, 4:12]))
    c.check(out[:, 4:12], f32=True)
    assert bool((out[:, :4] == 5).all()) and bool((out[:, 12:] == 5).all())


@pytest.mark.parametrize("R,T,P", [(3, 1, 900), (30, 4, 900), (3, 16, 2500)])
def test_equals_attention_over_the_whole(R, T, P):
    """The same as kv_attention_run over tables that list the prefix's pages first."""
    P -= P % 64
    c = Case(R, P, [T + 11 * i for i in range(R)], [T] * R)
    a = c.args()
    got = pkg.kv_prefix_attention_run(c.cache(), out_dtype=pkg.OUT_F32, **a)
    table = torch.cat([a["prefix_table"][:-1].expand(R, -1), a["table"]], 1).contiguous()
    whole = pkg.kv_attention_run(c.cache(), a["q"], a["q_start"], a["lens"] + P, table, T, out_dtype=pkg.OUT_F32)
    c.check(whole, f32=True)
    c.check(got, f32=True)


@pytest.mark.parametrize("R", [3, 40])
def test_captured_with_lengths_that_change(R):
    """Two graphs, a workspace each, replayed in turn with new lengths; every replay equals the eager call."""
    cases = [Case(R + i, 700, [40] * R, [2] * R, H=1, G=4) for i in range(2)]
    caches, args = [c.cache() for c in cases], [c.args() for c in cases]
    n = pkg.kv_prefix_attention_workspace_bytes(R, 2 * R, 4, 1, 128, 64, 2, args[0]["table"].shape[1] * 64, args[0]["prefix_table"].shape[0] * 64)
    ws = [torch.empty(n, dtype=torch.uint8, device=DEV) for _ in cases]
    outs = [torch.zeros(2 * R, 4, 128, dtype=torch.bfloat16, device=DEV) for _ in cases]
    graphs = [workloads.capture_graph(lambda i=i: pkg.kv_prefix_attention_run(caches[i], workspace=ws[i], out=outs[i], **args[i])) for i in range(2)]
    g = np.random.default_rng(1)
    for rep in range(6):
        for i, c in enumerate(cases):
            c.P, c.lens = int(g.integers(0, 701)), g.integers(2, 41, R)
            c.T = g.integers(0, 3, R)
            c.q_start = np.concatenate([[0], np.cumsum(c.T)])
            args[i]["prefix_len"].copy_(i32([c.P]))
            args[i]["lens"].copy_(i32(c.lens))
            args[i]["q_start"].copy_(i32(c.q_start))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i, c in enumerate(cases):
            m = int(c.q_start[-1])
            want = pkg.kv_prefix_attention_run(caches[i], **args[i])
            assert torch.equal(outs[i][:m], want[:m]), rep
            c.check(outs[i])
        _ = torch.randn(1000, device=DEV).sum().item()


def test_two_streams_and_repeated_runs():
    cases = [Case(i, 1500, [40] * 20, [1 + i] * 20) for i in range(2)]
    caches, args = [c.cache() for c in cases], [c.args() for c in cases]
    alone = [pkg.kv_prefix_attention_run(k, **a) for k, a in zip(caches, args)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(4):
        both = [pkg.kv_prefix_attention_run(k, stream=s, **a) for k, a, s in zip(caches, args, streams)]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(alone, both))


def test_a_large_call_by_some_of_its_rows():
    """48 requests behind 32768 tokens: rows of three of them."""
    c = Case(3, 32768, [1 + 30 * i for i in range(48)], [1] * 48, H=1, G=4)
    got = pkg.kv_prefix_attention_run(c.cache(), **c.args())
    torch.cuda.synchronize()
    pick = [0, 17, 47]
    c.lens, c.table, c.T, c.q = c.lens[pick], c.table[pick], c.T[pick], c.q[pick]
    c.q_start = np.arange(4)
    c.check(got[torch.tensor(pick, device=DEV)])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("rows", [24, 60, 120, 256])
@pytest.mark.parametrize("R", [3, 40])
def test_requests_that_join_the_prefix_themselves(R, rows, D):
    """Each number of row tiles, on both sides of a workgroup to a CU."""
    note("prefix joined by requests R=%d rows=%d D=%d" % (R, rows, D))
    Case(rows + D + R, 331, [32 + (i * 37) % 150 for i in range(R)], [rows // 8 - (i % 2) for i in range(R)], H=8, G=8, D=D, page=32).run()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("R", [1, 2, 3, 40])
def test_a_call_that_allows_more_rows_than_it_has(R, D):
    """max_q of 32 where the call's rows are few."""
    c = Case(R + D, 700, [1 + 11 * i for i in range(R)], [1] * R, D=D)
    c.run(max_q=32)
    c.run(max_q=5, max_len=c.cols * c.page)


@pytest.mark.parametrize("G", [1, 2, 4])
def test_more_requests_than_rows(G):
    """64 requests, of which few have a row: before, between and behind idle ones."""
    T = [0] * 64
    for r in (0, 7, 8, 63):
        T[r] = 1
    Case(G, 2003, [20 + 3 * i for i in range(64)], T, H=2, G=G).run()
    Case(G, 2003, [20 + 3 * i for i in range(64)], [0] * 63 + [4], H=3, G=G).run()


# the one line of work; the requests' own kernel joins; a kernel joins
PLANS = [dict(lens=[1, 40, 7], T=[1, 1, 1], G=4), dict(lens=[5 + i for i in range(40)], T=[1] * 40, G=4),
         dict(lens=[3000] * 3 + [5] * 3, T=[3] * 6, G=8, D=256)]


@pytest.mark.parametrize("plan", range(3))
@pytest.mark.parametrize("off", [1, 5])
def test_rows_around_the_requests_are_left(plan, off):
    """q_start[0] above 0, rows behind q_start[R]."""
    c = Case(off, 700, **PLANS[plan])
    a = c.args()
    q = torch.randn((c.M + 2 * off,) + c.q.shape[1:], device=DEV).to(torch.bfloat16)
    q[off: off + c.M] = a["q"]
    out = torch.full(q.shape, 7.0, device=DEV)
    pkg.kv_prefix_attention_run(c.cache(), **dict(a, q=q, q_start=a["q_start"] + off), out=out)
    torch.cuda.synchronize()
    c.check(out[off: off + c.M], f32=True)
    assert torch.all(out[:off] == 7) and torch.all(out[off + c.M:] == 7)


@pytest.mark.parametrize("plan", range(3))
@pytest.mark.parametrize("q_start_of", ["first", "last"])
def test_rows_out_of_order_see_no_prefix(plan, q_start_of):
    """q_start that does not ascend: rows outside q_start[0]..q_start[R] are not held
    against the prefix, and read nothing of its segments."""
    c = Case(plan, 700, **PLANS[plan])
    bad = c.q_start.copy()
    if q_start_of == "first":
        bad[0] = bad[2]  # request 0 has no rows, request 1 lies before the prefix's
        lone, none = [1], [0]
    else:
        bad[-1] = bad[1]  # the last has no rows, those behind the first lie behind the prefix's
        lone, none = list(range(1, len(c.T) - 1)), [len(c.T) - 1]
    out = torch.full(c.q.shape, 7.0, device=DEV)
    pkg.kv_prefix_attention_run(c.cache(), **dict(c.args(), q_start=i32(bad)), out=out)
    torch.cuda.synchronize()
    rows = lambda rs: torch.cat([torch.arange(c.q_start[r], c.q_start[r + 1]) for r in rs]).to(DEV)  # noqa: E731
    assert torch.all(out[rows(none)] == 7)
    def held(rs, P):
        k = rows(rs)
        d = Case(plan, 700, **PLANS[plan])
        d.lens, d.table, d.T, d.q, d.P = c.lens[rs], c.table[rs], c.T[rs], c.q[k.cpu().numpy()], P
        d.q_start = np.concatenate([[0], np.cumsum(d.T)])
        d.check(out[k], f32=True)
    held(lone, 0)
    held([r for r in range(len(c.T)) if r not in lone + none], 700)


def test_the_binding_refuses():
    c = Case(1, 100, [5, 6], [1, 1])
    cache, a = c.cache(), c.args()
    good = dict(a)
    pkg.kv_prefix_attention_run(cache, **good)
    for bad in (dict(prefix_table=a["prefix_table"][None]), dict(prefix_len=i32([1, 2])), dict(prefix_len=a["prefix_len"].long()),
                dict(q=a["q"].float()), dict(lens=a["lens"][:1]), dict(out=torch.empty(1, 8, 128, device=DEV)),
                dict(prefix_table=a["prefix_table"].cpu()), dict(tree_mask=i32([1]))):
        with pytest.raises(ValueError):
            pkg.kv_prefix_attention_run(cache, **{**good, **bad})
    for bad in (dict(max_prefix=-1), dict(max_prefix=100000), dict(max_q=33), dict(max_len=1 << 20), dict(scale=float("inf")),
                dict(workspace=torch.empty(16, dtype=torch.uint8, device=DEV))):
        with pytest.raises(pkg.QGError):
            pkg.kv_prefix_attention_run(cache, **{**good, **bad})
    empty = pkg.kv_prefix_attention_run(cache, **dict(good, q=a["q"][:0]))
    assert empty.shape == (0, 8, 128)
