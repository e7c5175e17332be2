"""GPU: attention behind a shared prefix where numbers come near their types'
ends, or far apart, in each kernel that reads the prefix; limits and tolerances
are those of the requests' attention (test_gpu_kv_attention.py)."""
import numpy as np
import pytest
import torch

import cache_ref
import step_ref as ref
import quantized_weight_decode_dequant_amd as pkg
from helpers import note, to_np
from test_gpu_kv_prefix import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
FMTS = [pkg.KV_INT8, pkg.KV_E4M3]
# (requests, new tokens, heads to a KV head, D): one line with the requests; one
# and two row tiles a wave, heads of 256 in four and eight waves
KERNELS = [(2, 1, 4, 64), (3, 1, 4, 256), (10, 1, 4, 64), (10, 1, 4, 128), (30, 2, 4, 128), (8, 1, 8, 256), (30, 1, 4, 256)]


def bits(values, fmt):
    return values.astype(np.int8).view(np.uint8) if fmt == pkg.KV_INT8 else cache_ref.e4m3_bits(np.asarray(values, np.float64))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("qexp,scale,kexp", [(122, None, -104), (120, -1.0, -100), (0, 2.0 ** 118, -104), (-100, 2.0 ** 126, -20), (90, 1.37, -2.3),
                                             (20, 1.37, 12.3), (14, 0.711, 9.7), (9, -1.13, 8.9), (5, 0.9, 6.3)])
@pytest.mark.parametrize("R,T,G,D", KERNELS)
def test_large_scores(R, T, G, D, qexp, scale, kexp, fmt):
    """Scores from 2^19 to near fp32's end: the token of the largest score, of the
    prefix or of the request, is all of the softmax."""
    note("prefix large scores", R, T, G, D, qexp, scale, kexp, fmt)
    P, n = 700, 40
    c = Case(R + D, P, [n] * R, [T] * R, H=1, G=G, D=D, page=32, fmt=fmt)
    c.q = np.full(c.q.shape, 1.25 * 2.0 ** qexp)
    c.ks[:] = 2.0 ** kexp
    first, second = (3.0, -3.0) if (scale or 1.0) > 0 else (-3.0, 3.0)
    dec = cache_ref.e4m3_value if fmt == pkg.KV_E4M3 else (lambda b: b.view(np.int8).astype(np.float64))
    for at in (17, 333, 699, None):  # of the prefix; of the request
        c.k[:] = bits(np.zeros(c.k.shape), fmt)
        c.k[c.prefix[5], 0, 3] = bits(np.full(D, second), fmt)
        place = [(c.table[r, 0], 9) if at is None else (c.prefix[at // 32], at % 32) for r in range(R)]
        for p, o in place:
            c.k[p, 0, o] = bits(np.full(D, first), fmt)
        got = to_np(pkg.kv_prefix_attention_run(c.cache(), scale=scale, **c.args()))
        torch.cuda.synchronize()
        for r, (p, o) in enumerate(place):
            want = dec(np.ascontiguousarray(c.v[p, 0, o])) * float(c.vs[p, 0])
            # the other tokens are below 2^-1000 of it; f16's and bf16's half steps
            tol = (2.0 ** -8 + 2.0 ** -11 + 2.0 ** -19) * np.abs(want) + 64 * 2.0 ** -24 * 448 * float(c.vs.max())
            mine = got[c.q_start[r]: c.q_start[r + 1]]
            assert np.all(np.abs(mine - want) <= tol), (at, r, float(np.abs(mine).max()))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("exp", [118, 100, -107])
@pytest.mark.parametrize("R,T,G,D", KERNELS)
def test_values_near_the_ends_of_fp32(R, T, G, D, exp, fmt):
    """The mean of all tokens (scores of 0), of values whose sums pass fp32's range, and of the smallest."""
    c = Case(R + D, 1500, [40] * R, [T] * R, H=1, G=G, D=D, page=32, fmt=fmt)
    c.q[:] = 0.0
    v = 60 + c.g.integers(0, 60, c.v.shape)
    c.v = bits(v, fmt)
    c.vs = ((0.5 + 0.5 * c.g.random(c.vs.shape)) * 2.0 ** exp).astype(np.float32)
    for dt in (pkg.OUT_BF16, pkg.OUT_F32):
        got = pkg.kv_prefix_attention_run(c.cache(), out_dtype=dt, **c.args())
        torch.cuda.synchronize()
        c.check(got, f32=dt == pkg.OUT_F32)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,T,G,D", KERNELS)
@pytest.mark.parametrize("where", ["prefix", "request"])
def test_weight_on_pages_of_small_scale(where, R, T, G, D, fmt):
    """All of a row's weight lies on a page whose value scale is 1.3 * 2^-20
    beside one of scale 1 that every row scores far below it: within the prefix,
    and in the request behind a prefix of scale 1."""
    c = Case(R + D, 64, [32] * R, [T] * R, H=1, G=G, D=D, page=32, fmt=fmt)
    c.q = to_np(torch.from_numpy(np.abs(c.q) + 1.0).to(torch.bfloat16))
    low = bits(np.full(D, -100.0 if fmt == pkg.KV_INT8 else -448.0), fmt)
    near = [int(c.prefix[1])] if where == "prefix" else [int(p) for p in c.table[:, 0]]
    c.k[:] = low
    c.k[near] = bits(np.zeros(D), fmt)
    c.ks[:] = 0.1
    c.vs[:] = 1.0
    c.vs[near] = 1.3 * 2.0 ** -20
    got = pkg.kv_prefix_attention_run(c.cache(), out_dtype=pkg.OUT_F32, **c.args())
    torch.cuda.synchronize()
    o, A, _ = ref.prefix_attention(c.k, c.v, c.ks.astype(np.float64), c.vs.astype(np.float64), fmt == pkg.KV_E4M3, c.q, c.q_start, c.lens,
                                   c.table, c.prefix, c.P)
    # the equal probabilities are normal in f16: half a step is 2^-11 of each, so of the
    # output; fp32 sums of 96 products, the scales, exp2 and the joins
    assert np.all(np.abs(to_np(got) - o) <= (2.0 ** -11 + 96 * 2.0 ** -24 + 2.0 ** -19) * A)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("R,T,G,D", KERNELS)
def test_first_pages_without_values(R, T, G, D, fmt):
    """The first 130 pages of the prefix are not there, or hold only zeros; the others' scales are small."""
    c = Case(R + D, 32 * 200, [9] * R, [T] * R, H=1, G=G, D=D, page=32, fmt=fmt)
    c.vs = ((0.3 + c.g.random(c.vs.shape)) * 2.0 ** -20).astype(np.float32)
    keep = c.prefix.copy()
    for zero in (False, True):
        c.prefix = keep.copy()
        c.prefix[:130] = keep[0] if zero else -1
        c.vs[keep[0]] = 0.0
        c.run()


@pytest.mark.parametrize("R,T,G,D", KERNELS)
def test_rows_depend_on_no_other_rows(R, T, G, D):
    """Bit-equal whatever the other requests' queries and pages hold: NaN, infinity, queries of 2^100."""
    c = Case(R + D, 900, [20 + i for i in range(R)], [T] * R, H=2, G=G, D=D, page=32)
    a = c.args()
    first = pkg.kv_prefix_attention_run(c.cache(), **a)
    r = R // 2
    mine = slice(int(c.q_start[r]), int(c.q_start[r + 1]))
    kept = set(int(p) for p in c.prefix) | set(int(p) for p in c.table[r])
    others = np.array([p not in kept for p in range(c.pages)])
    c.k[others], c.vs[others] = 77, c.vs[others] * 1000
    for fill in (float("nan"), float("inf"), 2.0 ** 100, 0.0):
        q = torch.full_like(a["q"], fill)
        q[mine] = a["q"][mine]
        got = pkg.kv_prefix_attention_run(c.cache(), **dict(a, q=q))
        torch.cuda.synchronize()
        assert torch.equal(got[mine], first[mine]), fill
        if fill != fill or fill == float("inf"):
            assert bool(got[: mine.start].isnan().all()) and bool(got[mine.stop:].isnan().all())


@pytest.mark.parametrize("R,T,G,D", KERNELS)
def test_same_every_time(R, T, G, D):
    c = Case(R + D, 5003, [20 + 9 * i for i in range(R)], [T] * R, H=2, G=G, D=D, page=64)
    a, cache = c.args(), c.cache()
    first = pkg.kv_prefix_attention_run(cache, **a)
    for _ in range(5):
        assert torch.equal(pkg.kv_prefix_attention_run(cache, **a), first)
