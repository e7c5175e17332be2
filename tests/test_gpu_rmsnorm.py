"""GPU: the root-mean-square norm with residual, bf16 and int8 outputs,
against its definition in 64 bits.

Tolerances.  residual_out is one fp32 addition rounded to its type: exact.
The codes are decided in fp64 from r * weight: exact.  y is one rounding to
bf16 (half a step, 2^-8) of a value whose relative error is that of the fp32
sum of squares (serial sums of at most 24 terms, a tree of 6 + 16: below
2^-18) and a few fp32 operations; scales carry the same without the bf16 step."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import oracle
import quantized_weight_decode_dequant_amd as pkg
from helpers import note, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
FP32_PART = 2.0 ** -17


def inputs(seed, M, K, xt, rt, spread=20.0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((M, K))
    x[:, :: max(1, K // 5)] *= spread
    x = torch.from_numpy(x).to(xt)
    res = None if rt is None else torch.from_numpy(2 * g.standard_normal((M, K))).to(rt)
    w = torch.from_numpy(1 + 0.2 * g.standard_normal(K)).to(torch.bfloat16)
    signs = torch.from_numpy((g.integers(0, 2, K) * 2 - 1).astype(np.int8))
    return x, res, w, signs


def check(x, res, w, signs, y, q, eps=1e-6, alias=False):
    M, K = x.shape
    dx, dr, dw, ds = (None if t is None else t.to(DEV) for t in (x, res, w, signs))
    out = None if res is None else (dr if alias else torch.empty_like(dr))
    yt = torch.empty(M, K, dtype=torch.bfloat16, device=DEV) if y else None
    Xq = torch.empty(M, K, dtype=torch.int8, device=DEV) if q else None
    sc = torch.empty(M, device=DEV) if q else None
    pkg.rmsnorm_quant_run(dx, dw, eps, residual=dr, residual_out=out, signs=ds, y=yt, Xq=Xq, x_scales=sc)
    torch.cuda.synchronize()
    r64, y64, q64, s64 = ref.norm(to_np(x), to_np(w), np.float64(np.float32(eps)), None if res is None else to_np(res),
                                  None if signs is None else to_np(signs))
    if res is not None:
        want = (x.float() + res.float()).to(res.dtype)
        assert torch.equal(out.cpu(), want)
    if y:
        tol = (2.0 ** -8 + FP32_PART) * np.abs(y64) + 1e-38
        assert np.all(np.abs(to_np(yt) - y64) <= tol), np.max(np.abs(to_np(yt) - y64) / tol)
    if q:
        assert np.array_equal(Xq.cpu().numpy(), q64), np.argwhere(Xq.cpu().numpy() != q64)[:4]
        assert np.all(np.abs(to_np(sc) - s64) <= FP32_PART * s64)


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rt", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("y,q,rot", [(1, 0, 0), (0, 1, 0), (1, 1, 0), (0, 1, 1), (1, 1, 1)])
def test_types_and_outputs(xt, rt, y, q, rot):
    note("rmsnorm", xt, rt, y, q, rot)
    x, res, w, signs = inputs(1, 5, 4128, xt, rt)
    check(x, res, w, signs if rot else None, y, q)


@pytest.mark.parametrize("M,K", [(1, 32), (3, 64), (1, 96), (2, 992), (1, 4096), (33, 2080), (2, 8192), (2, 8224),
                                 (3, 12288), (1, 16416), (2, 24576), (1031, 96), (70, 7168)])
@pytest.mark.parametrize("rot", [0, 1])
def test_sizes(M, K, rot):
    note("rmsnorm M=%d K=%d rot=%d" % (M, K, rot))
    x, res, w, signs = inputs(M * 100003 + K, M, K, torch.bfloat16, torch.bfloat16)
    check(x, res, w, signs if rot else None, 1, 1, alias=True)


@pytest.mark.parametrize("M,K", [(512, 4128), (511, 4128), (601, 8192), (513, 8224)])
@pytest.mark.parametrize("rot", [0, 1])
def test_many_long_rows(M, K, rot):
    """Rows whose threads hold four units, and the sizes beside them."""
    note("rmsnorm M=%d K=%d rot=%d" % (M, K, rot))
    x, res, w, signs = inputs(M * 100003 + K, M, K, torch.bfloat16, torch.bfloat16)
    check(x, res, w, signs if rot else None, 1, 1, alias=True)


def test_ties_zero_rows_and_one_value():
    """Codes that land on .5 (ties to even), a row of zeros, a row with one
    value, a row of equal values."""
    K = 96
    x = np.zeros((4, K))
    x[0, :5] = [254, 1, 3, -5, 7]       # 127, .5 -> 0, 1.5 -> 2, -2.5 -> -2, 3.5 -> 4
    x[2, 77] = -3.0
    x[3] = 0.25
    x = torch.from_numpy(x).to(torch.bfloat16)
    w = torch.ones(K, dtype=torch.bfloat16)
    check(x, None, w, None, 1, 1)
    Xq, sc = pkg.rmsnorm_quant_run(x.to(DEV), w.to(DEV), 1e-6)[2:]
    assert Xq[0, :5].tolist() == [127, 0, 2, -2, 4]
    assert not Xq[1].any() and float(sc[1]) == 0.0


@pytest.mark.parametrize("K", [64, 4128])
def test_tiny_values(K):
    """Rows whose products underflow in fp32, or lose bits there, beside
    ordinary ones; weights that are 0."""
    g = np.random.default_rng(K)
    x = g.standard_normal((7, K)) * np.array([1e-20, 1e-30, 1e-36, 3e-38, 1e-38, 0.0, 1.0])[:, None]
    w = torch.from_numpy(g.standard_normal(K) * np.where(np.arange(K) % 3 == 0, 1e-9, 1.0)).to(torch.bfloat16)
    w[::5] = 0.0
    x = torch.from_numpy(x).to(torch.bfloat16)
    for M in (7, 600):
        xx = x.repeat((M + 6) // 7, 1)[:M]
        Xq, sc = pkg.rmsnorm_quant_run(xx.to(DEV), w.to(DEV), 1e-30)[2:]
        torch.cuda.synchronize()
        _, _, q64, s64 = ref.norm(to_np(xx), to_np(w), np.float64(np.float32(1e-30)))
        assert np.array_equal(Xq.cpu().numpy(), q64), np.argwhere(Xq.cpu().numpy() != q64)[:4]
        big = s64 > 1e-30  # (the sum of squares of smaller rows underflows in fp32: eps decides)
        assert np.all(np.abs(to_np(sc) - s64)[big] <= FP32_PART * s64[big])
    Xq, sc = pkg.rmsnorm_quant_run((x * 0 + 1e-30).to(DEV), (w * 0 + 1e-20).to(DEV), 1e-6)[2:]
    assert bool((Xq == 127).all())  # every product is 0 in fp32


def test_rows_that_are_not_finite_stay_alone():
    x, res, w, _ = inputs(3, 4, 256, torch.bfloat16, torch.bfloat16)
    x[1, 17] = float("nan")
    x[2, 200] = float("inf")
    dx, dr, dw = x.to(DEV), res.to(DEV), w.to(DEV)
    y = torch.empty_like(dx)
    _, _, Xq, sc = pkg.rmsnorm_quant_run(dx, dw, 1e-6, residual=dr, y=y, Xq=torch.empty(4, 256, dtype=torch.int8, device=DEV))
    assert torch.isnan(sc[1:3]).all() and not Xq[1:3].any()
    clean = torch.tensor([0, 3], device=DEV)
    y2 = torch.empty(2, 256, dtype=torch.bfloat16, device=DEV)
    _, _, q2, s2 = pkg.rmsnorm_quant_run(dx[clean], dw, 1e-6, residual=dr[clean], y=y2, Xq=torch.empty(2, 256, dtype=torch.int8, device=DEV))
    assert torch.equal(y[clean], y2) and torch.equal(Xq[clean], q2) and torch.equal(sc[clean], s2)


def test_feeds_the_int8_product():
    """The codes and scales go straight into the 8-bit verification product."""
    from quantized_weight_decode_dequant_amd import synth, weights
    M, K, N = 16, 512, 100
    x, res, w, signs = inputs(5, M, K, torch.float32, torch.float32)
    Xq, sc = pkg.rmsnorm_quant_run(x.to(DEV), w.to(DEV), 1e-5, residual=res.to(DEV), signs=signs.to(DEV))[2:]
    m = synth.q8_matrix(6, N, K)
    Y = pkg.qgemm_skinny_run(pkg.FMT_Q8_SYM_G32, weights.pack_q8(m, DEV), M, N, K, Xq, sc, out_dtype=pkg.OUT_F32)
    torch.cuda.synchronize()
    _, _, q64, s64 = ref.norm(to_np(x), to_np(w), np.float64(np.float32(1e-5)), to_np(res), to_np(signs))
    want = oracle.q8_gemm(m.qw, m.sw, q64, s64.astype(np.float32))
    # fp32 sums of K products and scales off by FP32_PART
    lim = (FP32_PART + K * 2.0 ** -24) * np.abs(want) + K * 2.0 ** -24 * np.abs(want).max()
    assert np.all(np.abs(to_np(Y) - want) <= lim)


def test_other_stream_and_graph():
    from quantized_weight_decode_dequant_amd import workloads
    x, res, w, signs = inputs(7, 9, 1024, torch.bfloat16, torch.bfloat16)
    dx, dr, dw, ds = (t.to(DEV) for t in (x, res, w, signs))
    bufs = [torch.empty_like(dr), torch.empty_like(dx), torch.empty(9, 1024, dtype=torch.int8, device=DEV), torch.empty(9, device=DEV)]

    def run(b):
        pkg.rmsnorm_quant_run(dx, dw, 1e-6, residual=dr, residual_out=b[0], signs=ds, y=b[1], Xq=b[2], x_scales=b[3])

    graph = workloads.capture_graph(lambda: run(bufs))
    eager = [torch.empty_like(b) for b in bufs]
    for rep in range(4):
        dx.copy_(inputs(8 + rep, 9, 1024, torch.bfloat16, None)[0])
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run(eager)
        torch.cuda.current_stream().wait_stream(s)
        for b in bufs:
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, eager)), rep


@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("K", [64, 4128, 8224])
def test_products_past_fp32(K, res, xt):
    """Rows whose sum of squares is finite and whose products with the weight
    are not (in fp32): just past its end, far past it, and ordinary rows of
    the same call.  The codes are the definition's."""
    g = np.random.default_rng(K)
    x = g.standard_normal((7, K)) * np.array([1e17, 1e16, 5e16, 1.0, 1e12, 0.0, 1e-3])[:, None]
    w = g.standard_normal(K) * np.where(np.arange(K) % 3 == 0, 1e22, np.where(np.arange(K) % 7 == 0, 1e30, 1.0))
    x, w = torch.from_numpy(x).to(xt), torch.from_numpy(w).to(torch.bfloat16)
    r = torch.from_numpy(0.1 * to_np(x) * g.standard_normal((7, K))).to(xt) if res else None
    with np.errstate(over="ignore"):
        p = (to_np(x) + (to_np(r) if res else 0)).astype(np.float32) * to_np(w).astype(np.float32)
    assert np.isinf(p).any(1).tolist() == [True, True, True, False, True, False, False]
    for M in (7, 600):
        rep = lambda t: None if t is None else t.repeat((M + 6) // 7, 1)[:M]  # noqa: E731
        check(rep(x), rep(r), w, None, 1, 1)
