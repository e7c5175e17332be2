"""GPU: sample_run against its definition by sorting, in 64 bits.

Tokens have to be equal.  The kernel's weights are off by 2^-42 of the row's
largest at most, so a token could differ where u falls within n 2^-42 of a
border among n kept tokens (or a filter's border does): 10^-8 of all u for the
largest rows here, and the inputs are fixed.  Logprobs: fp32's rounding, 2^-24
of the value, and the sums' error, below 2^-24."""
import numpy as np
import pytest
import torch

import step_ref as ref
import quantized_weight_decode_dequant_amd as pkg
from helpers import note, to_np
from quantized_weight_decode_dequant_amd import workloads

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def dev(a, dtype=np.float32):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=dtype)).to(DEV)


def run(x, u, T=None, k=None, p=None, minp=None, **kw):
    logp = torch.full((x.shape[0],), 7.0, device=DEV)
    t, l = pkg.sample_run(x, dev(u), temperature=dev(T), top_k=dev(k, np.int32), top_p=dev(p), min_p=dev(minp),
                          logprobs=logp, **kw)
    torch.cuda.synchronize()
    assert l is logp
    return t, l


def check(x, u, T=None, k=None, p=None, minp=None, **kw):
    f = lambda v: None if v is None else np.asarray(v, np.float32).astype(np.float64)  # noqa: E731
    t, l = run(x, u, T, k, p, minp, **kw)
    want, logp, keeps = ref.sample(to_np(x), f(u), f(T), k, f(p), f(minp))
    got = t.cpu().numpy()
    bad = np.nonzero(got != want)[0]
    assert len(bad) == 0, [(int(m), int(got[m]), int(want[m]), float(u[m]), int(keeps[m].sum())) for m in bad[:5]]
    lg = to_np(l)
    assert np.array_equal(np.isnan(lg), np.isnan(logp))
    ok = ~np.isnan(logp)
    assert np.all(np.abs(lg - logp)[ok] <= 2.0 ** -24 * np.abs(logp[ok]) + 2.0 ** -24)
    return got, keeps


def logits(M, V, dtype, seed, spread=2.2, lift=True):
    g = torch.Generator().manual_seed(seed)
    x = spread * torch.randn(M, V, generator=g)
    if lift:
        at = torch.randint(0, V, (M, min(V, 40)), generator=g)
        x.scatter_add_(1, at, (5 + 3 * torch.rand(at.shape, generator=g)) * (0.2 + torch.rand(M, 1, generator=g)))
    return x.to(dtype).to(DEV)


MODES = {
    "plain": dict(),
    "cold": dict(T=0.4),
    "k": dict(T=0.9, k=50),
    "k2": dict(k=2),
    "p": dict(T=1.1, p=0.9),
    "p small": dict(p=0.05),
    "p near one": dict(p=0.99999),
    "kp": dict(T=0.8, k=40, p=0.9),
    "large k, p": dict(T=1.5, k=700, p=0.7),
    "minp": dict(T=1.3, minp=0.05),
    "all": dict(T=1.2, k=100, p=0.95, minp=0.02),
    "k of nearly all": dict(T=2.0, k=-1, p=0.5),
}


@pytest.mark.parametrize("V", [1, 2, 17, 255, 4095, 4097, 8192, 33001])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("mode", list(MODES))
def test_filters(V, dtype, mode):
    note("sample", V, dtype, mode)
    M = 5
    x = logits(M, V, dtype, V)
    g = np.random.default_rng(V)
    kw = {n: np.full(M, v if (n, v) != ("k", -1) else max(V - 3, 1)) for n, v in MODES[mode].items()}
    check(x, g.random(M), **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [151936, 262144])
def test_whole_vocabularies_with_settings_of_their_own(dtype, V):
    M = 9
    x = logits(M, V, dtype, 3)
    g = np.random.default_rng(V)
    check(x, g.random(M), T=[0, 0.5, 1, 1, 1.3, 0.7, 1, 2, 1], k=[0, 50, 0, 1, 0, 1000, 7, 100000, 0],
          p=[1, 0.9, 0.95, 1, 0.5, 0.8, 1, 0.9, 1], minp=[0, 0, 0, 0, 0.1, 0.01, 0, 0, 0.2])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.3])
def test_flat_rows(dtype, spread):
    """Ties by the thousand: a border's bin holds far more tokens than a list."""
    M, V = 6, 20011
    x = logits(M, V, dtype, 4, spread, lift=False) + torch.tensor(3.0, dtype=dtype, device=DEV)
    g = np.random.default_rng(1)
    check(x, g.random(M), T=[1, 1, 0.01, 1, 5, 1], k=[0, 5000, 0, 12345, 0, 20010], p=[0.5, 1, 0.3, 0.77, 0.001, 0.999],
          minp=[0, 0, 0, 0, 0, 0.99])


def test_ties_go_to_the_lower_token():
    x = torch.zeros(4, 9000, device=DEV)
    x[:, 5000:] = 1.0
    kept = 3
    got, keeps = check(x, [0.0, 0.34, 0.99, 0.5], T=[1, 1, 1, 0], k=[kept] * 4)
    assert got.tolist() == [5000, 5001, 5002, 5000]
    # over the border of two chunks: all of the larger, and the first of the others
    x = torch.zeros(3, 9000, device=DEV)
    x[:, 8190:8194] = 1.0
    got, _ = check(x, [0.0, 0.999999, 0.7], k=[6, 6, 6])
    assert got.tolist() == [0, 8193, 8192]


def test_negative_and_mixed_zeros():
    x = torch.full((2, 5000), -0.0, device=DEV)
    x[:, ::2] = 0.0
    x[:, 4000:] = -3.0
    check(x, [0.1, 0.9], k=[777, 777])
    check(x.bfloat16(), [0.1, 0.9], k=[777, 777], p=[0.5, 0.7])
    check(-4 - logits(3, 6000, BF16, 8).abs(), [0.2, 0.5, 0.8], k=[100, 300, 5], p=[0.9] * 3)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinities_nan_and_masks(dtype):
    V = 5001
    x = logits(8, V, dtype, 5)
    inf = float("inf")
    x[0] = -inf
    x[1] = float("nan")
    x[2, 1:] = -inf                       # one token left
    x[3, ::3] = float("nan")
    x[4, 7], x[4, 4999] = inf, inf        # two infinite ones
    x[5, 100:] = torch.finfo(dtype).min   # masked by the lowest value
    x[6] = -inf
    x[6, 4500:4510] = -100.0
    x[7, :4000] = -inf
    u = np.array([0.3, 0.3, 0.9, 0.6, 0.6, 0.999, 0.55, 0.1])
    for kw in (dict(), dict(p=[0.9] * 8), dict(k=[3] * 8), dict(k=[3] * 8, p=[0.5] * 8), dict(T=[0.0] * 8), dict(minp=[0.1] * 8),
               dict(k=[4999] * 8), dict(k=[4999] * 8, p=[0.999] * 8)):
        got, _ = check(x, u, **kw)
        assert got[0] == -1 and got[1] == -1 and got[2] == 0 and got[4] in (7, 4999) and got[5] < 100


def test_ends_of_the_parameters():
    x = logits(9, 3001, F32, 6)
    nan, inf = float("nan"), float("inf")
    check(x, [0.0, 1.0, -3.0, 2.0, 0.999999, 0.5, 0.5, 0.5, nan], T=[1, 1, 1, 1, 1, inf, 1e-30, 1e30, 1])
    check(x, [0.5] * 9, T=[-1.0, nan, 1e-45, 1, 1, 1, 1, 1, 1], p=[1, 1, 1, nan, 0, -1, 1e-30, 2, 0.5],
          minp=[0, 0, 0, 0, 0, 0, 0, nan, 7])
    check(x, [0.5] * 9, k=[-5, 0, 3001, 3002, 2 ** 31 - 1, 3000, 1, 2, -2 ** 31])
    huge = x * 1e37
    check(huge, np.linspace(0, 0.99, 9), T=[1, 1e37, 1e38, 3e38, 1, 1e36, 1, 1, 1], p=[1, 1, 0.9, 1, 1, 1, 1, 1, 1], k=[0, 0, 0, 9, 0, 5, 0, 0, 0])


def test_the_draws_follow_the_distribution():
    """One row, u on an even grid: each token as often as its share says, to within one."""
    x = logits(1, 700, F32, 7)
    n = 4096
    u = (np.arange(n) + 0.5) / n
    for kw in (dict(), dict(k=12), dict(p=0.8), dict(T=2.0, minp=0.05)):
        rows = x.expand(n, 700)
        t, _ = run(rows.contiguous(), u, **{a: np.full(n, b) for a, b in kw.items()})
        got = np.bincount(t.cpu().numpy(), minlength=700)
        _, _, keeps = ref.sample(to_np(x), np.array([0.5]), **{a: np.full(1, np.float32(b)) for a, b in kw.items()})
        w = np.exp((to_np(x)[0] - to_np(x)[0].max()) / kw.get("T", 1.0)) * keeps[0]
        assert np.all(np.abs(got - n * w / w.sum()) <= 1 + 1e-6)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_and_unaligned_rows(dtype):
    wide = logits(6, 9001, dtype, 9)
    g = np.random.default_rng(2)
    for a, b in ((0, 5000), (1, 4097), (3, 8999), (8, 9001), (5, 6)):
        x = wide[:, a:b]
        check(x, g.random(6), T=[0.8] * 6, k=[20] * 6, p=[0.9] * 6)
        check(x, g.random(6))
    check(wide[::2], g.random(3), p=[0.6] * 3)


def test_no_rows():
    t, l = pkg.sample_run(torch.empty(0, 50, device=DEV), torch.empty(0, device=DEV))
    assert t.shape == (0,) and l is None


def test_captured_graphs_and_streams():
    """Two graphs with a workspace each, replayed in turn with new inputs, equal the eager calls."""
    M, V = 4, 30011
    xs, us = [torch.zeros(M, V, dtype=BF16, device=DEV) for _ in range(2)], [torch.zeros(M, device=DEV) for _ in range(2)]
    T, k, p = dev([0.8, 1.0, 0.0, 1.2]), dev([50, 0, 0, 300], np.int32), dev([0.9, 0.95, 1.0, 1.0])
    outs = [torch.zeros(M, dtype=torch.int32, device=DEV) for _ in range(2)]
    ws = [torch.empty(pkg.sample_workspace_bytes(M, V), dtype=torch.uint8, device=DEV) for _ in range(2)]
    graphs = [workloads.capture_graph(lambda i=i: pkg.sample_run(xs[i], us[i], temperature=T, top_k=k, top_p=p, workspace=ws[i], tokens=outs[i]))
              for i in range(2)]
    for rep in range(6):
        for i in range(2):
            xs[i].copy_(logits(M, V, BF16, 10 * rep + i))
            us[i].copy_(torch.rand(M, generator=torch.Generator().manual_seed(rep + 50 * i)))
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            want, _ = pkg.sample_run(xs[i], us[i], temperature=T, top_k=k, top_p=p)
            assert torch.equal(outs[i], want), (rep, i)
        _ = torch.randn(1000, device=DEV).sum().item()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    torch.cuda.synchronize()
    for i in range(2):
        got.append(pkg.sample_run(xs[i], us[i], temperature=T, top_k=k, top_p=p, stream=streams[i])[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, outs))


def test_many_rows_and_the_same_row_twice():
    """Rows do not depend on each other, and every run gives the same."""
    x = logits(300, 5003, BF16, 12)
    x[150:] = x[:150]
    u = np.tile(np.random.default_rng(3).random(150), 2)
    kw = dict(T=np.tile(np.linspace(0.2, 2, 150), 2), k=np.tile(np.arange(150) * 7 % 400, 2), p=np.tile(np.linspace(0.3, 1.05, 150), 2))
    got, _ = check(x, u, **kw)
    assert np.array_equal(got[:150], got[150:])
    for _ in range(3):
        again, _ = run(x, u, **kw)
        assert np.array_equal(again.cpu().numpy(), got)


def test_the_binding_refuses():
    x, u = logits(4, 100, F32, 1), torch.rand(4, device=DEV)
    good = dict(logits=x, u=u)
    pkg.sample_run(**good)
    for bad in (dict(logits=x.half()), dict(logits=x.t()), dict(logits=x[0]), dict(u=u[:3]), dict(u=u.double()), dict(u=u.cpu()),
                dict(top_k=u), dict(top_p=u[:, None]), dict(temperature=torch.ones(1, device=DEV)), dict(min_p=0.1 * torch.ones(5, device=DEV)),
                dict(tokens=torch.empty(4, dtype=torch.int64, device=DEV)), dict(logprobs=torch.empty(4, dtype=BF16, device=DEV))):
        with pytest.raises(ValueError):
            pkg.sample_run(**{**good, **bad})
    with pytest.raises(pkg.QGError) as e:
        pkg.sample_run(x, u, workspace=torch.empty(64, dtype=torch.uint8, device=DEV))
    assert e.value.status == pkg.QG_ESIZE


@pytest.mark.parametrize("fill", [float("-inf"), -3e38, -1e4])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masks_that_leave_fewer_tokens_than_a_filter_asks_for(fill, dtype):
    """A grammar's mask: 30 of 40001 tokens left, top-k 50: they all stay in, and nothing masked is drawn."""
    M, V = 6, 40001
    x = torch.full((M, V), fill).to(dtype)
    g = torch.Generator().manual_seed(2)
    at = torch.stack([torch.randperm(V, generator=g)[:30] for _ in range(M)])
    x.scatter_(1, at, (3 * torch.randn(M, 30, generator=g)).to(dtype))
    u = np.random.default_rng(5).random(M)
    u[0] = 0.9999999
    for kw in (dict(k=[50] * M), dict(k=[50] * M, p=[0.9] * M), dict(p=[0.999999] * M), dict(), dict(k=[30] * M, p=[0.5] * M), dict(k=[31] * M, minp=[0.01] * M)):
        got, _ = check(x.to(DEV), u, **kw)
        assert all(int(got[m]) in at[m] for m in range(M))


def test_tokens_far_below_the_largest():
    """Weights around the last one that counts, 2^-44 of the largest, at many temperatures."""
    x = torch.linspace(0, -60, 5000)[None].repeat(6, 1).to(DEV)
    u = np.array([0.0, 0.5, 0.9, 0.99999, 0.9999999, 1.0])
    for T in (0.05, 0.5, 1.0, 1.9, 3.0):
        for kw in (dict(), dict(k=[4900] * 6), dict(k=[4900] * 6, p=[0.9999] * 6), dict(p=[0.99] * 6)):
            # (what lies below changes no sum by more than 2^-31 of it)
            check(x, np.minimum(u, 1 - 2.0 ** -22), T=[T] * 6, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.3, 2.2])
@pytest.mark.parametrize("M", [6, 140])
def test_top_p_under_a_small_top_k(dtype, spread, M):
    """On both sides of the size whose tokens are all listed, ties by the thousand."""
    V = 20011
    x = logits(M, V, dtype, 5, spread, lift=spread > 1) + torch.tensor(3.0, dtype=dtype, device=DEV)
    g = np.random.default_rng(M)
    check(x, g.random(M), T=g.choice([0.3, 0.8, 1.0, 4.0], M), k=g.choice([2, 3, 50, 99, 100, 101, 128, 129], M),
          p=g.choice([1e-6, 0.3, 0.9, 0.9999], M), minp=g.choice([0, 0, 0.05], M))


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_small_top_k_over_few_or_infinite_tokens(dtype):
    M, V = 8, 9001
    x = torch.full((M, V), float("-inf"), dtype=dtype, device=DEV)
    at = torch.arange(0, V, 300, device=DEV)
    x[:4, at] = logits(4, len(at), dtype, 6, lift=False)  # 31 tokens
    x[2, at[5]] = x[4, 17] = float("nan")
    x[3, at] = 1.0
    x[5, at] = float("inf")
    x[6, 8000] = float("inf")
    x[7, 3] = -3e38
    for p in (0.2, 0.95):
        for k in (2, 30, 31, 32, 100):
            check(x, np.linspace(0, 0.999, M), T=[0.7] * M, k=[k] * M, p=[p] * M)
