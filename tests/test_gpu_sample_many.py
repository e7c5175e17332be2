"""GPU: sampling where a call's rows and chunks are many (above 640 workgroups
the borders are found in a kernel of their own): the rows of test_gpu_sample.py's
kinds, against the definition, and over again until they are many, which has to
give every copy the same."""
import numpy as np
import pytest
import torch

import quantized_weight_decode_dequant_amd as pkg
from helpers import note, to_np
from quantized_weight_decode_dequant_amd import workloads
from test_gpu_sample import BF16, DEV, F32, check, logits, run

pytestmark = pytest.mark.gpu
FEW, CHUNK = 640, 4096  # workgroups, tokens of one


def many(x, u, **kw):
    """check() of these rows, and the same of as many copies as it takes, one row behind the other."""
    M, V = x.shape
    chunks = -(-V // CHUNK)
    assert M * chunks <= FEW
    check(x, u, **kw)
    want = run(x, u, **kw)
    n = FEW // (M * chunks) + 1
    got = run(x.repeat(n, 1), np.tile(u, n), **{a: None if v is None else np.tile(v, n) for a, v in kw.items()})
    for a, b in zip(got, want):
        assert np.array_equal(to_np(a).reshape(n, M), np.broadcast_to(to_np(b), (n, M)), equal_nan=True), kw


MIXED = dict(T=[0, 0.5, 1, 1, 1.3, 0.7, 1, 2, 1, 1, 0.8], k=[0, 50, 0, 1, 0, 1000, 7, 20000, 0, 0, 200],
             p=[1, 0.9, 0.95, 1, 0.5, 0.8, 1, 0.9, 1, 1, 1], minp=[0, 0, 0, 0, 0.1, 0.01, 0, 0, 0.2, 0, 0])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("V", [4095, 5003, 33001, 151936])
def test_rows_with_settings_of_their_own(dtype, V):
    """Greedy rows, rows without filters and rows of each filter side by side."""
    note("sample many", V, dtype)
    x = logits(11, V, dtype, 3)
    u = np.random.default_rng(V).random(11).astype(np.float32)
    many(x, u, **MIXED)
    for kw in (dict(), dict(T=MIXED["T"]), dict(k=MIXED["k"]), dict(T=MIXED["T"], p=MIXED["p"]), dict(minp=MIXED["minp"])):
        many(x, u, **kw)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("kw", [dict(p=0.9), dict(T=1.5, p=0.99), dict(k=130), dict(k=5000), dict(T=1.5, k=700, p=0.7), dict(k=100, p=0.95), dict(k=2)])
def test_one_filter(dtype, kw):
    x = logits(6, 20011, dtype, 8)
    many(x, np.random.default_rng(4).random(6).astype(np.float32), **{a: [v] * 6 for a, v in kw.items()})


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("spread", [0.0, 1e-3, 0.3])
def test_flat_rows(dtype, spread):
    """Ties by the thousand: lists that overflow, and cuts through one value."""
    x = logits(6, 20011, dtype, 4, spread, lift=False) + torch.tensor(3.0, dtype=dtype, device=DEV)
    u = np.random.default_rng(1).random(6).astype(np.float32)
    many(x, u, T=[1, 1, 0.01, 1, 5, 1], k=[0, 5000, 0, 12345, 0, 20010], p=[0.5, 1, 0.3, 0.77, 0.001, 0.999], minp=[0, 0, 0, 0, 0, 0.99])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_infinities_nan_and_masks(dtype):
    V, inf = 13001, float("inf")
    x = logits(9, V, dtype, 5)
    x[0] = -inf
    x[1] = float("nan")
    x[2, 1:] = -inf                       # one token left
    x[3, ::3] = float("nan")
    x[4, 7], x[4, 12999] = inf, inf       # two infinite ones, in two chunks
    x[5, 100:] = torch.finfo(dtype).min   # masked by the lowest value
    x[6] = -inf
    x[6, 9500:9510] = -100.0
    x[7, :9000] = -inf                    # whole chunks masked
    x[8, 5:] = float("nan")
    u = np.array([0.3, 0.3, 0.9, 0.6, 0.6, 0.999, 0.55, 0.1, 0.7], np.float32)
    for kw in (dict(), dict(p=[0.9] * 9), dict(k=[3] * 9), dict(k=[3] * 9, p=[0.5] * 9), dict(T=[0.0] * 9), dict(minp=[0.1] * 9),
               dict(k=[12999] * 9), dict(k=[12999] * 9, p=[0.999] * 9), dict(k=[300] * 9),
               dict(T=[1, 0, 1, 2, 1, 0, 1, 0.5, 1], k=[5, 0, 0, 500, 3, 9, 0, 150, 0], p=[0.9, 1, 0.5, 1, 0.9, 1, 0.3, 0.9, 1])):
        many(x, u, **kw)


def test_ends_of_the_parameters():
    x = logits(9, 9001, F32, 6)
    nan, inf = float("nan"), float("inf")
    many(x, np.array([0.0, 1.0, -3.0, 2.0, 0.999999, 0.5, 0.5, 0.5, nan], np.float32), T=[1, 1, 1, 1, 1, inf, 1e-30, 1e30, 1])
    half = np.full(9, 0.5, np.float32)
    many(x, half, T=[-1.0, nan, 1e-45, 1, 1, 1, 1, 1, 1], p=[1, 1, 1, nan, 0, -1, 1e-30, 2, 0.5], minp=[0, 0, 0, 0, 0, 0, 0, nan, 7])
    many(x, half, p=[-inf, -1e-30, -0.3, -1, -3e38, 0, 1e-45, 0.9, inf], k=[0, 0, 300, 50, 0, 9000, 0, 0, 0])
    many(x, half, k=[-5, 0, 9001, 9002, 2 ** 31 - 1, 9000, 1, 2, -2 ** 31])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_strided_rows(dtype):
    """Rows at any alignment, more of them than a call's few."""
    V, M = 4097, 330
    wide = logits(M, 4104, dtype, 9)
    u = np.random.default_rng(2).random(M).astype(np.float32)
    kw = dict(T=np.tile([0.8, 0.0, 1.2], 110), k=np.tile([20, 0, 300, 0, 1], 66), p=np.tile([0.9, 1.0, 0.5, 1.0, 0.99, 1.0], 55))
    for a in (0, 1, 3, 7):
        assert M * 2 > FEW
        check(wide[:, a:a + V], u, **kw)


def test_many_rows_and_the_same_row_twice():
    x = logits(700, 5003, BF16, 12)
    x[350:] = x[:350]
    u = np.tile(np.random.default_rng(3).random(350), 2)
    kw = dict(T=np.tile(np.linspace(0, 2, 350), 2), k=np.tile(np.arange(350) * 7 % 400, 2), p=np.tile(np.linspace(0.3, 1.05, 350), 2))
    got, _ = check(x, u, **kw)
    assert np.array_equal(got[:350], got[350:])
    for _ in range(3):
        again, _ = run(x, u, **kw)
        assert np.array_equal(again.cpu().numpy(), got)


def test_captured():
    """Replays with new inputs, greedy and filtered rows changing places."""
    M, V = 200, 20011
    x, u = torch.zeros(M, V, dtype=BF16, device=DEV), torch.zeros(M, device=DEV)
    T, k, p = torch.ones(M, device=DEV), torch.zeros(M, dtype=torch.int32, device=DEV), torch.ones(M, device=DEV)
    out, logp = torch.zeros(M, dtype=torch.int32, device=DEV), torch.zeros(M, device=DEV)
    ws = torch.empty(pkg.sample_workspace_bytes(M, V), dtype=torch.uint8, device=DEV)
    graph = workloads.capture_graph(lambda: pkg.sample_run(x, u, temperature=T, top_k=k, top_p=p, workspace=ws, tokens=out, logprobs=logp))
    for rep in range(5):
        g = torch.Generator().manual_seed(rep)
        x.copy_(logits(M, V, BF16, rep))
        u.copy_(torch.rand(M, generator=g))
        T.copy_(torch.tensor([0.0, 0.7, 1.0, 1.3])[torch.randint(0, 4, (M,), generator=g)])
        k.copy_(torch.tensor([0, 1, 20, 100, 500], dtype=torch.int32)[torch.randint(0, 5, (M,), generator=g)])
        p.copy_(torch.tensor([1.0, 0.5, 0.95])[torch.randint(0, 3, (M,), generator=g)])
        graph.replay()
        torch.cuda.synchronize()
        want = pkg.sample_run(x, u, temperature=T, top_k=k, top_p=p, logprobs=torch.zeros(M, device=DEV))
        assert torch.equal(out, want[0]) and torch.equal(logp, want[1]), rep
        check(x[:20], to_np(u)[:20], T=to_np(T)[:20], k=k[:20].cpu().numpy(), p=to_np(p)[:20])
        _ = torch.randn(1000, device=DEV).sum().item()
