"""GPU: rotation, attention behind a shared prefix and sampling at the largest
numbers of heads, requests, rows and tokens that a call may have."""
import numpy as np
import pytest
import torch

import step_ref as ref
import quantized_weight_decode_dequant_amd as pkg
from helpers import note, to_np
from test_gpu_kv_prefix import Case
from test_gpu_qk_rope import BF16, F32, check as check_rope, freqs, make
from test_gpu_sample import check as check_sample, logits, run as run_sample

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("M,Hq,Hkv,D,dtype", [(1, 8192, 1024, 8, BF16), (3, 8192, 1, 8, F32), (1, 1, 1024, 64, BF16), (70001, 2, 1, 8, BF16), (1, 700, 60, 512, F32)])
def test_rotation(M, Hq, Hkv, D, dtype):
    note("rope ends", M, Hq, Hkv, D)
    q, k, qw, kw = make(M, Hq, Hkv, D, dtype)
    rotated = D // 16 * 16
    p, f = torch.arange(M, dtype=torch.int32, device=DEV), freqs(rotated)
    qo, ko = pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw, k_weight=kw)
    torch.cuda.synchronize()
    check_rope(qo, q, qw, 1e-6, p, None, f, False)
    check_rope(ko, k, kw, 1e-6, p, None, f, False)


@pytest.mark.parametrize("H,G,R,T", [(1024, 1, 1, 1), (1024, 8, 1, 2), (1, 8192, 1, 1), (1, 1024, 3, 2), (1, 1, 4096, 1), (1, 2, 4096, 2)])
def test_prefix_heads_and_requests(H, G, R, T):
    note("prefix ends", H, G, R, T)
    g = np.random.default_rng(R)
    lens, n = (g.integers(T, 40, R), g.integers(0, T + 1, R)) if R > 3 else (np.full(R, 50), np.full(R, T))
    n[-1] = T
    c = Case(H + R, 90, list(lens), list(n), H=H, G=G, D=64, page=32)
    c.run()


def test_a_long_prefix():
    """Pages of a small pool, over and over; few rows, and many."""
    pool, page, cols = 300, 256, 1024
    for R, G in ((2, 2), (40, 1)):
        c = Case(R, page * pool, [3] * R, [1] * R, H=1, G=G, D=64, page=page)
        c.prefix = c.g.permutation(np.resize(c.prefix[:pool], cols))
        c.P = page * cols - 77
        a = c.args()
        for max_prefix in (None, c.P):
            got = pkg.kv_prefix_attention_run(c.cache(), max_prefix=max_prefix, **a)
            torch.cuda.synchronize()
            d = object.__new__(Case)
            d.__dict__.update(c.__dict__)
            rows = [0, R - 1]
            d.lens, d.table, d.T, d.q, d.q_start = c.lens[rows], c.table[rows], c.T[rows], c.q[rows], np.arange(3)
            d.check(got[torch.tensor(rows, device=DEV)])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_sampling(dtype):
    g = np.random.default_rng(1)
    check_sample(logits(2, 1 << 20, dtype, 1), g.random(2), T=[0.7, 1.3], k=[50, 0], p=[0.9, 0.8], minp=[0, 0.001])
    check_sample(logits(3, (1 << 20) - 1, dtype, 2), g.random(3), T=[0, 1, 1], k=[0, 300000, 0], p=[1, 1, 0.999])
    for V in (1, 3, 100):
        M = 5000
        x = logits(M, V, dtype, V)
        check_sample(x, g.random(M), T=g.choice([0, 0.5, 1.0], M), k=g.choice([0, 1, 2, 50], M), p=g.choice([1.0, 0.5], M))
    x = torch.zeros(2, 1 << 20, dtype=dtype, device=DEV)  # every token alike: masses sum to 2^62
    u = np.array([0.0, 0.75], np.float32)
    for kw in (dict(), dict(p=[0.5, 0.5]), dict(k=[1 << 19] * 2)):
        t, _ = run_sample(x, u, **kw)
        kept = (1 << 20) if not kw else 1 << 19
        assert t.tolist() == [0, int(0.75 * kept)]
