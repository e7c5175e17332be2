"""Rotation, shared-prefix attention and sampling where byte offsets pass 32 bits:
the same bits as from small tensors."""
import pytest
import torch

import quantized_weight_decode_dequant_amd as pkg
from test_gpu_kv_prefix import Case

pytestmark = pytest.mark.gpu
DEV = "cuda"
FAR = 1 << 30  # elements from row to row


def spread(x, stride=FAR):
    """x's rows in a tensor whose rows lie `stride` elements apart."""
    far = torch.empty((x.shape[0] - 1) * stride + x[0].numel(), dtype=x.dtype, device=DEV)
    y = far.as_strided(x.shape, (stride,) + x[0].contiguous().stride())
    y.copy_(x)
    return y


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_the_rotation(dtype):
    M, Hq, Hkv, D = 5, 8, 2, 128
    q, k = (torch.randn(M, H, D, device=DEV).to(dtype) for H in (Hq, Hkv))
    pos = torch.arange(M, dtype=torch.int32, device=DEV) * 1000
    freq = 10000.0 ** (-torch.arange(D // 2, device=DEV) / (D // 2))
    w = torch.rand(D, device=DEV).bfloat16()
    want = pkg.qk_norm_rope_run(q, k, pos, freq, w, w)
    out = spread(torch.zeros(M, Hq, D, dtype=torch.bfloat16, device=DEV))
    got = pkg.qk_norm_rope_run(spread(q), spread(k), pos, freq, w, w, q_out=out)
    torch.cuda.synchronize()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_of_the_sampling(dtype):
    M, V = 5, 33001
    x, u = torch.randn(M, V, device=DEV).to(dtype) * 3, torch.rand(M, device=DEV)
    far = spread(x)
    for kw in (dict(), dict(top_k=torch.full((M,), 50, dtype=torch.int32, device=DEV)),
               dict(top_p=torch.full((M,), 0.9, device=DEV)), dict(temperature=torch.zeros(M, device=DEV))):
        want, got = (pkg.sample_run(a, u, logprobs=torch.empty(M, device=DEV), **kw) for a in (x, far))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("fmt", [pkg.KV_INT8, pkg.KV_E4M3])
@pytest.mark.parametrize("R", [3, 20, 70])
def test_pages_of_a_long_cache(fmt, R):
    """The cache's last pages, 4 GiB and more behind its first."""
    c = Case(R, 700, [1 + 9 * i for i in range(R)], [1] * R, H=2, fmt=fmt)
    cache, a = c.cache(), c.args()
    want = pkg.kv_prefix_attention_run(cache, **a)
    pages = (5 << 30) // (2 * 64 * 128)
    off = pages - c.pages
    big = [torch.empty((pages,) + tuple(t.shape[1:]), dtype=t.dtype, device=DEV) for t in (cache.k, cache.v, cache.k_scales, cache.v_scales)]
    for to, t in zip(big, (cache.k, cache.v, cache.k_scales, cache.v_scales)):
        to[off:] = t
    move = lambda t: torch.where(t >= 0, t + off, t)  # noqa: E731
    got = pkg.kv_prefix_attention_run(pkg.KVCache(*big), **dict(a, table=move(a["table"]), prefix_table=move(a["prefix_table"])))
    torch.cuda.synchronize()
    assert torch.equal(want, got)
