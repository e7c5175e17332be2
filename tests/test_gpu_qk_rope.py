"""GPU: qk_norm_rope_run against its definition in 64 bits.

Tolerance, per element of a pair (a, b), each after the norm: the output's
rounding, 2^-8 of it; the norm in fp32 (a sum of up to 512 squares in lanes of
8 and a tree of 6: 16 roundings, half of that after the root; mean, eps, root,
inverse, two products: 16 * 2^-24 in all) and the rotation's two products and
one sum (3 * 2^-24), 2^-19 of |a| + |b|; sine and cosine to 2 ulp and the angle
rounded to fp32 below half a turn, 2^-21; the fp64 angle's two roundings,
2^-52 of it."""
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


def freqs(rotated, base=10000.0):
    return torch.from_numpy((base ** (-np.arange(rotated // 2) * 2.0 / max(rotated, 1))).astype(np.float32)).to(DEV)


def make(M, Hq, Hkv, D, dtype, seed=0, norm=True, extra=0):
    """q, k as views of one buffer (a joint projection's output) and the weights."""
    g = torch.Generator().manual_seed(seed)
    qkv = torch.randn(M, Hq + Hkv + extra, D, generator=g)
    qkv[:, :, ::3] *= 7
    qkv = qkv.to(dtype).to(DEV)
    w = [(1 + 0.3 * torch.randn(D, generator=g)).to(BF16).to(DEV) if norm else None for _ in range(2)]
    return qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], w[0], w[1]


def check(got, x, w, eps, positions, axis, inv_freq, interleaved):
    z, size, far = ref.rope(to_np(x), None if w is None else to_np(w), np.float64(np.float32(eps)), to_np(positions),
                            None if axis is None else to_np(axis), to_np(inv_freq), interleaved)
    tol = 2.0 ** -8 * np.abs(z) + (2.0 ** -19 + 2.0 ** -21 + 2.0 ** -52 * far) * size + 1e-38
    err = np.abs(to_np(got) - z)
    assert np.all(err <= tol), (float((err / tol).max()))


SHAPES = [  # M, Hq, Hkv, D, rotated, type, interleaved, axes
    (1, 32, 8, 128, 128, BF16, False, 1), (1, 1, 1, 64, 64, F32, True, 1), (3, 5, 1, 80, 32, BF16, False, 2),
    (7, 3, 3, 96, 96, F32, False, 3), (33, 12, 4, 256, 64, BF16, True, 1), (2, 8, 2, 512, 512, BF16, False, 4),
    (5, 4, 4, 512, 256, F32, True, 2), (2050, 6, 2, 64, 32, BF16, False, 1), (2049, 9, 7, 128, 128, BF16, True, 3),
    (4, 2, 1, 8, 0, BF16, False, 1), (9, 3, 1, 16, 16, F32, False, 1), (6, 7, 2, 104, 48, BF16, False, 1), (1, 300, 20, 128, 128, BF16, False, 1)]


@pytest.mark.parametrize("M,Hq,Hkv,D,rotated,dtype,inter,axes", SHAPES)
@pytest.mark.parametrize("norm", [True, False])
def test_shapes(M, Hq, Hkv, D, rotated, dtype, inter, axes, norm):
    note("rope", M, Hq, Hkv, D, rotated, dtype, inter, axes, norm)
    q, k, qw, kw = make(M, Hq, Hkv, D, dtype, M, norm, extra=Hkv)
    g = np.random.default_rng(M)
    pos = torch.from_numpy(g.integers(0, 40000, (axes, M) if axes > 1 else M).astype(np.int32)).to(DEV)
    f = freqs(rotated)
    axis = torch.from_numpy(g.integers(0, axes, rotated // 2).astype(np.uint8)).to(DEV) if axes > 1 else None
    qo, ko = pkg.qk_norm_rope_run(q, k, pos, f, q_weight=qw, k_weight=kw, eps=1e-5, axis=axis, interleaved=inter)
    torch.cuda.synchronize()
    check(qo, q, qw, 1e-5, pos, axis, f, inter)
    check(ko, k, kw, 1e-5, pos, axis, f, inter)


@pytest.mark.parametrize("pos", [0, 1, 2 ** 30, 2 ** 31 - 1, -5, -2 ** 31])
@pytest.mark.parametrize("inter", [False, True])
def test_far_positions(pos, inter):
    q, k, qw, kw = make(2, 4, 2, 128, BF16)
    p = torch.tensor([pos, pos - 1 if pos > 0 else pos + 1], dtype=torch.int32, device=DEV)
    f = freqs(128)
    qo, ko = pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw, k_weight=kw, interleaved=inter)
    check(qo, q, qw, 1e-6, p, None, f, inter)
    check(ko, k, kw, 1e-6, p, None, f, inter)


def test_an_axis_that_is_not_there_does_not_turn():
    q, k, _, _ = make(3, 2, 1, 64, BF16)
    p = torch.tensor([[5, 6, 7], [100, 200, 300]], dtype=torch.int32, device=DEV)
    axis = torch.tensor([0, 1, 2, 255] * 8, dtype=torch.uint8, device=DEV)
    f = freqs(64)
    qo, _ = pkg.qk_norm_rope_run(q, k, p, f, axis=axis)
    check(qo, q, None, 1e-6, p, axis, f, False)
    for i in (2, 3):
        assert torch.equal(qo[:, :, i::4], q[:, :, i::4])


def test_one_side_normed_and_one_side_alone():
    q, k, qw, _ = make(5, 6, 2, 128, F32)
    p, f = torch.arange(5, dtype=torch.int32, device=DEV), freqs(128)
    qo, ko = pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw)
    check(qo, q, qw, 1e-6, p, None, f, False)
    check(ko, k, None, 1e-6, p, None, f, False)
    alone, none = pkg.qk_norm_rope_run(q, None, p, f, q_weight=qw)
    assert none is None and torch.equal(alone, qo)


@pytest.mark.parametrize("D,M", [(128, 1), (64, 700), (256, 3), (80, 2100)])
def test_in_place_and_strided_outputs_equal(D, M):
    q, k, qw, kw = make(M, 8, 4, D, BF16, extra=4)
    p, f = torch.arange(M, dtype=torch.int32, device=DEV) * 3, freqs(D)
    qo, ko = pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw, k_weight=kw)
    joint = torch.full((M, 16, D), 3.0, dtype=BF16, device=DEV)
    pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw, k_weight=kw, q_out=joint[:, :8], k_out=joint[:, 12:])
    assert torch.equal(joint[:, :8], qo) and torch.equal(joint[:, 12:], ko) and bool((joint[:, 8:12] == 3).all())
    rest = q.as_strided((M, 4, D), q.stride(), q.storage_offset() + 12 * D).clone()
    pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw, k_weight=kw, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko)
    assert torch.equal(q.as_strided((M, 4, D), q.stride(), q.storage_offset() + 12 * D), rest)


def test_extreme_values():
    """Zero heads, heads near fp32's ends, infinities and NaN: each head by itself."""
    x = torch.randn(1, 6, 64, generator=torch.Generator().manual_seed(1))
    x[0, 0] = 0
    x[0, 1] *= 1e-25
    x[0, 2] *= 1e17
    x[0, 3, 5] = float("inf")
    x[0, 4, 6] = float("nan")
    x = x.to(DEV)
    w = torch.ones(64, dtype=BF16, device=DEV)
    p, f = torch.tensor([77], dtype=torch.int32, device=DEV), freqs(64)
    out, _ = pkg.qk_norm_rope_run(x, None, p, f, q_weight=w, eps=1e-6)
    keep = [0, 1, 2, 5]
    check(out[:, keep], x[:, keep], w, 1e-6, p, None, f, False)
    assert bool((out[0, 0] == 0).all()) and bool(out[0, 3, [5, 37]].isnan().all()) and bool(out[0, 4].isnan().all())
    flat, _ = pkg.qk_norm_rope_run(x, None, p, f)
    assert bool(flat[0, keep].isfinite().all()) and bool(flat[0, 4, [6, 38]].isnan().all())


def test_no_tokens():
    q = torch.empty(0, 4, 64, dtype=BF16, device=DEV)
    qo, ko = pkg.qk_norm_rope_run(q, q[:, :2], torch.empty(0, dtype=torch.int32, device=DEV), freqs(64))
    assert qo.shape == (0, 4, 64) and ko.shape == (0, 2, 64)


def test_captured_and_on_another_stream():
    q, k, qw, kw = make(9, 8, 2, 128, BF16)
    p, f = torch.arange(9, dtype=torch.int32, device=DEV), freqs(128)
    qo, ko = torch.zeros(9, 8, 128, dtype=BF16, device=DEV), torch.zeros(9, 2, 128, dtype=BF16, device=DEV)
    graph = workloads.capture_graph(lambda: pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw, k_weight=kw, q_out=qo, k_out=ko))
    for rep in range(4):
        p.add_(1000 * rep)
        q.mul_(1.5)
        graph.replay()
        torch.cuda.synchronize()
        want = pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw, k_weight=kw)
        assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = pkg.qk_norm_rope_run(q, k, p, f, q_weight=qw, k_weight=kw, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_the_binding_refuses():
    q, k, qw, kw = make(4, 4, 2, 64, BF16)
    p, f = torch.arange(4, dtype=torch.int32, device=DEV), freqs(64)
    good = dict(q=q, k=k, positions=p, inv_freq=f, q_weight=qw, k_weight=kw)
    pkg.qk_norm_rope_run(**good)
    for bad in (dict(k=k.float()), dict(k=k[:3]), dict(positions=p.long()), dict(positions=p[:3]), dict(q=q.half()),
                dict(inv_freq=f.double()), dict(q_weight=qw[:32]), dict(axis=torch.zeros(31, dtype=torch.uint8, device=DEV)),
                dict(q_out=q.float()), dict(k=None, k_out=k), dict(q=q.transpose(1, 2)), dict(positions=p.cpu()),
                dict(q_out=torch.empty(4, 4, 32, dtype=BF16, device=DEV))):
        with pytest.raises(ValueError):
            pkg.qk_norm_rope_run(**{**good, **bad})
    with pytest.raises(pkg.QGError):  # 40 rotated dimensions
        pkg.qk_norm_rope_run(q, k, p, f[:20])
