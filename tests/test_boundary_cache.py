"""Refusals of the norm and the cache operators, at the C ABI and in the
binding: every call fails validation before any HIP call, or is an empty
problem.  Fake device addresses are passed, so, like test_boundary.py, this
runs where no GPU is visible (on a GPU host in a child process:
test_zz_boundary_cache_isolated.py)."""
import ctypes as C
import os

import pytest
import torch

from conftest import gpu_visible
import quantized_weight_decode_dequant_amd as pkg
from quantized_weight_decode_dequant_amd import _lib as L

A = 0x10000
CHILD = os.environ.get("QG_BOUNDARY_CHILD") == "1"
if CHILD:
    assert not gpu_visible(), "the boundary child process still sees a GPU"
pytestmark = pytest.mark.skipif(not CHILD and gpu_visible(),
                                reason="a GPU is visible: runs in a child process with every GPU hidden")

NAN, INF = float("nan"), float("inf")


def expect(call, cases):
    for kw, want in cases:
        assert call(**kw) == want, (kw, pkg.status_string(call(**kw)), pkg.status_string(want))


def test_rmsnorm():
    lib = pkg.raw()

    def call(**kw):
        a = dict(x=A, xt=0, res=A, ro=A, rt=0, w=A, eps=1e-6, signs=A, M=4, K=64, y=A, Xq=A, sc=A)
        a.update(kw)
        return lib.rmsnorm_quant_run(a["x"], a["xt"], a["res"], a["ro"], a["rt"], a["w"], a["eps"], a["signs"], a["M"],
                                     a["K"], a["y"], a["Xq"], a["sc"], None)

    expect(call, [
        (dict(M=0), L.QG_OK), (dict(M=-1), L.QG_ESHAPE), (dict(M=(1 << 30) + 1), L.QG_ESHAPE), (dict(M=1 << 22), L.QG_ESHAPE),
        (dict(K=0), L.QG_ESHAPE), (dict(K=48), L.QG_ESHAPE), (dict(K=24576 + 32), L.QG_ESHAPE), (dict(K=-32), L.QG_ESHAPE),
        (dict(x=None), L.QG_EINVAL), (dict(w=None), L.QG_EINVAL), (dict(y=None, Xq=None, sc=None, signs=None), L.QG_EINVAL),
        (dict(Xq=None), L.QG_EINVAL), (dict(sc=None), L.QG_EINVAL), (dict(res=None), L.QG_EINVAL),
        (dict(Xq=None, sc=None), L.QG_EINVAL),  # signs without an int8 output
        (dict(eps=0.0), L.QG_EINVAL), (dict(eps=-1.0), L.QG_EINVAL), (dict(eps=NAN), L.QG_EINVAL), (dict(eps=INF), L.QG_EINVAL),
        (dict(xt=3), L.QG_EINVAL), (dict(rt=-1), L.QG_EINVAL), (dict(xt=2), L.QG_EUNSUPPORTED), (dict(rt=2), L.QG_EUNSUPPORTED),
    ] + [({k: A + 8}, L.QG_EALIGN) for k in ("x", "res", "ro", "w", "signs", "y", "Xq")] + [(dict(sc=A + 2), L.QG_EALIGN)])


def test_tables():
    lib = pkg.raw()
    names = ["R", "page", "pages", "nb", "mt", "lens", "keep", "add", "table", "free", "count", "q", "slots", "pos", "st"]
    base = dict(zip(names, [4, 64, 100, 10, 50] + [A] * 10))

    def call(**kw):
        return lib.kv_tables_run(*[{**base, **kw}[n] for n in names], None)

    expect(call, [
        (dict(R=0, q=None), L.QG_EINVAL), (dict(R=-1), L.QG_ESHAPE), (dict(R=4097), L.QG_ESHAPE), (dict(page=16), L.QG_ESHAPE),
        (dict(page=48), L.QG_ESHAPE), (dict(page=512), L.QG_ESHAPE), (dict(page=0), L.QG_ESHAPE), (dict(pages=0), L.QG_ESHAPE),
        (dict(pages=(1 << 31) // 64), L.QG_ESHAPE), (dict(nb=0), L.QG_ESHAPE), (dict(nb=(1 << 30) // 64 + 1), L.QG_ESHAPE),
        (dict(mt=-1), L.QG_ESHAPE), (dict(mt=(1 << 30) + 1), L.QG_ESHAPE),
    ] + [({k: None}, L.QG_EINVAL) for k in ("lens", "add", "table", "free", "count", "q", "slots", "pos", "st")]
      + [({k: A + 2}, L.QG_EALIGN) for k in names[5:]])


def cache(**kw):
    a = dict(k=A, v=A, k_scales=A, v_scales=A, pages=10, page=64, Hkv=2, D=128, fmt=0)
    a.update(kw)
    return L.CacheDesc(**a)


BAD_CACHES = [
    (dict(fmt=2), L.QG_EINVAL), (dict(fmt=-1), L.QG_EINVAL), (dict(page=16), L.QG_ESHAPE), (dict(page=96), L.QG_ESHAPE),
    (dict(D=96), L.QG_ESHAPE), (dict(D=512), L.QG_ESHAPE), (dict(Hkv=0), L.QG_ESHAPE), (dict(Hkv=1025), L.QG_ESHAPE),
    (dict(pages=0), L.QG_ESHAPE), (dict(pages=-5), L.QG_ESHAPE), (dict(pages=1 << 25), L.QG_ESHAPE), (dict(k=None), L.QG_EINVAL),
    (dict(v=None), L.QG_EINVAL), (dict(k_scales=None), L.QG_EINVAL), (dict(v_scales=None), L.QG_EINVAL), (dict(k=A + 8), L.QG_EALIGN),
    (dict(v=A + 4), L.QG_EALIGN), (dict(k_scales=A + 2), L.QG_EALIGN), (dict(v_scales=A + 1), L.QG_EALIGN)]


def test_append():
    lib = pkg.raw()

    def call(c=None, **kw):
        a = dict(M=5, K=A, ks=256, V=A, vs=256, slots=A)
        a.update(kw)
        desc = cache(**(c or {}))
        return lib.kv_append_run(C.addressof(desc), a["M"], a["K"], a["ks"], a["V"], a["vs"], a["slots"], None)

    assert lib.kv_append_run(None, 1, A, 256, A, 256, A, None) == L.QG_EINVAL
    expect(call, [(dict(c=c), want) for c, want in BAD_CACHES] + [
        (dict(M=0), L.QG_OK), (dict(M=-1), L.QG_ESHAPE), (dict(M=(1 << 30) + 1), L.QG_ESHAPE), (dict(ks=248), L.QG_ESHAPE),
        (dict(vs=260), L.QG_ESHAPE), (dict(ks=1 << 31), L.QG_ESHAPE), (dict(K=None), L.QG_EINVAL), (dict(V=None), L.QG_EINVAL),
        (dict(slots=None), L.QG_EINVAL), (dict(K=A + 2), L.QG_EALIGN), (dict(V=A + 8), L.QG_EALIGN), (dict(slots=A + 2), L.QG_EALIGN)])


def test_attention():
    lib = pkg.raw()
    ws = pkg.kv_attention_workspace_bytes(3, 5, 8, 2, 128, 64, 4, 2560)
    assert ws > 0

    def call(c=None, **kw):
        a = dict(R=3, M=5, Hq=8, q=A, qs=1024, q_start=A, lens=A, table=A, nb=40, tree=None, window=0, scale=0.1, max_q=4,
                 max_len=2560, ws=A, wsb=ws, out=A, os=1024, od=0)
        a.update(kw)
        desc = cache(**(c or {}))
        return lib.kv_attention_run(C.addressof(desc), a["R"], a["M"], a["Hq"], a["q"], a["qs"], a["q_start"], a["lens"], a["table"],
                                    a["nb"], a["tree"], a["window"], a["scale"], a["max_q"], a["max_len"], a["ws"], a["wsb"],
                                    a["out"], a["os"], a["od"], None)

    assert lib.kv_attention_run(None, 1, 1, 8, A, 1024, A, A, A, 10, None, 0, 1.0, 1, 64, A, ws, A, 1024, 0, None) == L.QG_EINVAL
    expect(call, [(dict(c=c), want) for c, want in BAD_CACHES] + [
        (dict(R=0), L.QG_OK), (dict(M=0, wsb=0, ws=None), L.QG_OK), (dict(R=-1), L.QG_ESHAPE), (dict(R=65536), L.QG_ESHAPE),
        (dict(M=-1), L.QG_ESHAPE), (dict(M=(1 << 30) + 1), L.QG_ESHAPE), (dict(Hq=7), L.QG_ESHAPE), (dict(Hq=0), L.QG_ESHAPE),
        (dict(Hq=8194, qs=1 << 21, os=1 << 21), L.QG_ESHAPE), (dict(qs=1016), L.QG_ESHAPE), (dict(qs=1028), L.QG_ESHAPE),
        (dict(os=512), L.QG_ESHAPE), (dict(os=1 << 31), L.QG_ESHAPE), (dict(nb=0), L.QG_ESHAPE), (dict(nb=(1 << 30) // 64 + 1), L.QG_ESHAPE),
        (dict(R=4096, Hq=512, qs=1 << 16, os=1 << 16, max_q=32, max_len=64, wsb=1 << 40), L.QG_ESHAPE),  # more joins than a launch holds
        (dict(max_q=0), L.QG_ESHAPE), (dict(max_q=33), L.QG_ESHAPE), (dict(max_len=0), L.QG_ESHAPE), (dict(max_len=2561), L.QG_ESHAPE),
        (dict(window=-1), L.QG_ESHAPE), (dict(window=(1 << 30) + 1), L.QG_ESHAPE), (dict(tree=A, window=5), L.QG_EUNSUPPORTED),
        (dict(od=2), L.QG_EUNSUPPORTED), (dict(od=3), L.QG_EINVAL), (dict(scale=NAN), L.QG_EINVAL), (dict(scale=INF), L.QG_EINVAL),
        (dict(wsb=ws - 1), L.QG_ESIZE), (dict(ws=None), L.QG_EINVAL), (dict(ws=A + 8), L.QG_EALIGN), (dict(tree=A + 2), L.QG_EALIGN),
    ] + [({k: None}, L.QG_EINVAL) for k in ("q", "q_start", "lens", "table", "out")]
      + [({k: A + 2}, L.QG_EALIGN) for k in ("q", "q_start", "lens", "table", "out")])


def test_workspace_size():
    f = pkg.kv_attention_workspace_bytes
    assert f(1, 1, 8, 2, 128, 64, 1, 64) == 0                    # one chunk: nothing to join
    few, many = f(1, 1, 8, 2, 128, 64, 1, 1 << 14), f(48, 48, 8, 2, 128, 64, 1, 1 << 14)
    assert 0 < few <= many < 1 << 26
    assert f(1, 1, 7, 2, 128, 64, 1, 1 << 14) == 0 and f(1, 1, 8, 2, 100, 64, 1, 1 << 14) == 0
    assert f(4096, 1 << 30, 8192, 1, 256, 32, 32, 1 << 30) == 0  # refused: the work does not fit 31 bits


def test_binding_refuses_host_tensors_and_wrong_types():
    """The binding's own checks, before the library is called."""
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        pkg.rmsnorm_quant_run(x, w, 1e-6)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        pkg.rmsnorm_quant_run(x.half(), w, 1e-6)
    with pytest.raises(ValueError, match=r"\[M, K\]"):
        pkg.rmsnorm_quant_run(x[0], w, 1e-6)
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="device tensor"):
        pkg.kv_tables_run(64, i, i, i.view(2, 2), i, i[:1], 3)
    with pytest.raises(ValueError, match="at least 3"):
        pkg.kv_tables_run(64, i, i, i.view(2, 2), i, i[:1], 3, slots=i[:2])
    codes, scales = torch.zeros(4, 2, 64, 64, dtype=torch.int8), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="device tensor"):
        pkg.KVCache(codes, codes, scales, scales)
    with pytest.raises(ValueError, match="int8 or float8_e4m3fn"):
        pkg.KVCache(codes.half(), codes.half(), scales, scales)
    with pytest.raises(ValueError, match="unknown cache format"):
        pkg.KVCache.empty(4, 64, 2, 64, fmt=9, device="cpu")


def test_attention_scales_past_fp32_in_powers_of_two():
    """scale * log2(e) is what the kernels take: it has to be finite too."""
    lib = pkg.raw()
    ws = pkg.kv_attention_workspace_bytes(3, 5, 8, 2, 128, 64, 4, 2560)
    desc = cache()
    for scale, want in ((3e38, L.QG_EINVAL), (-3e38, L.QG_EINVAL), (2.3e38, L.QG_EALIGN), (-2.0 ** 127, L.QG_EALIGN)):
        assert lib.kv_attention_run(C.addressof(desc), 3, 5, 8, A + 2, 1024, A, A, A, 40, None, 0, scale, 4, 2560, A, ws, A, 1024, 0, None) == want


def test_attention_joins_that_fill_a_launch():
    """2731 * 3 * 8191 = 2^26 - 1 joins: 2^23 workgroups of 512 are 2^32 threads."""
    lib = pkg.raw()
    desc = cache(Hkv=1)

    def call(R, max_q, Hq, q=A):
        return lib.kv_attention_run(C.addressof(desc), R, 5, Hq, q, Hq * 128, A, A, A, 40, None, 0, 0.1, max_q, 64, A, 1 << 40, A,
                                    Hq * 128, 0, None)

    assert call(2731, 3, 8191) == L.QG_ESHAPE
    assert call(2731, 3, 8190, A + 2) == L.QG_EALIGN
    assert pkg.kv_attention_workspace_bytes(2731, 5, 8191, 1, 128, 64, 3, 5000) == 0
    assert pkg.kv_attention_workspace_bytes(2731, 5, 8190, 1, 128, 64, 3, 5000) > 0
