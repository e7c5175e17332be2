"""Refusals of the head norm with rotation, the attention behind a shared
prefix and the sampling, at the C ABI and in the binding: every call fails
validation before any HIP call, or is an empty problem.  Fake device addresses
are passed, so this runs where no GPU is visible (on a GPU host in a child
process: test_zz_boundary_step_isolated.py)."""
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


def test_rope():
    lib = pkg.raw()

    def call(**kw):
        a = dict(q=A, qs=512, k=A, ks=256, xt=0, M=4, Hq=4, Hkv=2, D=128, qw=A, kw=A, eps=1e-6, pos=A, axes=1, axis=None, f=A,
                 rot=128, il=0, qo=A, qos=512, ko=A, kos=256)
        a.update(kw)
        return lib.qk_norm_rope_run(a["q"], a["qs"], a["k"], a["ks"], a["xt"], a["M"], a["Hq"], a["Hkv"], a["D"], a["qw"], a["kw"],
                                    a["eps"], a["pos"], a["axes"], a["axis"], a["f"], a["rot"], a["il"], a["qo"], a["qos"], a["ko"],
                                    a["kos"], None)

    expect(call, [
        (dict(M=0), L.QG_OK), (dict(Hq=0, Hkv=0), L.QG_OK), (dict(M=0, axes=4, axis=A + 1), L.QG_OK), (dict(M=-1), L.QG_ESHAPE),
        (dict(M=(1 << 26) - 7), L.QG_ESHAPE), (dict(M=0, rot=0, pos=None, f=None), L.QG_OK), (dict(M=0, qw=None, kw=None, eps=NAN), L.QG_OK),
        (dict(M=0, Hkv=0, k=None, ko=None, ks=0, kos=0), L.QG_OK), (dict(Hq=-1), L.QG_ESHAPE), (dict(Hq=8193, qs=1 << 21, qos=1 << 21), L.QG_ESHAPE),
        (dict(Hkv=1025, ks=1 << 18, kos=1 << 18), L.QG_ESHAPE), (dict(D=4), L.QG_ESHAPE), (dict(D=132, qs=1 << 12, ks=1 << 12, qos=1 << 12, kos=1 << 12), L.QG_ESHAPE),
        (dict(D=520, qs=1 << 12, ks=1 << 12, qos=1 << 12, kos=1 << 12), L.QG_ESHAPE), (dict(rot=120), L.QG_ESHAPE), (dict(rot=144), L.QG_ESHAPE),
        (dict(rot=-16), L.QG_ESHAPE), (dict(axes=0), L.QG_ESHAPE), (dict(axes=5), L.QG_ESHAPE), (dict(qs=504), L.QG_ESHAPE), (dict(qs=516), L.QG_ESHAPE),
        (dict(ks=248), L.QG_ESHAPE), (dict(qos=1 << 31), L.QG_ESHAPE), (dict(kos=255), L.QG_ESHAPE), (dict(xt=2), L.QG_EUNSUPPORTED),
        (dict(xt=3), L.QG_EINVAL), (dict(il=2), L.QG_EINVAL), (dict(eps=0.0), L.QG_EINVAL), (dict(eps=INF), L.QG_EINVAL),
        (dict(kw=None, eps=NAN), L.QG_EINVAL),
    ] + [({k: None}, L.QG_EINVAL) for k in ("q", "k", "pos", "f", "qo", "ko")]
      + [({k: A + 8}, L.QG_EALIGN) for k in ("q", "k", "qw", "kw", "qo", "ko")] + [(dict(pos=A + 2), L.QG_EALIGN), (dict(f=A + 1), L.QG_EALIGN)])


def cache(**kw):
    a = dict(k=A, v=A, k_scales=A, v_scales=A, pages=10, page=64, Hkv=2, D=128, fmt=0)
    a.update(kw)
    return L.CacheDesc(**a)


def test_prefix_attention():
    lib = pkg.raw()
    ws = pkg.kv_prefix_attention_workspace_bytes(3, 5, 8, 2, 128, 64, 4, 2560, 1920)
    assert ws > 0

    def call(c=None, **kw):
        a = dict(R=3, M=5, Hq=8, q=A, qs=1024, q_start=A, lens=A, table=A, nb=40, pt=A, pb=30, pl=A, tree=None, scale=0.1, max_q=4,
                 max_len=2560, mp=1920, ws=A, wsb=ws, out=A, os=1024, od=0)
        a.update(kw)
        desc = cache(**(c or {}))
        return lib.kv_prefix_attention_run(C.addressof(desc), a["R"], a["M"], a["Hq"], a["q"], a["qs"], a["q_start"], a["lens"], a["table"],
                                           a["nb"], a["pt"], a["pb"], a["pl"], a["tree"], a["scale"], a["max_q"], a["max_len"], a["mp"],
                                           a["ws"], a["wsb"], a["out"], a["os"], a["od"], None)

    assert lib.kv_prefix_attention_run(None, 1, 1, 8, A, 1024, A, A, A, 10, A, 10, A, None, 1.0, 1, 64, 64, A, ws, A, 1024, 0, None) == L.QG_EINVAL
    expect(call, [
        (dict(c=dict(fmt=2)), L.QG_EINVAL), (dict(c=dict(page=96)), L.QG_ESHAPE), (dict(c=dict(D=96)), L.QG_ESHAPE), (dict(c=dict(k=None)), L.QG_EINVAL),
        (dict(c=dict(v=A + 4)), L.QG_EALIGN), (dict(R=0), L.QG_OK), (dict(M=0, wsb=0, ws=None), L.QG_OK), (dict(R=-1), L.QG_ESHAPE),
        (dict(R=4097), L.QG_ESHAPE), (dict(M=-1), L.QG_ESHAPE), (dict(M=1 << 23), L.QG_ESHAPE), (dict(Hq=7), L.QG_ESHAPE), (dict(Hq=0), L.QG_ESHAPE),
        (dict(qs=1016), L.QG_ESHAPE), (dict(os=512), L.QG_ESHAPE), (dict(os=1028), L.QG_ESHAPE), (dict(nb=0), L.QG_ESHAPE), (dict(nb=1 << 25), L.QG_ESHAPE),
        (dict(pb=0), L.QG_ESHAPE), (dict(pb=1 << 25), L.QG_ESHAPE), (dict(mp=-1), L.QG_ESHAPE), (dict(mp=1921), L.QG_ESHAPE), (dict(max_q=0), L.QG_ESHAPE),
        (dict(max_q=33), L.QG_ESHAPE), (dict(max_len=0), L.QG_ESHAPE), (dict(max_len=2561), L.QG_ESHAPE), (dict(od=2), L.QG_EUNSUPPORTED),
        (dict(od=5), L.QG_EINVAL), (dict(scale=NAN), L.QG_EINVAL), (dict(scale=3e38), L.QG_EINVAL), (dict(wsb=ws - 1), L.QG_ESIZE),
        (dict(ws=None), L.QG_EINVAL), (dict(ws=A + 8), L.QG_EALIGN), (dict(tree=A + 2), L.QG_EALIGN),
        (dict(R=4096, Hq=512, qs=1 << 16, os=1 << 16, max_q=32, max_len=64, wsb=1 << 40), L.QG_ESHAPE),  # more joins than a launch holds
    ] + [({k: None}, L.QG_EINVAL) for k in ("q", "q_start", "lens", "table", "pt", "pl", "out")]
      + [({k: A + 2}, L.QG_EALIGN) for k in ("q", "q_start", "lens", "table", "pt", "pl", "out")])


def test_prefix_workspace_size():
    f = pkg.kv_prefix_attention_workspace_bytes
    assert f(0, 5, 8, 2, 128, 64, 1, 64, 64) == 0 and f(5, 0, 8, 2, 128, 64, 1, 64, 64) == 0
    assert 0 < f(1, 1, 8, 2, 128, 64, 1, 64, 0) <= f(48, 48, 32, 8, 128, 64, 1, 2048, 32768) < 1 << 28
    assert f(1, 1, 7, 2, 128, 64, 1, 64, 64) == 0 and f(1, 1, 8, 2, 100, 64, 1, 64, 64) == 0 and f(1, 1, 8, 2, 128, 48, 1, 64, 64) == 0
    assert f(4096, 8192, 8192, 1, 256, 32, 1, 1 << 30, 1 << 30) == 0  # refused: the work does not fit 31 bits
    # every shape of call: sizes that stay in proportion to what is cut
    for D in (64, 128, 256):
        for R in (1, 4, 5, 8, 16, 17, 48, 100, 1000, 4096):
            for T in (1, 7, 32):
                for P in (0, 1, 333, 8192, 131072):
                    assert 0 < f(R, R * T, 16, 4, D, 64, T, 512, P) < (1 << 28) + R * T * 16 * D * 4 * 130, (D, R, T, P)


def test_sample():
    lib = pkg.raw()
    ws = pkg.sample_workspace_bytes(4, 5000)
    assert ws > 0

    def call(**kw):
        a = dict(x=A, xt=0, M=4, V=5000, s=5000, u=A, T=A, k=A, p=A, mp=A, ws=A, wsb=ws, t=A, l=A)
        a.update(kw)
        return lib.sample_run(a["x"], a["xt"], a["M"], a["V"], a["s"], a["u"], a["T"], a["k"], a["p"], a["mp"], a["ws"], a["wsb"],
                              a["t"], a["l"], None)

    expect(call, [
        (dict(M=0, wsb=0, ws=None), L.QG_OK), (dict(M=-1), L.QG_ESHAPE), (dict(V=0), L.QG_ESHAPE), (dict(V=-3), L.QG_ESHAPE),
        (dict(V=(1 << 20) + 1, s=1 << 21, wsb=1 << 40), L.QG_ESHAPE), (dict(s=4999), L.QG_ESHAPE), (dict(s=1 << 31), L.QG_ESHAPE),
        (dict(M=1 << 23, wsb=1 << 50), L.QG_ESHAPE), (dict(xt=2), L.QG_EUNSUPPORTED), (dict(xt=-1), L.QG_EINVAL), (dict(x=None), L.QG_EINVAL),
        (dict(u=None), L.QG_EINVAL), (dict(t=None), L.QG_EINVAL), (dict(ws=None), L.QG_EINVAL), (dict(wsb=ws - 1), L.QG_ESIZE),
        (dict(ws=A + 8), L.QG_EALIGN), (dict(x=A + 1), L.QG_EALIGN), (dict(x=A + 2, xt=1), L.QG_EALIGN),
    ] + [({k: A + 2}, L.QG_EALIGN) for k in ("u", "T", "k", "p", "mp", "t", "l")])
    assert pkg.sample_workspace_bytes(0, 5000) == 0 and pkg.sample_workspace_bytes(1, 0) == 0
    assert pkg.sample_workspace_bytes(1, (1 << 20) + 1) == 0 and pkg.sample_workspace_bytes(1 << 24, 100) == 0
    assert pkg.sample_workspace_bytes(1, 1 << 20) > 0


def test_binding_refuses_host_tensors_and_wrong_types():
    bf = torch.zeros(4, 2, 64, dtype=torch.bfloat16)
    p, f = torch.zeros(4, dtype=torch.int32), torch.zeros(32)
    with pytest.raises(ValueError, match="device tensor"):
        pkg.qk_norm_rope_run(bf, bf, p, f)
    with pytest.raises(ValueError, match=r"\[M, Hq, D\]"):
        pkg.qk_norm_rope_run(bf[0], None, p, f)
    with pytest.raises(ValueError, match="bfloat16 or float32"):
        pkg.qk_norm_rope_run(bf.half(), None, p, f)
    with pytest.raises(ValueError, match="device tensor"):
        pkg.sample_run(torch.zeros(4, 100), torch.zeros(4))
    with pytest.raises(ValueError, match=r"\[M, V\]"):
        pkg.sample_run(torch.zeros(100), torch.zeros(4))
    with pytest.raises(ValueError, match="prefix_table"):
        pkg.kv_prefix_attention_run(None, bf, p, p, p.view(2, 2), p.view(2, 2), p[:1], 1)
