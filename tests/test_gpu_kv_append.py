"""GPU: writing keys and values into the 8-bit cache, against the definition
(codes and scales are the results of stated fp32 operations: bit-equal)."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import quantized_weight_decode_dequant_amd as pkg
from helpers import note, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"


def make(seed, pages, H, page, D, fmt):
    g = np.random.default_rng(seed)
    shape = (pages, H, page, D)
    codes = []
    for _ in range(2):
        if fmt == pkg.KV_INT8:
            codes.append(g.integers(-127, 128, shape).astype(np.int8).view(np.uint8))
        else:
            codes.append(ref.e4m3_bits(np.clip(140 * g.standard_normal(shape), -448, 448)))
    scales = [(0.02 * g.random((pages, H))).astype(np.float32) for _ in range(2)]
    dt = torch.int8 if fmt == pkg.KV_INT8 else torch.float8_e4m3fn
    cache = pkg.KVCache(*[torch.from_numpy(c.copy()).to(DEV).view(dt) for c in codes],
                        *[torch.from_numpy(s.copy()).to(DEV) for s in scales])
    return cache, codes, scales


def run_and_check(cache, codes, scales, kv, slots, fmt, stride=None):
    """kv: float64 [2, M, H, D] of bf16 values."""
    M, H, D = kv.shape[1:]
    t = torch.from_numpy(kv).to(torch.bfloat16)
    if stride is None:
        K, V = t[0].to(DEV), t[1].to(DEV)
    else:
        buf = torch.full((M, stride), float("nan"), dtype=torch.bfloat16, device=DEV)
        K = buf[:, 8:8 + H * D].view(M, H, D)
        V = buf[:, stride - H * D:].view(M, H, D)
        K.copy_(t[0])
        V.copy_(t[1])
    x = [to_np(a) for a in t]
    pkg.kv_append_run(cache, K, V, torch.tensor(np.asarray(slots), dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    out = []
    for name, i in (("k", 0), ("v", 1)):
        want, ws = ref.append(codes[i], scales[i], x[i], slots, bool(i), fmt == pkg.KV_E4M3)
        got = getattr(cache, name).view(torch.uint8).cpu().numpy()
        sc = getattr(cache, name + "_scales").cpu().numpy()
        assert np.array_equal(sc, ws.astype(np.float32)), name
        bad = np.argwhere(got != want)
        assert not len(bad), (name, len(bad), bad[:4], got[tuple(bad[0])], want[tuple(bad[0])])
        out.append((want, ws.astype(np.float32)))
    return [o[0] for o in out], [o[1] for o in out]


def slots_for(g, pages, page, lens, add):
    """Slots of add[r] tokens behind lens[r], on random pages."""
    need = [-(-(n + a) // page) for n, a in zip(lens, add)]
    perm = g.permutation(pages)
    out, at = [], 0
    for n, a, c in zip(lens, add, need):
        out += [int(perm[at + p // page]) * page + p % page for p in range(n, n + a)]
        at += c
    assert at <= pages
    return out


@pytest.mark.parametrize("fmt", [pkg.KV_INT8, pkg.KV_E4M3])
@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_shapes(fmt, page, D):
    note("append fmt=%d page=%d D=%d" % (fmt, page, D))
    g = np.random.default_rng(page + D)
    H = 3
    lens, add = [0, 5, page - 1, page, 17, 3], [2 * page + 3, 1, 2, page, 0, 29]
    pages = 14
    cache, codes, scales = make(page * D, pages, H, page, D, fmt)
    slots = slots_for(g, pages, page, lens, add)
    kv = g.standard_normal((2, len(slots), H, D)) * np.exp(g.uniform(-3, 1, (2, len(slots), 1, 1)))
    run_and_check(cache, codes, scales, kv, slots, fmt)


@pytest.mark.parametrize("fmt", [pkg.KV_INT8, pkg.KV_E4M3])
def test_token_by_token_and_strided(fmt):
    """A page filled one token at a time, from a joint buffer with wide rows:
    growing and shrinking magnitudes, so that codes are rounded again."""
    g = np.random.default_rng(5)
    page, H, D = 32, 2, 64
    cache, codes, scales = make(6, 3, H, page, D, fmt)
    for t in range(page + 5):
        slot = (2 if t < page else 0) * page + t % page
        kv = g.standard_normal((2, 1, H, D)) * (1.3 ** t if t < 12 else 1.0)
        codes, scales = run_and_check(cache, codes, scales, kv, [slot], fmt, stride=2 * H * D + 72)


@pytest.mark.parametrize("fmt", [pkg.KV_INT8, pkg.KV_E4M3])
@pytest.mark.parametrize("M", [1, 64, 1024, 1025, 3001])
def test_many_tokens(fmt, M):
    note("append fmt=%d M=%d" % (fmt, M))
    g = np.random.default_rng(M)
    page, H, D = 64, 2, 64
    first = [0, 40, 63][M % 3]
    pages = -(-(first + M) // page) + 2
    cache, codes, scales = make(M, pages, H, page, D, fmt)
    slots = slots_for(g, pages, page, [first], [M]) + [-1, -1]
    kv = g.standard_normal((2, M + 2, H, D))
    run_and_check(cache, codes, scales, kv, slots, fmt)


@pytest.mark.parametrize("fmt", [pkg.KV_INT8, pkg.KV_E4M3])
def test_one_token_of_many_requests(fmt):
    g = np.random.default_rng(21)
    page, H, D, R = 32, 2, 128, 1100
    lens = g.integers(0, page, R).tolist()
    cache, codes, scales = make(22, R, H, page, D, fmt)
    slots = slots_for(g, R, page, lens, [1] * R)
    run_and_check(cache, codes, scales, g.standard_normal((2, R, H, D)) * 2, slots, fmt)


@pytest.mark.parametrize("fmt", [pkg.KV_INT8, pkg.KV_E4M3])
def test_slots_that_are_skipped_and_odd_values(fmt):
    """Padding and slots past the pool are skipped; zeros, tiny values, the
    largest bf16, infinities and NaN."""
    page, H, D = 32, 1, 64
    cache, codes, scales = make(9, 4, H, page, D, fmt)
    g = np.random.default_rng(10)
    slots = [-1, 4 * page, 5 * page - 1, 2 ** 31 - 1, -2 ** 31, 0, 1, 2, -1, 3 * page + 4, page, 2 * page + 7]
    kv = g.standard_normal((2, len(slots), H, D))
    kv[:, 5] = 0.0
    kv[:, 6] = 2.0 ** -120
    kv[:, 7, 0, :3] = [np.inf, -np.inf, np.nan]
    kv[:, 7, 0, 3:] = 2.0 ** -110
    kv[:, 9, 0, 7] = np.nan
    kv[:, 9, 0, 9] = -np.inf
    kv[:, 10] *= 2.0 ** 120
    kv[0, 10, 0, 5] = 3.3895313892515355e38
    kv[:, 11] = 0.0
    run_and_check(cache, codes, scales, kv, slots, fmt)


def test_whole_chunks_and_page_ends():
    """Runs that end with a page, start at the chunks a workgroup takes and
    are a single token long, in one call of more than 1024 tokens."""
    g = np.random.default_rng(31)
    page, H, D = 32, 1, 64
    lens = [0, 31, 31, 0, 16, 1, 0] + [30] * 40
    add = [32 * 30, 1, 2, 16, 16, 15, 31] + [2] * 40
    pages = sum(-(-(n + a) // page) for n, a in zip(lens, add))
    cache, codes, scales = make(32, pages, H, page, D, pkg.KV_INT8)
    slots = slots_for(g, pages, page, lens, add)
    assert len(slots) > 1024
    run_and_check(cache, codes, scales, g.standard_normal((2, len(slots), H, D)), slots, pkg.KV_INT8)


def test_past_32_bits():
    """A pool of more than 4 GiB of codes: the last pages are written."""
    page, H, D = 128, 8, 256
    pages = (1 << 32) // (page * H * D) + 40
    note("append pool of %.1f GiB" % (pages * page * H * D / 2 ** 30))
    k = torch.zeros(pages, H, page, D, dtype=torch.uint8, device=DEV).view(torch.int8)
    v = torch.zeros(pages, H, page, D, dtype=torch.uint8, device=DEV).view(torch.int8)
    sc = [torch.zeros(pages, H, device=DEV) for _ in range(2)]
    cache = pkg.KVCache(k, v, *sc)
    g = np.random.default_rng(3)
    M = page + 9
    slots = [(pages - 1) * page + i for i in range(page)] + [(pages - 3) * page + i for i in range(9)]
    kv = g.standard_normal((2, M, H, D))
    t = torch.from_numpy(kv).to(torch.bfloat16)
    pkg.kv_append_run(cache, t[0].to(DEV), t[1].to(DEV), torch.tensor(slots, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    tail = [slots[i] - (pages - 4) * page for i in range(M)]
    for i, (c, s) in enumerate(((k, sc[0]), (v, sc[1]))):
        want, ws = ref.append(np.zeros((4, H, page, D), np.uint8), np.zeros((4, H)), to_np(t[i]), tail, bool(i), False)
        assert np.array_equal(c[-4:].view(torch.uint8).cpu().numpy(), want)
        assert np.array_equal(s[-4:].cpu().numpy(), ws.astype(np.float32))
        assert not s[:-4].any()
        assert not c[:40].view(torch.uint8).any()
