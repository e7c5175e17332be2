"""GPU: the operators around the products as one decode loop uses them.

A prompt, verification tiles with drafts thrown away, single tokens and a
finished request go through norm, the quantized projection, cache tables,
append and attention; each operator's result is checked against its 64-bit
definition on what the one before it left on the GPU.  The same step captured
in a HIP graph and replayed with new lengths equals the eager one."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import quantized_weight_decode_dequant_amd as pkg
from quantized_weight_decode_dequant_amd import synth, weights, workloads
from helpers import note, to_np

pytestmark = pytest.mark.gpu
DEV = "cuda"
H, G, D, PAGE, HID = 2, 4, 64, 32, 256
Hq = H * G
WIDTH = (Hq + 2 * H) * D


def i32(a):
    return torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)


class Loop:
    """One layer's state and one step of it."""

    def __init__(self, fmt, R, max_tokens, pages=64, nb=24, seed=0, q8=False):
        g = np.random.default_rng(seed)
        self.fmt, self.R, self.pages, self.nb, self.max_tokens, self.q8 = fmt, R, pages, nb, max_tokens, q8
        free = g.permutation(pages)
        self.plain = ref.Tables(PAGE, [0] * R, np.full((R, nb), -1), free)
        self.lens, self.table, self.free, self.count = i32([0] * R), i32(np.full((R, nb), -1)), i32(free), i32([pages])
        self.add, self.keep = i32([0] * R), i32([0] * R)
        self.cache = pkg.KVCache.empty(pages, PAGE, H, D, fmt, DEV)
        self.norm_w = torch.from_numpy(1 + 0.1 * g.standard_normal(HID)).to(torch.bfloat16).to(DEV)
        self.signs = torch.from_numpy((g.integers(0, 2, HID) * 2 - 1).astype(np.int8)).to(DEV)
        m = synth.q8_matrix(7, WIDTH, HID) if q8 else synth.q4_matrix(7, WIDTH, HID)
        self.w = weights.pack_q8(m, DEV) if q8 else weights.pack_q4(m, DEV)
        M = max_tokens
        self.x = torch.zeros(M, HID, dtype=torch.bfloat16, device=DEV)
        self.res = torch.zeros(M, HID, dtype=torch.bfloat16, device=DEV)
        self.res_out = torch.zeros_like(self.res)
        self.y = torch.zeros(M, HID, dtype=torch.bfloat16, device=DEV)
        self.Xq, self.sx = torch.zeros(M, HID, dtype=torch.int8, device=DEV), torch.zeros(M, device=DEV)
        self.qkv = torch.zeros(M, WIDTH, dtype=torch.bfloat16, device=DEV)
        self.out = torch.zeros(M, Hq, D, dtype=torch.bfloat16, device=DEV)
        self.q_start, self.slots, self.pos, self.status = (i32([0] * n) for n in (R + 1, M, M, 1))
        n = pkg.kv_attention_workspace_bytes(R, M, Hq, H, D, PAGE, 32, nb * PAGE)
        self.ws = torch.empty(max(n, 1), dtype=torch.uint8, device=DEV)

    def run(self):
        M = self.max_tokens
        pkg.kv_tables_run(PAGE, self.lens, self.add, self.table, self.free, self.count, M, keep=self.keep,
                          q_start=self.q_start, slots=self.slots, positions=self.pos, status=self.status)
        if self.q8:
            pkg.rmsnorm_quant_run(self.x, self.norm_w, 1e-6, residual=self.res, residual_out=self.res_out, signs=self.signs,
                                  Xq=self.Xq, x_scales=self.sx)
            pkg.qgemm_skinny_run(pkg.FMT_Q8_SYM_G32, self.w, M, WIDTH, HID, self.Xq, self.sx, Y=self.qkv)
        else:
            pkg.rmsnorm_quant_run(self.x, self.norm_w, 1e-6, residual=self.res, residual_out=self.res_out, y=self.y)
            pkg.qgemm_skinny_run(pkg.FMT_Q4_ASYM_G64, self.w, M, WIDTH, HID, self.y, Y=self.qkv)
        rows = self.qkv.view(M, Hq + 2 * H, D)
        pkg.kv_append_run(self.cache, rows[:, Hq:Hq + H], rows[:, Hq + H:], self.slots)
        pkg.kv_attention_run(self.cache, rows[:, :Hq], self.q_start, self.lens, self.table, 32, workspace=self.ws, out=self.out)

    def state(self):
        return [t.clone() for t in (self.lens, self.table, self.free, self.count, self.cache.k.view(torch.uint8),
                                    self.cache.v.view(torch.uint8), self.cache.k_scales, self.cache.v_scales, self.out,
                                    self.q_start, self.slots, self.pos, self.status, self.res_out)]

    def set(self, add, keep, seed):
        self.add.copy_(i32(add))
        self.keep.copy_(i32(keep))
        g = torch.Generator().manual_seed(seed)
        self.x.copy_(torch.randn(self.max_tokens, HID, generator=g).to(torch.bfloat16))
        self.res.copy_(torch.randn(self.max_tokens, HID, generator=g).to(torch.bfloat16))

    def checked(self, add, keep, seed):
        M, e4m3 = self.max_tokens, self.fmt == pkg.KV_E4M3
        self.set(add, keep, seed)
        old = [to_np(t.view(torch.uint8)).astype(np.uint8) if t.element_size() == 1 else to_np(t)
               for t in (self.cache.k, self.cache.v, self.cache.k_scales, self.cache.v_scales)]
        self.out.fill_(9.0)
        self.run()
        torch.cuda.synchronize()
        status, q_start, slots, pos = self.plain.step(add, keep, M)
        assert int(self.status) == status
        assert np.array_equal(self.q_start.cpu(), q_start) and np.array_equal(self.slots.cpu(), slots) and np.array_equal(self.pos.cpu(), pos)
        assert np.array_equal(self.lens.cpu(), self.plain.lens) and np.array_equal(self.table.cpu(), self.plain.table)
        if not self.q8:
            r, y, _, _ = ref.norm(to_np(self.x), to_np(self.norm_w), np.float64(np.float32(1e-6)), to_np(self.res))
            assert np.all(np.abs(to_np(self.y) - y) <= (2.0 ** -8 + 2.0 ** -17) * np.abs(y))
        qkv = to_np(self.qkv).reshape(M, Hq + 2 * H, D)
        new = []
        for i, (a, b) in enumerate(((Hq, Hq + H), (Hq + H, Hq + 2 * H))):
            want, sc = ref.append(old[i], old[2 + i], qkv[:, a:b], slots, bool(i), e4m3)
            got = (self.cache.k, self.cache.v)[i].view(torch.uint8).cpu().numpy()
            gsc = (self.cache.k_scales, self.cache.v_scales)[i].cpu().numpy()
            assert np.array_equal(got, want) and np.array_equal(gsc, sc.astype(np.float32))
            new.append((ref.to_rows(want, bool(i)), sc))
        o, A, S = ref.attention(new[0][0], new[1][0], new[0][1], new[1][1], e4m3, qkv[:, :Hq], q_start, self.plain.lens, self.plain.table)
        n = max(self.plain.lens)
        vmax = new[1][1].max() * (448 if e4m3 else 127)
        tol = 2.0 ** -8 * np.abs(o) + (2.0 ** -11 + (D + 4) * 2.0 ** -22 * S[:, :, None] + 2 * n * 2.0 ** -24 + 2.0 ** -20) * A + n * 2.0 ** -24 * vmax
        got, seen = to_np(self.out), ~np.isnan(o)
        assert np.all(np.abs(got - o)[seen] <= tol[seen] + 1e-30)
        assert np.all(got[q_start[-1]:] == 9.0)
        return status


@pytest.mark.parametrize("fmt", [pkg.KV_INT8, pkg.KV_E4M3])
@pytest.mark.parametrize("q8", [False, True])
def test_a_decode_loop(fmt, q8):
    note("decode loop fmt=%d q8=%s" % (fmt, q8))
    p = Loop(fmt, 3, 32, q8=q8)
    lens = lambda: list(p.plain.lens)  # noqa: E731
    assert p.checked([29, 0, 3], lens(), 1) == 0              # prompts
    assert p.checked([16, 0, 16], lens(), 2) == 0             # a verification tile
    a, b, c = lens()
    assert p.checked([8, 16, 1], [a - 11, b, c - 16], 3) == 0  # most drafts rejected, a request comes in
    for k in range(4):
        assert p.checked([1, 1, 1], lens(), 4 + k) == 0
    a, b, c = lens()
    assert p.checked([1, 1, 30], [a, b, 0], 9) == 0           # the third is finished and replaced
    assert p.checked([32, 0, 0], lens(), 10) == 0
    assert p.checked([0, 0, 0], [0, 0, 0], 11) == 0           # all finished
    assert int(p.count) == p.pages


def test_a_step_that_cannot_be_done_changes_nothing():
    p = Loop(pkg.KV_INT8, 2, 32, pages=3, nb=4)
    assert p.checked([30, 2], [0, 0], 1) == 0
    assert p.checked([16, 16], list(p.plain.lens), 2) == 0    # the third page
    assert p.checked([20, 12], list(p.plain.lens), 3) == 1    # no page left: append and attention do nothing
    assert p.checked([1, 1], list(p.plain.lens), 4) == 0


@pytest.mark.parametrize("nb", [24, 80])
def test_captured_steps_equal_eager_ones(nb):
    """Two loops captured as two graphs, each with its own workspace, replayed
    in turn with new lengths and inputs; a third runs the same steps eagerly."""
    loops = [Loop(pkg.KV_INT8, 3, 32, nb=nb, pages=200, seed=5) for _ in range(3)]
    first = loops[0].state()
    graphs = [workloads.capture_graph(p.run) for p in loops[:2]]
    # capturing ran each step once with nothing to do
    assert all(torch.equal(a, b) for a, b in zip(first[:4], loops[0].state()[:4]))
    g = np.random.default_rng(3)
    lens = np.zeros(3, np.int64)
    for rep in range(12):
        add = [28, 3, 1] if rep == 0 else g.integers(0, 11, 3).tolist()
        keep = np.maximum(lens - g.integers(0, 9, 3) * (rep % 2), 0).tolist()
        for p, run in zip(loops, (graphs[0].replay, graphs[1].replay, loops[2].run)):
            p.set(add, keep, 100 + rep)
            run()
        torch.cuda.synchronize()
        states = [p.state() for p in loops]
        for s in states[1:]:
            assert all(torch.equal(a, b) for a, b in zip(states[0], s)), rep
        assert int(loops[0].status) == 0
        lens = loops[0].lens.cpu().numpy().copy()
        _ = torch.randn(1000, device=DEV).sum().item()  # unrelated eager work in between


def test_two_streams_at_once():
    """Two requests' loops on two streams, run together, equal each alone."""
    alone, both = [], []
    for mode, keep in ((0, alone), (1, both)):
        loops = [Loop(pkg.KV_E4M3, 2, 32, nb=40, pages=100, seed=i) for i in range(2)]
        streams = [torch.cuda.Stream() for _ in loops]
        for step in range(5):
            for p in loops:
                p.set([9 + step, 16 - step], [10 ** 6] * 2, step)
            torch.cuda.synchronize()
            for p, s in zip(loops, streams):
                with torch.cuda.stream(s):
                    p.run()
                if not mode:
                    torch.cuda.synchronize()
            torch.cuda.synchronize()
        keep += [p.state() for p in loops]
    for a, b in zip(alone, both):
        assert all(torch.equal(x, y) for x, y in zip(a, b))
