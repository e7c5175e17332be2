"""GPU: block tables, slot maps, lengths and the free list, against the
bookkeeping done with lists (whole numbers: equal)."""
import numpy as np
import pytest
import torch

import cache_ref as ref
import quantized_weight_decode_dequant_amd as pkg
from helpers import note

pytestmark = pytest.mark.gpu
DEV = "cuda"


class Both:
    """The list form and the GPU's buffers, stepped together."""

    def __init__(self, page, R, nb, pages, seed=0):
        self.page, self.pages = page, pages
        free = np.random.default_rng(seed).permutation(pages)
        self.plain = ref.Tables(page, [0] * R, np.full((R, nb), -1), free)
        t = lambda a: torch.tensor(np.asarray(a), dtype=torch.int32, device=DEV)  # noqa: E731
        self.lens, self.table, self.free = t([0] * R), t(np.full((R, nb), -1)), t(free)
        self.count = t([pages])
        self.t = t

    def step(self, add, keep=None, max_tokens=None):
        n = int(sum(max(a, 0) for a in add)) + 3 if max_tokens is None else max_tokens
        status, q_start, slots, pos = self.plain.step(add, keep, n)
        got = pkg.kv_tables_run(self.page, self.lens, self.t(add), self.table, self.free, self.count, n,
                                keep=None if keep is None else self.t(keep))
        torch.cuda.synchronize()
        assert int(got[3]) == status
        for name, a, b in (("q_start", got[0], q_start), ("slots", got[1], slots), ("positions", got[2], pos),
                           ("lens", self.lens, self.plain.lens), ("table", self.table, self.plain.table)):
            assert np.array_equal(a.cpu().numpy(), np.asarray(b)[: a.numel()] if name in ("slots", "positions") else b), name
        n = int(self.count)
        assert n == len(self.plain.free) and self.free[:n].tolist() == self.plain.free
        return status


@pytest.mark.parametrize("page", [32, 64, 128, 256])
@pytest.mark.parametrize("R", [1, 2, 63, 1025, 4096])
def test_random_steps(page, R):
    note("tables page=%d R=%d" % (page, R))
    g = np.random.default_rng(page * 7919 + R)
    nb = 9
    b = Both(page, R, nb, R * 6 + 5, seed=R)
    refused = 0
    for step in range(12):
        lens = np.array(b.plain.lens)
        kind = g.integers(0, 4, R)
        add = np.where(kind == 0, g.integers(0, 17, R), np.where(kind == 1, g.integers(0, 2 * page, R), 1))
        add = np.minimum(add, nb * page - lens)
        keep = None if step % 3 == 0 else np.where(g.random(R) < 0.4, g.integers(-3, lens + 20, R), lens)
        refused += b.step(add.tolist(), None if keep is None else keep.tolist()) != 0
    assert refused < 12


@pytest.mark.parametrize("max_tokens", [0, 5, 5000])
def test_no_requests(max_tokens):
    """Nothing to do, but the outputs that later calls read are written."""
    t = lambda *a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    none, free, count = torch.empty(0, dtype=torch.int32, device=DEV), t(2, 0, 1), t(3)
    q_start, slots, pos, status = t(7), t(7).repeat(max_tokens), t(7).repeat(max_tokens), t(7)
    pkg.kv_tables_run(32, none, none, torch.empty(0, 4, dtype=torch.int32, device=DEV), free, count, max_tokens,
                      q_start=q_start, slots=slots, positions=pos, status=status)
    assert int(q_start) == 0 and int(status) == 0 and bool((slots == -1).all()) and not bool(pos.any())
    assert free.tolist() == [2, 0, 1] and int(count) == 3


def test_release_restores_the_list():
    b = Both(32, 5, 40, 300, seed=3)
    b.step([70, 0, 33, 1, 600])
    free, table = b.free.clone(), b.table.clone()
    b.step([16, 40, 1, 0, 500])
    b.step([0] * 5, keep=[70, 0, 33, 1, 600])
    n = int(b.count)
    assert torch.equal(free[:n], b.free[:n]) and torch.equal(table, b.table)


def test_refused_steps_change_nothing():
    b = Both(64, 3, 4, 6, seed=1)
    assert b.step([64, 65, 1]) == 0                      # 4 of 6 pages
    assert b.step([64, 64, 64]) == 1                     # 3 more: too few
    assert b.step([200, 0, 0]) in (2, 3)                 # a request past its table
    assert b.step([1, 1, 1], max_tokens=2) == 4
    assert b.step([193, 0, 100], max_tokens=5) & 6 == 6
    assert b.step([1, 0, 1]) == 0
    assert b.step([0, 0, 0], keep=[0, 0, 0]) == 0 and int(b.count) == 6


def test_empty_and_negative():
    b = Both(32, 4, 3, 20)
    assert b.step([0, 0, 0, 0]) == 0
    assert b.step([-5, 31, 0, -1]) == 0
    assert b.step([0, 1, 0, 0], keep=[-1, 100, 3, 0]) == 0
    assert b.step([0, 0, 0, 0], max_tokens=0) == 0
    assert b.step([1, 2, 3, 4], keep=[0, 0, 0, 0]) == 0


def test_a_free_count_that_cannot_be():
    for bad in (-1, 21):
        b = Both(32, 2, 3, 20)
        b.count.fill_(bad)
        table = b.table.clone()
        got = pkg.kv_tables_run(32, b.lens, b.t([1, 1]), b.table, b.free, b.count, 4)
        assert int(got[3]) == 1 and torch.equal(table, b.table) and int(b.count) == bad
        assert got[1].tolist() == [-1] * 4 and not b.lens.any()


def test_many_tokens_and_long_tables():
    """Prompts of many thousand tokens, and max_tokens far past them."""
    b = Both(32, 6, 4096, 9000, seed=9)
    note("tables long prompts")
    assert b.step([100003, 1, 0, 32, 33, 70001], max_tokens=200000) == 0
    assert b.step([1, 1, 1, 1, 1, 1]) == 0
    assert b.step([0, 5, 0, 0, 0, 0], keep=[5, 0, 0, 0, 0, 69000]) == 0


def test_graph_steps_on_its_own_buffers():
    """A captured step, replayed with new lengths written between, equals the
    list form each time."""
    from quantized_weight_decode_dequant_amd import workloads
    R, page, nb, pages = 33, 32, 30, 800
    plain = Both(page, R, nb, pages, seed=4)
    add, keep = plain.t([0] * R), plain.t([0] * R)
    outs = [torch.empty(n, dtype=torch.int32, device=DEV) for n in (R + 1, 2000, 2000, 1)]
    run = lambda: pkg.kv_tables_run(page, plain.lens, add, plain.table, plain.free, plain.count, 2000, keep=keep,  # noqa: E731
                                    q_start=outs[0], slots=outs[1], positions=outs[2], status=outs[3])
    graph = workloads.capture_graph(run)
    g = np.random.default_rng(11)
    for rep in range(6):
        lens = np.array(plain.plain.lens)
        a = g.integers(0, 50, R)
        k = np.where(g.random(R) < 0.3, g.integers(0, lens + 1), lens)
        add.copy_(plain.t(a))
        keep.copy_(plain.t(k))
        graph.replay()
        torch.cuda.synchronize()
        status, q_start, slots, pos = plain.plain.step(a, k, 2000)
        assert int(outs[3]) == status
        for x, y in ((outs[0], q_start), (outs[1], slots), (outs[2], pos), (plain.lens, plain.plain.lens), (plain.table, plain.plain.table)):
            assert np.array_equal(x.cpu().numpy(), y)
        assert plain.free[: int(plain.count)].tolist() == plain.plain.free


@pytest.mark.parametrize("max_tokens", [50, 5000])
@pytest.mark.parametrize("page", [32, 256])
def test_slots_of_pages_that_are_not_there(page, max_tokens):
    """Page ids outside the pool, from the table or the free list, give slots
    outside it too (-1), however large they are."""
    pages, bits = 20, page.bit_length() - 1
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    bad = [-1, pages, 1 << (32 - bits), (1 << (32 - bits)) + 3, 1 << (31 - bits), 2 ** 31 - 1, -2 ** 31]
    ids = bad + [3]
    lens, add = t([5] * len(ids) + [0] * len(ids)), t([3] * (2 * len(ids)))
    table = t([[i, -1] for i in ids] + [[-1, -1]] * len(ids))
    free, count = t(ids[::-1] + [-1] * (pages - len(ids))), t([len(ids)])
    got = pkg.kv_tables_run(page, lens, add, table, free, count, max_tokens)
    torch.cuda.synchronize()
    assert int(got[3]) == 0 and table[len(ids):, 0].tolist() == ids
    want = []
    for first in (5, 0):
        want += [3 * page + first + k if i == 3 else -1 for i in ids for k in range(3)]
    assert got[1].tolist() == want + [-1] * (max_tokens - len(want))


def test_outputs_that_are_longer_than_asked_for():
    """Buffers given for the largest step come back as they are, their tails
    untouched; the append takes no more slots than it has rows."""
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=DEV)  # noqa: E731
    big = [torch.full((40,), 7, dtype=torch.int32, device=DEV) for _ in range(4)]
    got = pkg.kv_tables_run(32, t([0, 0]), t([3, 2]), t([[-1], [-1]]), t([1, 0]), t([2]), 6, q_start=big[0], slots=big[1],
                            positions=big[2], status=big[3])
    assert all(a is b for a, b in zip(got, big))
    assert [x[:n].tolist() for x, n in zip(got, (3, 6, 6, 1))] == [[0, 3, 5], [0, 1, 2, 32, 33, -1], [0, 1, 2, 0, 1, 0], [0]]
    assert all(bool((b[n:] == 7).all()) for b, n in zip(big, (3, 6, 6, 1)))
    cache = pkg.KVCache.empty(2, 32, 1, 64)
    rows = torch.zeros(6, 1, 64, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="slots must be"):
        pkg.kv_append_run(cache, rows, rows, got[1])
