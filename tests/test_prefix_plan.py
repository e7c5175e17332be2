"""The plan of an attention call behind a shared prefix (tests/prefix_plan.py):
the library's workspace sizes are the plain rule's."""
import random
import time

import pytest

import quantized_weight_decode_dequant_amd as pkg
from prefix_plan import plan


def calls(seed, n):
    r = random.Random(seed)
    far = lambda top: int(2 ** r.uniform(0, top))  # noqa: E731
    for _ in range(n):
        R, Hkv, G, max_q = far(12), far(6), r.choice([1, 2, 3, 4, 5, 7, 8, 16, 71]), far(5)
        M = r.choice([R, R * max_q, far(5), far(15), 1])
        max_len, max_prefix = far(14), r.choice([0, far(8), far(20), far(30)])
        if Hkv * G <= 8192 and M * Hkv * G <= 1 << 26 and R * max_q * Hkv * G < 1 << 26:
            yield R, M, Hkv * G, Hkv, r.choice([64, 128, 256]), max_q, max_len, max_prefix


@pytest.mark.parametrize("seed", range(4))
def test_sizes_are_the_rules(seed):
    seen, n = set(), 0
    for R, M, Hq, Hkv, D, max_q, max_len, max_prefix in calls(seed, 700):
        got = pkg.kv_prefix_attention_workspace_bytes(R, M, Hq, Hkv, D, 64, max_q, max_len, max_prefix)
        if got == 0:  # (refused: too much work for 31 bits)
            continue
        want = plan(R, M, Hq, Hkv, D, max_q, max_len, max_prefix)
        assert got == want["bytes"], (R, M, Hq, Hkv, D, max_q, max_len, max_prefix, want)
        seen.add((want["kind"], want["shape"]))
        n += 1
    assert n > 300 and {k for k, _ in seen} == {"line", "last", "cut", "even"}


@pytest.mark.parametrize("R,Hq,Hkv", [(1, 8, 1), (1, 32, 8), (24, 1, 1), (8, 64, 1), (48, 32, 8)])
@pytest.mark.parametrize("max_prefix", [32768, 131072, 1 << 20])
def test_sizes_cost_no_search_of_all_parts(R, Hq, Hkv, max_prefix):
    """A call plans on the host each time, beside kernels of 20 us: with a long
    prefix no more than eight times what it takes with a page (trying each number
    of parts: up to 13)."""
    f = pkg.raw().qg_kv_prefix_attention_workspace_bytes

    def least(P):
        best = 1.0
        for _ in range(300):
            t = time.perf_counter()
            f(R, R, Hq, Hkv, 128, 64, 1, 4096, P)
            best = min(best, time.perf_counter() - t)
        return best

    assert least(max_prefix) < 8 * least(32)
