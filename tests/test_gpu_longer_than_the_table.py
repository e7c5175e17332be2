"""GPU: a prefix, or a request, of more tokens than its table's pages hold is
longer than the call was told of, also where that is all the table holds: rows
of NaN."""
import pytest
import torch

import quantized_weight_decode_dequant_amd as pkg
from helpers import note
from test_gpu_kv_attention import Case as Alone
from test_gpu_kv_prefix import Case, i32

pytestmark = pytest.mark.gpu
# the one line; the requests' kernel joins; a kernel joins
PLANS = [dict(lens=[1, 40, 7], T=[1, 1, 1], G=4), dict(lens=[5 + i for i in range(40)], T=[1] * 40, G=4),
         dict(lens=[3000] * 3 + [5] * 3, T=[3] * 6, G=8, D=256)]


@pytest.mark.parametrize("plan", range(3))
@pytest.mark.parametrize("P", [704, 705, 2 ** 31 - 1])
def test_prefix(plan, P):
    note("prefix of %d tokens in 11 pages, plan %d" % (P, plan))
    c = Case(plan, 704, **PLANS[plan])
    a = dict(c.args(), prefix_table=i32(c.prefix[:11]), prefix_len=i32([P]))
    got = pkg.kv_prefix_attention_run(c.cache(), **a)
    torch.cuda.synchronize()
    if P == 704:
        c.check(got)
    else:
        assert bool(got.isnan().all())


@pytest.mark.parametrize("plan", range(3))
@pytest.mark.parametrize("more", [1, 2 ** 30])
def test_request_behind_a_prefix(plan, more):
    c = Case(plan, 700, **PLANS[plan])
    a = c.args()
    want = pkg.kv_prefix_attention_run(c.cache(), **a)
    r = 1
    a["lens"][r] = c.cols * c.page + more
    got = pkg.kv_prefix_attention_run(c.cache(), **a)
    torch.cuda.synchronize()
    lo, hi = int(c.q_start[r]), int(c.q_start[r + 1])
    assert bool(got[lo:hi].isnan().all()) and bool(got[:lo].isfinite().all()) and bool(got[hi:].isfinite().all())
    c.check(want)


@pytest.mark.parametrize("lens", [[100, 90], [3000, 2500]])
@pytest.mark.parametrize("kw", [dict(), dict(window=64)])
def test_request_alone(lens, kw):
    c = Alone(34, lens, [6, 3], D=64)
    a = c.args()
    a["lens"][0] = a["table"].shape[1] * c.page + 1
    got = pkg.kv_attention_run(c.cache(), **a, **kw)
    torch.cuda.synchronize()
    assert bool(got[:6].isnan().all()) and bool(got[6:].isfinite().all())
