"""GPU: rows of the windowed calls that are easily lost: rows behind the last
sequence of a padded batch, which every kernel leaves as they were, and rows
whose query or only visible key is not a number, which show it however the work
was split."""

import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from test_gpu_window import Case, kernel  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.mark.parametrize("lens,ns,W", [
    ([3000, 2000], [6, 6], 1000),             # keys split over blocks
    ([3000, 500, 2000], [6, 0, 0], 1000),
    ([300, 90], [70, 33], 64),
    ([5000], [40], 4500),                     # items in parts
    ([700] * 40, [100] * 40, 200),
])
def test_rows_of_the_padding_are_left_alone(lens, ns, W, kernel):  # noqa: F811
    c = Case(lens, ns, W=W, S=4, seed=1).upload()
    pad = 77
    q = torch.full((c.T + pad, 8, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[:c.T] = c.d["q"]
    out = torch.full_like(q, 7.5)
    d = c.d
    pa.pa_prefill_window(q, d["start"], d["k"], d["v"], d["table"], d["lens"], c.scale, c.W, c.S, out, max(ns),
                         max(lens), c.plan)
    torch.cuda.synchronize()
    assert bool((out[c.T:] == 7.5).all())
    c.check(out[:c.T], prefill=True, rows=set(range(0, c.T, 1 + c.T // 40)))


@pytest.mark.parametrize("lens,ns,W", [
    ([3000, 2000], [6, 6], 1000),             # keys split over blocks
    ([300, 190], [70, 33], 64),
    ([5000], [40], 4500),                     # items in parts
])
def test_a_query_that_is_not_a_number_shows_in_the_prefill(lens, ns, W, kernel):  # noqa: F811
    c = Case(lens, ns, W=W, S=4, seed=2)
    c.q[3, 5] = float("nan")
    c.upload()
    out = c.run(prefill=True)
    assert bool(torch.isnan(out[3, 5]).all())
    out[3, 5] = 0
    assert bool(torch.isfinite(out).all())
    c.check(out, prefill=True, rows=set(range(c.T)) - {3})


def test_the_only_key_of_a_part_shows(kernel):  # noqa: F811
    # 769 visible indices for six queries: seven chunks in three parts, the last
    # of one token, which only the last query sees.
    c = Case([2001], [6], W=760, S=0, seed=3)
    c.k[int(c.table[0, 2000 // 16]), 0, 2000 % 16] = float("nan")
    c.upload()
    out = c.run(prefill=True)
    assert bool(torch.isnan(out[5, :4]).all())
    out[5, :4] = 0
    assert bool(torch.isfinite(out).all())
    c.check(out, prefill=True, rows=set(range(5)))


@pytest.mark.parametrize("lens,Hq,Hkv,W", [
    ([300, 3000], 8, 2, 500), ([20000], 8, 1, 8191), ([40000], 8, 1, 33000), ([40000], 16, 1, 33000),
    ([40000, 38000], 12, 1, 33000),
])
def test_a_query_that_is_not_a_number_shows_in_the_decode(lens, Hq, Hkv, W):
    c = Case(lens, Hq=Hq, Hkv=Hkv, W=W, S=4, seed=2)
    c.q[0, 3] = float("nan")
    c.upload()
    for dtype in (torch.bfloat16, torch.float32):
        out = c.run(out_dtype=dtype)
        assert bool(torch.isnan(out[0, 3]).all())
        out[0, 3] = 0
        assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("Hq", [4, 12])
def test_keys_of_a_whole_part_show_in_the_split_decode(Hq):
    # Every key but those of the sinks' and of the last page.
    c = Case([40000], Hq=Hq, Hkv=1, W=33000, S=16, seed=5)
    for p in range(1, 40000 // 16 - 1):
        if 0 <= c.table[0, p] < c.NB:
            c.k[int(c.table[0, p])] = float("nan")
    c.upload()
    out = c.run()
    assert c.plan.info()[1] > 8
    assert bool(torch.isnan(out).all())
