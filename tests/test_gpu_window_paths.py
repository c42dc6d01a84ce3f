"""GPU: every build behind the windowed calls, each shown to be the one that
ran: the persistent prefill that cuts its last turn's items into parts after
complete turns, the split decode in all head and block sizes, the workspace of
the split decode under capture, and the cluster decode's fixed order of sums."""

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from test_gpu_window import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


@pytest.fixture
def two_tile():
    pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_TWO_TILE)
    try:
        yield
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def runs_in_parts(c):
    """One call on a fresh plan; whether it took the memory of the parts (133 KB
    for every SM, in place of an item list of some KB)."""
    out = torch.empty(c.q.shape, dtype=torch.bfloat16, device="cuda")
    c.plan = pa.Plan()
    c.run(prefill=True, out=out)
    c.plan.free()
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    c.run(prefill=True, out=out)
    torch.cuda.synchronize()
    return free - torch.cuda.mem_get_info()[0] > sms() * 100_000


def mixed(seed, n):
    """Sequences of many lengths and query counts, whole tiles in most."""
    rng = np.random.default_rng(seed)
    ns = [64 if rng.random() < 0.8 else int(rng.integers(1, 200)) for _ in range(n)]
    lens = [int(x + rng.integers(0, 5000)) for x in ns]
    return lens, ns


@pytest.mark.parametrize("lens,ns,W,S", [
    ([4300] * 80, [64] * 80, 4096, 4),        # 160 items: one turn, then a few in parts
    ([5200] * 166, [64] * 166, 3400, 70),     # 332: two turns before
    (*mixed(1, 72), 4096, 4),                 # the host's estimate is not the number of items
    (*mixed(2, 154), 3100, 0),
])
@pytest.mark.parametrize("bs", [16, 32])
def test_parts_after_complete_turns(lens, ns, W, S, bs, two_tile):
    Hkv, g = 2, 4
    estimate = -(-sum(ns) // 64) * Hkv
    assert estimate > sms() and 0 < 2 * (estimate % sms()) <= sms(), "not cut: other counts are needed"
    c = Case(lens, ns, Hq=Hkv * g, Hkv=Hkv, W=W, S=S, bs=bs, seed=W).upload()
    assert runs_in_parts(c)
    out = c.run(prefill=True)
    again = [c.run(prefill=True) for _ in range(3)]
    # Rows of every sequence at the front and back, whose items are whole or in parts.
    rows, at = set(), 0
    for b, n in enumerate(ns):
        if b % 7 == 0 or b > len(ns) - 8:
            rows |= {at, at + n - 1}
        at += n
    c.check(out, prefill=True, rows=rows)
    assert bool(torch.isfinite(out).all())
    for x in again:
        assert torch.equal(out, x)


def test_calls_that_are_not_cut(two_tile):
    # More than half of the blocks in the last turn; a short window.
    for lens, ns, W in (([4300] * 120, [64] * 120, 4096), ([4300] * 80, [64] * 80, 2000)):
        c = Case(lens, ns, Hq=8, Hkv=2, W=W, S=4, seed=W).upload()
        assert not runs_in_parts(c)
        c.check(c.run(prefill=True), prefill=True, rows={0, 100, c.T - 1})


@pytest.mark.parametrize("Hq", [1, 4, 8, 9, 16])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32])
def test_split_decode_of_every_size(Hq, D, bs):
    c = Case([40000], Hq=Hq, Hkv=1, D=D, W=33000, S=19, bs=bs, seed=Hq + D).upload()
    c.check(c.run())
    assert c.plan.info()[1] > 8          # more blocks than a cluster has
    c.check(c.run(out_dtype=torch.float32))


def test_split_decode_wrong_lengths_and_entries():
    c = Case([40000, 39000], Hq=4, Hkv=1, W=33000, S=19, seed=1).upload()
    good = c.run()
    c.check(good)
    assert c.plan.info()[1] > 16
    c.d["lens"][0] = 50000
    out = c.run(max_len=40000)
    assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_SEQ_LEN
    assert bool((out[0] == 0).all())
    d0, d1 = out[1].double(), good[1].double()
    assert float((d0 - d1).abs().max()) <= 2.0 ** -7 * float(d1.abs().max())
    c.upload()
    c.d["table"][1, 39000 // 16 - 5] = c.NB
    out = c.run()
    assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_TABLE
    assert bool((out[1] == 0).all())
    c.upload()
    c.check(c.run())


def test_split_decode_graph_outlives_a_growing_plan():
    c = Case([40000], Hq=4, Hkv=1, W=33000, S=19, seed=1).upload()
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    c.run(out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(out=out)
    big = Case([40000, 36000, 39999], Hq=16, Hkv=1, W=33000, S=4, seed=2)
    big.plan = c.plan
    big.upload()
    before = c.plan.info()[1]
    big.check(big.run())
    assert before > 8 and c.plan.info()[1] > 24
    for seed in (3, 4):
        other = Case([40000], Hq=4, Hkv=1, W=33000, S=19, seed=seed)
        for name in ("q", "k", "v"):
            c.d[name].copy_(getattr(other, name))
        c.d["table"].copy_(torch.from_numpy(other.table))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        other.plan = c.plan
        other.check(out)


def test_a_capture_cannot_grow_the_split_decode():
    c = Case([700], Hq=4, Hkv=1, W=5000, S=0, seed=1).upload()
    d, res = c.d, torch.empty(c.q.shape, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode(d["q"], d["k"], d["v"], d["table"], d["lens"], c.scale, res, 700, c.plan)   # a small workspace
    big = Case([40000, 36000, 39999], Hq=16, Hkv=1, W=33000, S=4, seed=2)
    big.plan = c.plan
    big.upload()
    out = torch.zeros(big.q.shape, dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(pa.PagedAttentionError) as e:
            big.run(out=out)
        assert e.value.status == pa.PA_ERR_WORKSPACE
        out.add_(1.0)                    # the capture goes on
    g.replay()
    torch.cuda.synchronize()
    assert bool((out == 1.0).all())
    big.check(big.run())


@pytest.mark.parametrize("lens,W", [([3000, 40, 900], 500), ([9000], 8191), ([700] * 200, 256)])
def test_cluster_decode_gives_the_same_bits(lens, W):
    c = Case(lens, W=W, S=4).upload()
    a = c.run()
    assert c.plan.info()[1] in {len(lens) * 2 * n for n in (1, 2, 4, 8)}    # a cluster for every (sequence, kv head)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = c.run(stream=side)
    side.synchronize()
    assert torch.equal(a, b)
    for _ in range(3):
        assert torch.equal(a, c.run())
    c.check(a, rows=set(range(0, len(lens), 1 + len(lens) // 10)))
