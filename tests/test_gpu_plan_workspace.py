"""GPU: what a plan's memory holds from call to call, and for how long. Calls of
every kind share a plan's workspace in any order, among them graphs captured
earlier and replayed in between; memory that a later call outgrows."""

import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from test_gpu_window import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def decode(c, plan, out=None):
    """pa_decode of a case whose window covers its sequences."""
    d = c.d
    if out is None:
        out = torch.full(c.q.shape, 7.5, dtype=torch.bfloat16, device="cuda")
    pa.pa_decode(d["q"], d["k"], d["v"], d["table"], d["lens"], c.scale, out, max(c.lens), plan)
    return out


def captured(call):
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    return g


def test_fused_merges_between_replays_of_a_windowed_graph():
    # The fused merge counts partials in memory that every call leaves zero. A
    # windowed graph that is replayed in between must not write there.
    few = Case([3000, 2500, 700, 40], Hq=16, Hkv=2, W=5000, S=0, seed=4).upload()
    c = Case([5000, 4500], [32, 32], W=4096, S=4, seed=1).upload()
    plan = c.plan
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    rows = set(range(0, c.T, 7))
    decode(few, plan)
    plan.set_merge(pa.PA_MERGE_FUSED)
    few.compare(decode(few, plan))
    c.run(prefill=True, out=out)
    g = captured(lambda: c.run(prefill=True, out=out))
    for _ in range(3):
        few.compare(decode(few, plan))
        g.replay()
    few.compare(decode(few, plan))
    assert plan.last_device_error() == 0
    c.check(out, prefill=True, rows=rows)


def test_a_captured_fused_merge_between_windowed_calls():
    few = Case([3000, 2500, 700, 40], Hq=16, Hkv=2, W=5000, S=0, seed=4).upload()
    c = Case([5000, 4500], [32, 32], W=4096, S=4, seed=1).upload()
    plan = c.plan
    res = torch.zeros(few.q.shape, dtype=torch.bfloat16, device="cuda")
    c.run(prefill=True)
    decode(few, plan)
    plan.set_merge(pa.PA_MERGE_FUSED)
    g = captured(lambda: decode(few, plan, res))    # the plan's first fused call
    for _ in range(2):
        c.check(c.run(prefill=True), prefill=True, rows={0, 40})
        res.fill_(7.5)
        g.replay()
        torch.cuda.synchronize()
        few.compare(res)
        few.compare(decode(few, plan))
    assert plan.last_device_error() == 0

@pytest.mark.parametrize("multi", [False, True])
def test_graph_replay_of_plain_calls_outlives_a_growing_plan(multi):
    # A captured pa_decode, or pa_decode_multi with its keys split over blocks,
    # and a larger call afterwards: the graph's memory stays its own.
    ns = [6, 6] if multi else None
    c = Case([3000, 2000], ns, W=5000, S=0, seed=1).upload()
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")

    def call():
        if not multi:
            return decode(c, c.plan, out)
        d = c.d
        pa.pa_decode_multi(d["q"], d["start"], d["k"], d["v"], d["table"], d["lens"], c.scale, out, 6, 3000, c.plan)

    call()
    g = captured(call)
    big = Case([2500] * 40, Hq=32, Hkv=8, W=5000, S=0, seed=2).upload()
    decode(big, c.plan)
    other = torch.randn(64 << 20, device="cuda")      # whatever was freed may be taken
    torch.cuda.synchronize()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    c.check(out, prefill=multi)
    assert bool(torch.isfinite(other).all())


@pytest.mark.parametrize("after_capture", [False, True])
def test_growing_calls_keep_a_bounded_amount_of_memory(after_capture):
    # Rows that creep up, in calls that each need over 20 MB: what is kept
    # stays within a few times of what the largest of them needs.
    T = 64 * 72
    c = Case([6000], [T], Hq=4, Hkv=1, W=4096, S=4, seed=3).upload()
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    starts = [torch.tensor([0, n], dtype=torch.int32, device="cuda") for n in range(64, T + 1, 64)]

    def call(start, n):
        d = c.d
        pa.pa_prefill_window(d["q"][:n], start, d["k"], d["v"], d["table"], d["lens"], c.scale, c.W, c.S,
                             out[:n], n, 6000, plan)

    pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_TWO_TILE)
    try:
        plan = c.plan
        call(starts[0], 64)
        g = captured(lambda: call(starts[0], 64)) if after_capture else None
        torch.cuda.synchronize()
        free = torch.cuda.mem_get_info()[0]
        for i, start in enumerate(starts):
            call(start, 64 * (i + 1))
        torch.cuda.synchronize()
        grown = free - torch.cuda.mem_get_info()[0]
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)
    assert grown < 100 << 20
    c.check(out, prefill=True, rows=set(range(0, T, 397)) | {T - 1})
    if g is not None:
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert plan.last_device_error() == 0


def one_segment(Hq, seed=0):
    """A windowed decode that runs the split kernels and uses the workspace."""
    return Case([40000], Hq=Hq, Hkv=1, W=33000, S=19, seed=seed).upload()


def test_a_forced_schedule_does_not_apply_to_windowed_calls():
    # A schedule in small pieces needs more memory: if a windowed call took it,
    # the capture would be refused.
    c = one_segment(8)
    c.check(c.run())
    c.plan.set_schedule(500, 1)
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    g = captured(lambda: c.run(out=out))
    g.replay()
    torch.cuda.synchronize()
    c.check(out)
