"""GPU: calls from a thread that has made no CUDA call before, such as a
server's worker, with a plan that another thread has used."""

import threading

import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from test_gpu_window import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


def prefill(c, out, plan, stream):
    d, n = c.d, max(c.ns)
    pa.pa_prefill(d["q"], d["start"], d["k"], d["v"], d["table"], d["lens"], c.scale, out, n, max(c.lens), stream=stream)


def multi(c, out, plan, stream):
    d, n = c.d, max(c.ns)
    pa.pa_decode_multi(d["q"], d["start"], d["k"], d["v"], d["table"], d["lens"], c.scale, out, n, max(c.lens), plan,
                       stream=stream)


def decode(c, out, plan, stream):
    d = c.d
    pa.pa_decode(d["q"], d["k"], d["v"], d["table"], d["lens"], c.scale, out, max(c.lens), plan, stream=stream)


def noalloc(c, out, plan, stream):
    d = c.d
    pa.pa_decode_noalloc(d["q"], d["k"], d["v"], d["table"], d["lens"], c.scale, out, max(c.lens), stream=stream)


def windowed(prefill):
    def call(c, out, plan, stream):
        c.plan = plan
        c.run(prefill=prefill, out=out, stream=stream)
    return call


@pytest.mark.parametrize("call,ns", [
    (prefill, [40, 70]), (multi, [40, 70]), (multi, [2, 3]), (decode, None), (noalloc, None),
    (windowed(True), [40, 70]), (windowed(False), None),
], ids=["prefill", "multi_tiles", "multi_columns", "decode", "noalloc", "prefill_window", "decode_window"])
def test_a_thread_new_to_cuda(call, ns):
    # The window covers the sequences, so that all calls compute the same.
    cases = [Case([300, 500], ns, W=1000, S=0, seed=s).upload() for s in (1, 2)]
    plan, stream = pa.Plan(), torch.cuda.current_stream()
    outs = [torch.full(c.q.shape, 7.5, dtype=torch.bfloat16, device="cuda") for c in cases]
    call(cases[0], outs[0], plan, stream)        # the plan exists, other pools follow
    torch.cuda.synchronize()
    errors = []

    def work():
        try:
            call(cases[1], outs[1], plan, stream)
        except Exception as e:  # noqa: BLE001
            errors.append(e)

    t = threading.Thread(target=work)
    t.start()
    t.join()
    torch.cuda.synchronize()
    assert not errors, errors
    for c, out in zip(cases, outs):
        c.compare(out, prefill=ns is not None)
    plan.free()
