"""GPU: calls whose kernels ask for different amounts of shared memory, one
after the other and at the same time. The limit on a kernel's dynamic shared
memory belongs to the function in the whole process, so what one call sets
must do for every other call, whatever its plan, thread or sizes."""

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


def plain(c, plan, noalloc=False):
    """The whole context (the case's window covers it) by the plain decode."""
    d, out = c.d, torch.full(c.q.shape, 7.5, dtype=torch.bfloat16, device="cuda")
    if noalloc:
        pa.pa_decode_noalloc(d["q"], d["k"], d["v"], d["table"], d["lens"], c.scale, out, max(c.lens))
    else:
        pa.pa_decode(d["q"], d["k"], d["v"], d["table"], d["lens"], c.scale, out, max(c.lens), plan)
    torch.cuda.synchronize()
    return out


def small(B, Hq, Hkv=1, D=128):
    rng = np.random.default_rng(B + Hq)
    return Case(rng.integers(1, 200, size=B).tolist(), Hq=Hq, Hkv=Hkv, D=D, W=1000, S=0, seed=B + Hq).upload()


@pytest.mark.parametrize("plans", ["one_plan", "own_plans", "no_plan"])
@pytest.mark.parametrize("sizes", [
    [(4, 8), (4, 4), (4, 8)],          # query heads per kv head of one kernel
    [(4, 16), (4, 9), (4, 16)],        # ... and of the one for more than eight
    [(900, 8), (4, 8), (900, 8)],      # sequences
], ids=["groups_to_8", "groups_to_16", "batches"])
def test_plain_decodes_of_different_sizes(sizes, plans):
    cases = {}
    shared = pa.Plan()
    own = {}
    for B, Hq in sizes:
        if (B, Hq) not in cases:
            cases[B, Hq] = small(B, Hq)
        c = cases[B, Hq]
        plan = shared if plans == "one_plan" else own.setdefault((B, Hq), pa.Plan())
        c.compare(plain(c, plan, noalloc=plans == "no_plan"), rows=set(range(0, B, max(1, B // 8))))
    for p in [shared, *own.values()]:
        p.free()


@pytest.mark.parametrize("one_plan", [True, False])
@pytest.mark.parametrize("groups", [(8, 4, 8), (16, 9, 16)])
def test_split_windowed_decodes_of_different_sizes(groups, one_plan):
    plan, cases = pa.Plan(), {}
    for Hq in groups:
        if Hq not in cases:
            cases[Hq] = Case([40000], Hq=Hq, Hkv=1, W=33000, S=19, seed=Hq)
            cases[Hq].plan = plan if one_plan else pa.Plan()
            cases[Hq].upload()
        c = cases[Hq]
        c.check(c.run())
        assert c.plan.info()[1] > 8      # the split kernels, not a cluster


@pytest.mark.parametrize("B,Hq", [(512, 9), (600, 9), (6783, 36)])
@pytest.mark.parametrize("noalloc", [False, True])
def test_decodes_that_fill_the_shared_memory(B, Hq, noalloc):
    # Sizes at which the stages, the query rows and the lengths come within a
    # few bytes of what a block may have.
    c = small(B, Hq)
    with pa.Plan() as plan:
        c.compare(plain(c, plan, noalloc), rows=set(range(0, B, B // 8)))
