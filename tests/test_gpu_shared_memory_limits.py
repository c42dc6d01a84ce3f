"""GPU: calls whose kernels ask for different amounts of shared memory, one
after the other and at the same time. The limit on a kernel's dynamic shared
memory belongs to the function in the whole process, so what one call sets
must do for every other call, whatever its plan, thread or sizes."""

import ctypes
import subprocess

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


# Two threads in C, which meet more often than Python's: each makes one call
# again and again, its arguments as 64-bit words (the scale in millionths).
HAMMER = r"""
#include <pthread.h>
typedef long long w;
typedef void* p;
typedef int (*prefill)(p, p, int, int, p, p, p, int, p, int, int, int, int, int, int, int, float, int, int, int, p, int, p, p);
typedef int (*maps)(p, p, int, p, int, p, p, int, int, int, int, p, p, p, p, int, p, p, p);
typedef int (*scores)(p, p, p, int, p, int, int, int, int, int, int, int, p, p, p, p);
struct job { int kind; p f; const w* a; int times, status; };
#define P(i) ((p)a[i])
#define I(i) ((int)a[i])
static int call(int kind, p f, const w* a) {
    if (kind == 0)
        return ((prefill)f)(P(0), P(1), I(2), I(3), P(4), P(5), P(6), I(7), P(8), I(9), I(10), I(11), I(12), I(13), I(14),
                            I(15), a[16] * 1e-6f, I(17), I(18), I(19), P(20), I(21), P(22), P(23));
    if (kind == 1)
        return ((maps)f)(P(0), P(1), I(2), P(3), I(4), P(5), P(6), I(7), I(8), I(9), I(10), P(11), P(12), P(13), P(14),
                         I(15), P(16), P(17), P(18));
    return ((scores)f)(P(0), P(1), P(2), I(3), P(4), I(5), I(6), I(7), I(8), I(9), I(10), I(11), P(12), P(13), P(14), P(15));
}
static void* work(void* x) {
    struct job* j = x;
    for (int i = 0; i < j->times && j->status == 0; ++i) j->status = call(j->kind, j->f, j->a);
    return 0;
}
int hammer(int kind, p f, const w* a, const w* b, int times) {
    struct job j[2] = {{kind, f, a, times, 0}, {kind, f, b, times, 0}};
    pthread_t t[2];
    for (int i = 0; i < 2; ++i) pthread_create(&t[i], 0, work, &j[i]);
    for (int i = 0; i < 2; ++i) pthread_join(t[i], 0);
    return j[0].status ? j[0].status : j[1].status;
}
"""
PREFILL, MAPS, SCORES = range(3)


@pytest.fixture(scope="module")
def hammer(tmp_path_factory):
    at = tmp_path_factory.mktemp("hammer")
    (at / "hammer.c").write_text(HAMMER)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-pthread", "-o", at / "hammer.so", at / "hammer.c"], check=True)
    f = ctypes.CDLL(str(at / "hammer.so")).hammer
    f.argtypes = [ctypes.c_int, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_void_p, ctypes.c_int]

    def run(kind, fn, first, second, times):
        streams = [torch.cuda.Stream() for _ in range(2)]   # the last argument of every call
        words = [(ctypes.c_longlong * (len(a) + 1))(*[x or 0 for x in a], s.cuda_stream)
                 for a, s in zip((first, second), streams)]
        torch.cuda.synchronize()
        assert f(kind, ctypes.cast(fn, ctypes.c_void_p), *words, times) == pa.PA_OK
        torch.cuda.synchronize()
    return run


def test_windowed_prefills_of_two_threads(hammer):
    rng = np.random.default_rng(1)
    cases = [Case(rng.integers(1, 40, size=B).tolist(), [1] * B, Hq=2, Hkv=1, W=16, S=0, seed=B, scale=0.125).upload()
             for B in (7000, 3)]
    p = lambda t: t.data_ptr()  # noqa: E731
    pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_TWO_TILE)
    try:
        want = [c.run(prefill=True) for c in cases]
        got = [torch.zeros_like(w) for w in want]
        args = []
        for c, out in zip(cases, got):
            d = c.d
            args.append((p(d["q"]), p(d["start"]), c.T, 1, p(d["k"]), p(d["v"]), p(d["table"]), c.MB, p(d["lens"]), c.B,
                         2, 1, 128, c.bs, c.NB, max(c.lens), 125000, c.W, c.S, pa.PA_BF16, p(out), pa.PA_BF16,
                         ctypes.addressof(c.plan.handle)))
        hammer(PREFILL, pa.lib().pa_prefill_window, *args, times=3000)
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)
    for c, w, g in zip(cases, want, got):
        assert torch.equal(w, g)
        c.check(g, prefill=True, rows=set(range(0, c.B, max(1, c.B // 40))))


def test_step_maps_of_two_threads(hammer):
    from test_gpu_step_maps import Step, check
    p = lambda t: t.data_ptr()  # noqa: E731
    steps = [Step([5] * B, [1] * B).upload() for B in (8192, 6000)]
    args = []
    for s in steps:
        s.call()
        check(s)
        d, o = s.d, s.o
        args.append((p(d["cache"]), p(d["new"]), s.B, p(d["free"]), len(s.free), p(d["count"]), p(d["table"]),
                     s.MB, s.bs, s.NB, s.limit, p(o["seq"]), p(o["start"]), p(o["pos"]), p(o["slots"]), s.T,
                     p(o["left"]), p(o["err"])))
    hammer(MAPS, pa.lib().pa_step_maps, *args, times=10000)
    for s in steps:
        check(s)


def test_page_scores_of_two_threads(hammer):
    def inputs(B, Hkv, D, NB=50, bs=16):
        g = torch.Generator(device="cuda")
        g.manual_seed(B)
        k, v = (torch.randn(NB, Hkv, bs, D, generator=g, device="cuda").bfloat16() for _ in range(2))
        table = torch.randint(0, NB, (B, 4), generator=g, device="cuda", dtype=torch.int32)
        lens = torch.randint(1, 64, (B,), generator=g, device="cuda", dtype=torch.int32)
        return [k, v, table, lens, torch.zeros(B, 4, device="cuda"), torch.zeros(B, dtype=torch.int32, device="cuda")]

    p = lambda t: t.data_ptr()  # noqa: E731
    data, args, want = [inputs(2000, 1, 128), inputs(3, 1, 64)], [], []
    for k, v, table, lens, scores, victims in data:
        pa.pa_page_scores(k, v, table, lens, 64, scores, victims)
        torch.cuda.synchronize()
        want.append((scores.clone(), victims.clone()))
        args.append((p(k), p(v), p(table), 4, p(lens), len(lens), 1, k.shape[3], 16, 50, 64, pa.PA_BF16,
                     p(scores), p(victims), None))
    hammer(SCORES, pa.lib().pa_page_scores, *args, times=5000)
    for w, (*_, scores, victims) in zip(want, data):
        assert torch.equal(w[0], scores) and torch.equal(w[1], victims)


@pytest.mark.parametrize("B,D,bs,dtype", [
    (8192, 128, 16, torch.bfloat16), (8192, 64, 32, torch.float32), (4500, 128, 16, torch.bfloat16),
    (9, 128, 32, torch.float32), (8192, 128, 32, torch.float32),
])
def test_page_scores_of_many_sequences_and_large_pages(B, D, bs, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(B + D)
    k, v = (torch.randn(40, 2, bs, D, generator=g, device="cuda").to(dtype) for _ in range(2))
    table = torch.randint(0, 40, (B, 3), generator=g, device="cuda", dtype=torch.int32)
    lens = torch.randint(1, 3 * bs + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    scores = torch.full((B, 3), -7.0, device="cuda")
    victims = torch.zeros(B, dtype=torch.int32, device="cuda")
    pa.pa_page_scores(k, v, table, lens, 3 * bs, scores, victims)
    torch.cuda.synchronize()
    norm = lambda x: x.double().pow(2).sum((1, 3)).sqrt()  # noqa: E731
    ratio = (norm(v) / norm(k))[table.long()]                     # [B, 3, bs]
    left = (lens[:, None] - torch.arange(3, device="cuda") * bs).clamp(0, bs)
    valid = torch.arange(bs, device="cuda") < left[:, :, None]
    want = (ratio * valid).sum(-1) / left.clamp(min=1)
    # Sums of 2 D squares and a mean of bs quotients in 32 bits: below 1e-4 of the value.
    assert bool(((scores - want).abs() <= 1e-4 * want)[left > 0].all())
    assert bool((scores[left == 0] == -7.0).all())
    full = lens % bs == 0
    assert bool((victims[~full] == -1).all())
    at = victims.long().clamp(min=0)
    least = torch.where(left == bs, want, torch.inf).min(1).values
    assert bool((want.gather(1, at[:, None])[:, 0] <= least * (1 + 2e-4))[full].all())
