"""GPU: sliding-window attention with sinks, one query and several per
sequence, against the 64-bit definition. Windows that begin and end anywhere
in a page, that touch or cover the sinks, sequences shorter than either; pages
that were given back (table entries -1 or outside the pool), NaN and infinities
in every hidden place; head groups, head sizes, block sizes, both prefill
kernels and the key split; wrong lengths and tables; captured graphs, side
streams and plans that grow. Tolerances: window_reference.tolerance."""

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from window_reference import attend, tokens_seen, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


class Case:
    def __init__(self, lens, ns=None, Hq=8, Hkv=2, D=128, bs=16, W=20, S=4, seed=0, hidden="nan", scale=None,
                 k_scale=1.0):
        self.lens, self.ns = list(lens), [1] * len(lens) if ns is None else list(ns)
        self.__dict__.update(Hq=Hq, Hkv=Hkv, D=D, bs=bs, W=W, S=S, scale=scale or D ** -0.5)
        rng = np.random.default_rng(seed)
        B = len(lens)
        self.B, self.T, self.MB = B, sum(self.ns), max(1, max(-(-max(x, 0) // bs) for x in lens)) + 1
        seen = []     # the tokens that some query of each sequence sees
        for L, n in zip(self.lens, self.ns):
            u = [tokens_seen(p, W, S) for p in {max(0, L - n), L - 1}] if L > 0 and n > 0 else []
            t = set(u[0]) if u else set()
            if u:
                t |= set(range(max(0, L - n - W + 1), L)) | set(range(min(S, L)))
            seen.append(t)
        pages = [sorted({t // bs for t in s}) for s in seen]
        self.NB = sum(map(len, pages)) + 3
        ids = rng.permutation(self.NB).astype(np.int32)
        bad = [-1, -5, self.NB, 2 ** 31 - 1]
        self.table = np.array([[bad[(b + i) % 4] for i in range(self.MB)] for b in range(B)], dtype=np.int32).reshape(B, self.MB)
        shape = (self.NB, Hkv, bs, D)
        bf = lambda x: torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)  # noqa: E731
        k, v = bf(rng.standard_normal(shape) * k_scale), bf(rng.standard_normal(shape))
        fill = {"nan": float("nan"), "inf": float("inf")}[hidden]
        keep = torch.zeros(self.NB, bs, dtype=torch.bool)
        at = 0
        for b, pg in enumerate(pages):
            for p in pg:
                self.table[b, p] = ids[at]
                for o in range(bs):
                    keep[ids[at], o] = p * bs + o in seen[b]
                at += 1
        hide = ~keep[:, None, :, None].expand(shape)
        k[hide], v[hide] = fill, fill
        self.k, self.v, self.q = k, v, bf(rng.standard_normal((self.T, Hq, D)))
        self.plan = None

    def upload(self):
        c = lambda x: x.cuda()  # noqa: E731
        self.d = dict(q=c(self.q), k=c(self.k), v=c(self.v), table=c(torch.from_numpy(self.table)),
                      lens=torch.tensor(self.lens, dtype=torch.int32, device="cuda"),
                      start=torch.tensor(np.concatenate([[0], np.cumsum(self.ns)]), dtype=torch.int32).cuda())
        self.plan = self.plan or pa.Plan()
        return self

    def run(self, prefill=False, out_dtype=torch.bfloat16, stream=None, out=None, max_q=None, max_len=None):
        d = self.d
        if out is None:
            out = torch.full(self.q.shape, 7.5, dtype=out_dtype, device="cuda")
        max_len = max_len or max(1, max(self.lens))
        if prefill:
            pa.pa_prefill_window(d["q"], d["start"], d["k"], d["v"], d["table"], d["lens"], self.scale, self.W,
                                 self.S, out, max_q or max(self.ns), max_len, self.plan, stream=stream)
        else:
            pa.pa_decode_window(d["q"], d["k"], d["v"], d["table"], d["lens"], self.scale, self.W, self.S, out,
                                max_len, self.plan, stream=stream)
        return out

    def check(self, out, prefill=False, rows=None):
        assert pa.pa_last_device_error(self.plan) == 0
        self.compare(out, prefill, rows)

    def compare(self, out, prefill=False, rows=None):
        got = out.double().cpu().numpy()
        q, k, v = (x.float().numpy() for x in (self.q, self.k, self.v))
        t = 0
        for b, (L, n) in enumerate(zip(self.lens, self.ns)):
            for i in range(n):
                if rows is None or t in rows:
                    ref, wv, mag = attend(q[t], k, v, self.table[b], L - n + i, self.scale, self.W, self.S)
                    tol = tolerance(ref, wv, mag, self.D, 8 if prefill else 16, out.dtype == torch.bfloat16)
                    bad = ~(np.abs(got[t] - ref) <= tol)
                    assert not bad.any(), (f"sequence {b} (length {L}) query {i}: {bad.sum()} off, worst "
                                           f"{np.nanmax(np.abs(got[t] - ref) / tol):.2f} of the tolerance")
                t += 1


# Lengths around a window of 20 (16-token pages), sinks inside and past a page.
EDGES = [1, 2, 15, 16, 17, 19, 20, 21, 23, 24, 25, 31, 32, 33, 36, 37, 40, 47, 48, 49, 63, 64, 65, 100, 333]


@pytest.mark.parametrize("W,S", [(1, 0), (1, 1), (16, 0), (20, 4), (20, 16), (20, 17), (33, 40), (5, 400),
                                 (1000, 4), (64, 64), (15, 1)])
@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_edges(W, S, bs, D):
    c = Case(EDGES, W=W, S=S, bs=bs, D=D, seed=W + S).upload()
    c.check(c.run())


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (3, 3), (6, 2), (8, 1), (9, 1), (16, 1), (32, 2), (40, 2), (34, 1), (128, 8)])
@pytest.mark.parametrize("hidden", ["nan", "inf"])
def test_decode_head_groups(Hq, Hkv, hidden):
    c = Case([1, 30, 77, 500, 129], Hq=Hq, Hkv=Hkv, W=50, S=5, hidden=hidden, seed=Hq).upload()
    c.check(c.run())
    c.check(c.run(out_dtype=torch.float32))


@pytest.mark.parametrize("B,lens,W,S", [
    (1, [4000], 1500, 4), (1, [20000], 8191, 64), (3, [9000, 40, 7000], 4096, 17), (64, None, 256, 4),
    (300, None, 100, 1), (40, None, 3000, 0),
])
def test_decode_sizes(B, lens, W, S):
    rng = np.random.default_rng(B)
    lens = lens or rng.integers(1, 4 * W, size=B).tolist()
    c = Case(lens, Hq=8, Hkv=2, W=W, S=S, bs=32 if B == 3 else 16, seed=B).upload()
    c.check(c.run(), rows=set(range(0, B, max(1, B // 40))))


def test_a_window_past_the_sequence_is_plain_decode():
    c = Case([5, 100, 700, 33], W=5000, S=2).upload()
    out = c.run()
    c.check(out)
    plain = torch.empty_like(out)
    with pa.Plan() as plan:
        pa.pa_decode(c.d["q"], c.d["k"], c.d["v"], c.d["table"], c.d["lens"], c.scale, plain, 700, plan)
        assert pa.pa_last_device_error(plan) == 0
    c.compare(plain)


def test_large_scores_stay_finite():
    c = Case([50, 400, 90], W=60, S=3, k_scale=60.0).upload()
    c.check(c.run())
    p = Case([50, 400, 90], [3, 40, 90], W=60, S=3, k_scale=60.0).upload()
    p.check(p.run(prefill=True), prefill=True)


@pytest.mark.parametrize("prefill", [False, True])
@pytest.mark.parametrize("where", ["k", "v"])
def test_visible_values_that_are_not_numbers_show(prefill, where):
    # A key or value that is NaN and visible is the caller's data: its rows are
    # NaN, others are not touched.
    c = Case([300, 400, 90], [1, 1, 1] if prefill else None, Hq=8, Hkv=2, W=60, S=3, seed=2)
    getattr(c, where)[int(c.table[1, 390 // 16]), 1, 390 % 16] = float("nan")
    c.upload()
    out = c.run(prefill=prefill)
    assert pa.pa_last_device_error(c.plan) == 0
    assert bool(torch.isnan(out[1, 4:]).all())
    assert bool(torch.isfinite(out[1, :4]).all()) and bool(torch.isfinite(out[[0, 2]]).all())


def test_decode_wrong_lengths_and_entries():
    c = Case([40, 100, 60, 80], W=20, S=4).upload()
    good = c.run()
    c.check(good)
    c.d["lens"].copy_(torch.tensor([0, 100, 2000, 80], dtype=torch.int32))
    out = c.run(max_len=100)
    assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_SEQ_LEN
    assert bool((out[[0, 2]] == 0).all()) and torch.equal(out[[1, 3]], good[[1, 3]])
    c.upload()
    c.d["table"][1, 6] = c.NB          # the window of the second: tokens 80 .. 99 in pages 5, 6
    c.d["table"][3, 0] = -1            # the sinks of the last
    out = c.run()
    assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_TABLE
    assert bool((out[[1, 3]] == 0).all()) and torch.equal(out[[0, 2]], good[[0, 2]])


def test_a_wrong_entry_anywhere_zeroes_its_rows():
    c = Case([900, 900, 40], Hq=8, Hkv=4, W=800, S=4, seed=5).upload()
    good = c.run()
    c.check(good)
    for page in (0, 7, 30, 56):
        c.upload()
        c.d["table"][1, page] = -3
        out = c.run()
        assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_TABLE
        assert bool((out[1] == 0).all()) and torch.equal(out[[0, 2]], good[[0, 2]])


def test_rows_behind_are_left_alone():
    c = Case([70, 9, 200], W=30, S=2).upload()
    big = torch.full((5, 8, 128), 7.5, dtype=torch.bfloat16, device="cuda")
    c.run(out=big[1:4])
    torch.cuda.synchronize()
    assert bool((big[0] == 7.5).all()) and bool((big[4] == 7.5).all())
    c.check(big[1:4])


def test_forced_paths_and_merges_do_not_apply():
    c = Case([70, 9], W=30, S=2).upload()
    c.run()
    c.plan.set_merge(pa.PA_MERGE_FUSED)
    c.plan.set_path(pa.PA_PATH_SIMPLE)
    c.check(c.run())


@pytest.mark.parametrize("lens,Hq,Hkv,W,bs", [
    ([40000], 8, 1, 33000, 16), ([21000, 40000], 4, 1, 20000, 32), ([30000], 12, 1, 29000, 16), ([30000], 34, 2, 29000, 16),
])
def test_decode_of_few_long_segments(lens, Hq, Hkv, W, bs):
    c = Case(lens, Hq=Hq, Hkv=Hkv, W=W, S=19, bs=bs, seed=Hq).upload()
    c.check(c.run())


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 16), (128, 32)])
@pytest.mark.parametrize("Hq,Hkv", [(4, 1), (16, 1), (8, 4), (32, 32)])
@pytest.mark.parametrize("B", [1, 2, 5, 9, 17, 40, 130])
def test_decode_cluster_shapes(B, Hq, Hkv, D, bs):
    # From one segment to more than the device holds blocks at a time: every
    # cluster size and number of warps, with sequences that leave some blocks of
    # a cluster, and some warps of a block, without a chunk.
    rng = np.random.default_rng(B + Hq)
    lens = rng.integers(1, 900, size=B).tolist()
    c = Case(lens, Hq=Hq, Hkv=Hkv, D=D, bs=bs, W=600, S=7, seed=B).upload()
    c.check(c.run(), rows=set(range(0, B, max(1, B // 12))))


KERNELS = [pa.PA_PREFILL_AUTO, pa.PA_PREFILL_ONE_TILE, pa.PA_PREFILL_TWO_TILE]


@pytest.fixture(params=KERNELS, ids=["auto", "one_tile", "two_tile"])
def kernel(request):
    pa.pa_debug_set_prefill_kernel(request.param)
    try:
        yield request.param
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)


@pytest.mark.parametrize("W,S", [(1, 0), (20, 4), (16, 16), (33, 40), (100, 0), (130, 129), (128, 128), (300, 17),
                                 (5, 400), (2000, 3)])
@pytest.mark.parametrize("bs", [16, 32])
def test_prefill_edges(W, S, bs, kernel):
    lens = [1, 17, 40, 64, 129, 200, 300, 333, 500]
    ns = [1, 17, 3, 64, 100, 1, 0, 65, 33]
    c = Case(lens, ns, W=W, S=S, bs=bs, seed=W).upload()
    c.check(c.run(prefill=True), prefill=True)


@pytest.mark.parametrize("Hq,Hkv,lens,ns", [
    (8, 8, [300, 700], [300, 150]), (2, 1, [200], [130]), (16, 1, [400, 90], [60, 20]), (32, 4, [350], [40]),
    (64, 2, [260, 20], [9, 20]), (128, 1, [150, 33], [5, 1]),
])
def test_prefill_head_groups(Hq, Hkv, lens, ns, kernel):
    c = Case(lens, ns, Hq=Hq, Hkv=Hkv, W=90, S=6, seed=Hq).upload()
    c.check(c.run(prefill=True), prefill=True, rows=set(range(0, c.T, 1 + c.T // 60)) | {c.T - 1})


@pytest.mark.parametrize("lens,ns,W,S", [
    ([5000], [5000], 700, 4), ([6000], [7], 4096, 5), ([9000, 200], [6, 6], 3000, 64), ([3000] * 3, [1, 2, 4], 2500, 0),
    ([2000] * 30, [5] * 30, 300, 4), ([1500] * 20, [256] * 20, 300, 20),
])
def test_prefill_sizes(lens, ns, W, S):
    c = Case(lens, ns, Hq=8, Hkv=2, W=W, S=S, seed=len(lens)).upload()
    out = c.run(prefill=True)
    c.check(out, prefill=True, rows=set(range(0, c.T, 1 + c.T // 50)) | {c.T - 1})
    assert bool(torch.isfinite(out).all())


@pytest.mark.parametrize("Hq,Hkv,lens,ns,W,S", [
    (8, 2, [5000], [64], 4096, 5),                    # four parts of nine chunks and less
    (8, 2, [6000], [40], 4090, 64),
    (8, 2, [4500, 1500, 30], [40, 64, 17], 4096, 600),  # parts, two of eight chunks and four, and none
    (4, 4, [6000, 400], [256, 100], 4000, 0),         # rows that see nothing of the last part
    (8, 1, [9000], [128], 6000, 2000),
    (8, 2, [4300] * 80, [50] * 80, 4096, 4),          # a complete turn of the blocks before
])
@pytest.mark.parametrize("bs", [16, 32])
def test_prefill_items_in_parts(Hq, Hkv, lens, ns, W, S, bs):
    c = Case(lens, ns, Hq=Hq, Hkv=Hkv, W=W, S=S, bs=bs, seed=W).upload()
    pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_TWO_TILE)
    try:
        out = c.run(prefill=True)
        again = [c.run(prefill=True) for _ in range(3)]
        f32 = c.run(prefill=True, out_dtype=torch.float32)
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)
    rows = set(range(0, c.T, 1 + c.T // 60)) | {c.T - 1}
    c.check(out, prefill=True, rows=rows)
    c.check(f32, prefill=True, rows=rows)
    assert bool(torch.isfinite(out).all())
    for x in again:                  # the parts are merged in one order
        assert torch.equal(out, x)


def test_prefill_parts_show_nan_of_a_visible_key():
    c = Case([5000], [40], W=4500, S=4, seed=3)
    last = 4999                      # only the last query sees it, in the last part
    c.k[int(c.table[0, last // c.bs]), :, last % c.bs] = float("nan")
    c.upload()
    pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_TWO_TILE)
    try:
        out = c.run(prefill=True)
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)
    assert bool(torch.isnan(out[-1]).all())
    c.check(out, prefill=True, rows=set(range(39)))


def test_prefill_of_single_queries_is_the_decode():
    c = Case([1, 40, 300, 1000], W=64, S=4).upload()
    c.check(c.run(prefill=True), prefill=True)
    c.check(c.run())


def test_prefill_wrong_lengths_and_entries(kernel):
    c = Case([300, 200, 400], [40, 50, 70], W=64, S=4).upload()
    good = c.run(prefill=True)
    c.check(good, prefill=True)
    c.d["lens"].copy_(torch.tensor([39, 200, 4000], dtype=torch.int32))
    out = c.run(prefill=True, max_len=400)
    assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_SEQ_LEN
    assert bool((out[:40] == 0).all()) and bool((out[90:] == 0).all()) and torch.equal(out[40:90], good[40:90])
    c.upload()
    c.d["table"][1, 0] = c.NB + 7
    out = c.run(prefill=True)
    assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_TABLE
    assert bool((out[40:90] == 0).all()) and torch.equal(out[:40], good[:40]) and torch.equal(out[90:], good[90:])


def test_prefill_rows_behind_are_left_alone(kernel):
    c = Case([300, 90], [70, 33], W=64, S=4).upload()
    big = torch.full((c.T + 2, 8, 128), 7.5, dtype=torch.bfloat16, device="cuda")
    c.run(prefill=True, out=big[1:-1])
    torch.cuda.synchronize()
    assert bool((big[0] == 7.5).all()) and bool((big[-1] == 7.5).all())
    c.check(big[1:-1], prefill=True)


@pytest.mark.parametrize("prefill", [False, True])
def test_graph_replay_outlives_a_growing_plan(prefill):
    ns = [6, 6] if prefill else None
    c = Case([3000, 2000], ns, W=1000, S=4, seed=1).upload()
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    c.run(prefill=prefill, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(prefill=prefill, out=out)
    # A larger call on the same plan, then the graph with other values.
    big = Case([9000] * 3, [9] * 3 if prefill else None, Hq=64, Hkv=4, W=8000, S=4, seed=2)
    big.plan = c.plan
    big.upload()
    big.check(big.run(prefill=prefill), prefill, rows={0})
    other = Case([3000, 2000], ns, W=1000, S=4, seed=3)
    for name in ("q", "k", "v"):
        c.d[name].copy_(getattr(other, name))
    c.d["table"].copy_(torch.from_numpy(other.table))
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    other.plan = c.plan
    other.check(out, prefill)


def test_graph_replay_outlives_plain_calls_that_outgrow_the_plan():
    c = Case([3000, 2000], [6, 6], W=1000, S=4, seed=1).upload()
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    c.run(prefill=True, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.run(prefill=True, out=out)
    big = Case([2500] * 40, Hq=32, Hkv=8, W=5000, S=0, seed=2).upload()
    res = torch.empty_like(big.d["q"])
    pa.pa_decode(big.d["q"], big.d["k"], big.d["v"], big.d["table"], big.d["lens"], big.scale, res, 2500, c.plan)
    torch.cuda.synchronize()
    out.zero_()
    g.replay()
    torch.cuda.synchronize()
    c.check(out, True)


@pytest.mark.parametrize("prefill", [False, True])
def test_a_capture_cannot_grow_a_plan(prefill):
    c = Case([3000, 2000], [6, 6] if prefill else None, W=1000, S=4).upload()
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        with pytest.raises(pa.PagedAttentionError) as e:
            c.run(prefill=prefill, out=out)
        assert e.value.status == pa.PA_ERR_WORKSPACE
        out.add_(1.0)                 # the capture goes on
    g.replay()
    torch.cuda.synchronize()
    assert bool((out == 1.0).all())
    c.check(c.run(prefill=prefill), prefill)


@pytest.mark.parametrize("prefill", [False, True])
def test_side_stream_and_same_bits(prefill):
    c = Case([3000, 40, 900], [5, 40, 200] if prefill else None, W=500, S=4).upload()
    a = c.run(prefill=prefill)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    b = c.run(prefill=prefill, stream=side)
    side.synchronize()
    if prefill:      # the decode's dynamic tail may split its sums elsewhere
        assert torch.equal(a, b)
    c.check(b, prefill)


@pytest.mark.parametrize("prefill", [False, True])
def test_expired_waits_are_reported_and_the_next_call_is_right(prefill):
    c = Case([700, 90], [40, 20] if prefill else None, W=200, S=4).upload()
    pa.pa_debug_set_wait_probe(True)
    try:
        c.run(prefill=prefill)
        assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_TIMEOUT
    finally:
        pa.pa_debug_set_wait_probe(False)
    c.check(c.run(prefill=prefill), prefill)


# The persistent kernel, whole items and items in parts.
PERSISTENT = [dict(lens=[700, 90], ns=[70, 20], W=200, S=4), dict(lens=[5000], ns=[40], W=4500, S=4)]


@pytest.mark.parametrize("kw", PERSISTENT)
def test_expired_waits_of_the_persistent_kernel(kw):
    c = Case(**kw).upload()
    pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_TWO_TILE)
    try:
        c.run(prefill=True)
        torch.cuda.synchronize()
        pa.pa_debug_set_wait_probe(True)
        try:
            c.run(prefill=True)
            assert pa.pa_last_device_error(c.plan) == pa.PA_DEVERR_TIMEOUT
        finally:
            pa.pa_debug_set_wait_probe(False)
        for _ in range(2):
            c.check(c.run(prefill=True), prefill=True)
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)


@pytest.mark.parametrize("kw", PERSISTENT)
def test_graph_of_the_persistent_kernel(kw):
    c = Case(seed=1, **kw).upload()
    out = torch.zeros(c.q.shape, dtype=torch.bfloat16, device="cuda")
    pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_TWO_TILE)
    try:
        c.run(prefill=True, out=out)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(prefill=True, out=out)
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)
    for seed in (2, 3):
        other = Case(seed=seed, **kw)
        for name in ("q", "k", "v"):
            c.d[name].copy_(getattr(other, name))
        c.d["table"].copy_(torch.from_numpy(other.table))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        other.plan = c.plan
        other.check(out, prefill=True)


def test_binding_refuses_shapes_and_types():
    c = Case([70, 9], W=30, S=2).upload()
    for name, t, e in (("lens", c.d["lens"][:1], ValueError), ("lens", c.d["lens"].long(), TypeError),
                       ("table", c.d["table"][:1], ValueError), ("k", c.d["k"].float(), TypeError),
                       ("q", c.d["q"].float(), TypeError)):
        keep, c.d[name] = c.d[name], t
        with pytest.raises(e):
            c.run()
        c.d[name] = keep
    c.W = 0
    with pytest.raises(pa.PagedAttentionError):
        c.run()
    c.W, c.S = 4, -1
    with pytest.raises(pa.PagedAttentionError):
        c.run()
    torch.cuda.synchronize()
