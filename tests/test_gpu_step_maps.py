"""GPU: block tables and slot maps of a step against a token-by-token reference
in whole numbers: idle requests, empty caches, padded rows, one request and the
largest batch, chained and captured steps, lengths and tables that are wrong,
and a free list that is too short. Results are whole numbers: compared exactly."""

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from step_reference import step_maps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


I32 = torch.int32
NAMES = ("seq_lens", "q_start", "positions", "slots", "block_tables", "free_left")


class Step:
    def __init__(self, cache, new, bs=16, MB=None, spare=3, pad=0, seed=0, T=None, free=None, limit=None):
        rng = np.random.default_rng(seed)
        cache, new = np.asarray(cache, dtype=np.int32), np.asarray(new, dtype=np.int32)
        self.B, self.bs = len(cache), bs
        had = -(-np.clip(cache, 0, None) // bs)
        most = int((-(-np.clip(cache.astype(np.int64) + new, 0, 1 << 20) // bs)).max(initial=0))
        self.MB = MB or most + 1
        fresh = int(np.clip(-(-(cache.astype(np.int64) + new) // bs) - had, 0, 1 << 20).sum())
        self.NB = int(np.minimum(had, self.MB).sum()) + min(fresh, 1 << 20) + spare
        ids = rng.permutation(self.NB).astype(np.int32)
        table = np.full((self.B, self.MB), -7, dtype=np.int32)
        at = 0
        for b in range(self.B):
            h = min(int(had[b]), self.MB)
            table[b, :h] = ids[at:at + h]
            at += h
        self.free = ids[at:] if free is None else np.asarray(free, dtype=np.int32)
        self.cache, self.new, self.table = cache, new, table
        self.T = int(np.clip(new, 0, None).sum()) + pad if T is None else T
        self.limit = limit or self.MB * bs

    def upload(self):
        d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
        self.d = dict(cache=d(self.cache), new=d(self.new), free=d(self.free),
                      count=torch.tensor([len(self.free)], dtype=I32, device="cuda"),
                      table=d(self.table))
        f = lambda n, dt=I32: torch.full((n,), -77, dtype=dt, device="cuda")  # noqa: E731
        self.o = dict(seq=f(self.B), start=f(self.B + 1), pos=f(self.T), slots=f(self.T, torch.int64),
                      left=f(1), err=torch.zeros(1, dtype=I32, device="cuda"))
        return self

    def call(self, stream=None):
        d, o = self.d, self.o
        pa.pa_step_maps(d["cache"], d["new"], d["free"], d["count"], d["table"], self.bs, self.NB,
                        self.limit, o["seq"], o["start"], o["pos"], o["slots"], o["left"],
                        device_error=o["err"], stream=stream)

    def results(self):
        torch.cuda.synchronize()
        o = self.o
        return [x.cpu().numpy() for x in (o["seq"], o["start"], o["pos"], o["slots"], self.d["table"])] + \
            [int(o["left"])], int(o["err"])

    def expect(self, count=None):
        r = step_maps(self.cache, self.new, self.free, len(self.free) if count is None else count,
                      self.table, self.bs, self.NB, self.limit, self.T)
        return list(r[:6]), r[6]


def check(s, count=None):
    got, err = s.results()
    want, want_err = s.expect(count)
    for name, g, w in zip(NAMES, got, want):
        np.testing.assert_array_equal(g, w, err_msg=name)
    assert err == want_err
    return err


def lens(seed, B, hi_cache, hi_new, idle=0.0):
    rng = np.random.default_rng(seed)
    new = rng.integers(1, hi_new + 1, size=B)
    new[rng.random(B) < idle] = 0
    return rng.integers(0, hi_cache + 1, size=B), new


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("cache,new,pad", [
    ([0], [1], 0),                               # the first token of the only request
    ([15], [1], 0), ([16], [1], 0), ([31], [2], 0), ([32], [33], 5),
    ([0, 0, 0], [0, 0, 0], 0),                   # nothing at all
    ([0, 0, 0], [0, 0, 0], 4),                   # padding only
    ([5, 0, 100, 16], [0, 7, 1, 16], 3),
    ([0] * 40, list(range(40)), 1),
    lens(1, 64, 2000, 1) + (0,), lens(2, 33, 500, 300, 0.3) + (64,),
    lens(3, 513, 100, 40, 0.1) + (0,), lens(4, 8192, 40, 3, 0.5) + (1000,),
    lens(5, 1, 10000, 100000) + (7,),
])
def test_step_maps(bs, cache, new, pad):
    s = Step(cache, new, bs=bs, pad=pad, seed=len(cache)).upload()
    s.call()
    assert check(s) == 0


@pytest.mark.parametrize("pad", [0, 5, 700])
def test_no_requests_leave_padding(pad):
    s = Step([], [], bs=16, pad=pad).upload()
    for name in ("start", "pos", "slots", "left"):
        s.o[name].fill_(9)               # a step before
    s.call()
    assert check(s) == 0


def test_chained_steps_walk_the_free_list():
    # Two buffers of the free count in turn; each step's cached lengths are the
    # lengths of the one before.
    rng = np.random.default_rng(8)
    B, bs, MB, NB = 9, 16, 40, 500
    free = rng.permutation(NB).astype(np.int32)
    table = np.full((B, MB), -1, dtype=np.int32)
    cache = np.zeros(B, dtype=np.int32)
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    dt, df = d(table), d(free)
    counts = [torch.tensor([NB], dtype=I32, device="cuda"), torch.zeros(1, dtype=I32, device="cuda")]
    seqs = [d(cache), torch.zeros(B, dtype=I32, device="cuda")]
    count = NB
    for i in range(6):
        new = rng.integers(0, 60, size=B).astype(np.int32)
        T = int(new.sum())
        start, pos = torch.zeros(B + 1, dtype=I32, device="cuda"), torch.zeros(T, dtype=I32, device="cuda")
        slots = torch.zeros(T, dtype=torch.int64, device="cuda")
        pa.pa_step_maps(seqs[i % 2], d(new), df, counts[i % 2], dt, bs, NB, MB * bs, seqs[1 - i % 2],
                        start, pos, slots, counts[1 - i % 2])
        want = step_maps(cache, new, free, count, table, bs, NB, MB * bs, T)
        cache, table, count = want[0], want[4], want[5]
        np.testing.assert_array_equal(slots.cpu().numpy(), want[3])
        np.testing.assert_array_equal(dt.cpu().numpy(), table)
        np.testing.assert_array_equal(seqs[1 - i % 2].cpu().numpy(), cache)
        assert int(counts[1 - i % 2]) == count
    assert pa.pa_last_device_error(None) == 0
    used = table[table >= 0]
    assert len(set(used.tolist())) == len(used) == NB - count


@pytest.mark.parametrize("name,kw,bits", [
    ("negative cached length", dict(cache=[5, -1, 7], new=[1, 1, 1]), pa.PA_DEVERR_SEQ_LEN),
    ("negative new tokens", dict(cache=[5, 6, 7], new=[1, -4, 20], T=21), pa.PA_DEVERR_SEQ_LEN),
    ("past the table", dict(cache=[5, 60, 7], new=[1, 5, 1], MB=4), pa.PA_DEVERR_SEQ_LEN),
    ("past the limit", dict(cache=[5, 60, 7], new=[1, 5, 1], limit=50), pa.PA_DEVERR_SEQ_LEN),
    ("sum past 32 bits", dict(cache=[2 ** 31 - 1, 3], new=[2 ** 31 - 1, 2], MB=4, T=9), pa.PA_DEVERR_SEQ_LEN),
    ("rows past num_rows", dict(cache=[5, 0, 7, 8], new=[3, 40, 2, 0], T=20), pa.PA_DEVERR_SEQ_LEN),
    ("no row at all", dict(cache=[5, 0], new=[3, 4], T=0), pa.PA_DEVERR_SEQ_LEN),
    ("too few free blocks", dict(cache=[5, 16, 20], new=[1, 1, 40], free=[3, 4]), pa.PA_DEVERR_NO_BLOCKS),
    ("no free block", dict(cache=[0, 3], new=[1, 1], free=[]), pa.PA_DEVERR_NO_BLOCKS),
    ("a free block outside the pool", dict(cache=[0, 0], new=[20, 1], free=[0, 9999, -3]), pa.PA_DEVERR_TABLE),
])
def test_wrong_data_is_reported_and_contained(name, kw, bits):
    s = Step(**kw).upload()
    s.call()
    assert check(s) == bits, name


@pytest.mark.parametrize("count", [-1, 6, 2 ** 31 - 1])
def test_a_wrong_free_count_takes_no_block(count):
    s = Step([15, 16], [1, 1], free=[1, 2, 3, 4, 5]).upload()
    s.d["count"].fill_(count)
    s.call()
    assert check(s, count) == pa.PA_DEVERR_TABLE | pa.PA_DEVERR_NO_BLOCKS


def test_a_wrong_table_entry_gives_no_slot():
    s = Step([20, 20], [3, 13])
    s.table[0, 1], s.table[1, 0] = s.NB, 12345678   # the second is not read: its rows lie behind
    s.upload().call()
    assert check(s) == pa.PA_DEVERR_TABLE


def test_nothing_else_is_written():
    s = Step(*lens(6, 50, 300, 40, 0.2), pad=13).upload()
    guard = {}
    for name, t in list(s.o.items()):
        big = torch.full((t.numel() + 64,), -99, dtype=t.dtype, device="cuda")
        big[32:32 + t.numel()] = t
        guard[name], s.o[name] = big, big[32:32 + t.numel()]
    s.call()
    check(s)
    for name, big in guard.items():
        assert bool((big[:32] == -99).all()) and bool((big[-32:] == -99).all()), name


def test_side_stream_and_graph_replay():
    s = Step(*lens(7, 40, 300, 30, 0.1), pad=9).upload()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    s.call(stream=side)
    assert check(s) == 0
    s = Step(*lens(7, 40, 300, 30, 0.1), pad=9).upload()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        s.call()
    # New lengths through the same captured step.
    other = Step(*lens(9, 40, 300, 30, 0.1), MB=s.MB, T=s.T, seed=40)
    for k, v in (("cache", other.cache), ("new", other.new), ("table", other.table)):
        s.d[k].copy_(torch.from_numpy(v))
    s.cache, s.new, s.table = other.cache, other.new, other.table
    g.replay()
    got, err = s.results()
    want, want_err = s.expect()
    for name, x, w in zip(NAMES, got, want):
        np.testing.assert_array_equal(x, w, err_msg=name)
    assert err == want_err


def test_binding_refuses_shapes_and_types():
    s = Step([3, 4], [1, 1]).upload()
    d, o = s.d, s.o

    def call(**kw):
        a = dict(cache=d["cache"], new=d["new"], seq=o["seq"], start=o["start"], pos=o["pos"],
                 slots=o["slots"], left=o["left"], table=d["table"])
        a.update(kw)
        pa.pa_step_maps(a["cache"], a["new"], d["free"], d["count"], a["table"], 16, s.NB, s.limit,
                        a["seq"], a["start"], a["pos"], a["slots"], a["left"])

    for kw in (dict(new=d["new"][:1]), dict(start=o["seq"]), dict(pos=o["pos"][:1]),
               dict(table=d["table"][:1]), dict(cache=torch.zeros(2, 2, dtype=I32, device="cuda")[:, 0])):
        with pytest.raises(ValueError):
            call(**kw)
    for kw in (dict(slots=o["pos"]), dict(cache=d["cache"].long()), dict(left=o["left"].float())):
        with pytest.raises(TypeError):
            call(**kw)
    with pytest.raises(pa.PagedAttentionError):
        call(seq=d["cache"])
    torch.cuda.synchronize()
