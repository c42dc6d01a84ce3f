"""Windowed attention on the host (no GPU): the calls refuse bad arguments
before any CUDA call and create no plan; empty calls are no-ops. The visible
pages and masks of a window, as the kernels number them, are checked against
the definition for every small case."""

import ctypes

import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from paged_kv_cache_202_gb300 import _build
from window_reference import tokens_seen


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return pa.lib()


A = 0x10000  # a fake, 16-byte aligned device address: never dereferenced


def _call(lib, prefill, **kw):
    a = dict(q=A, qs=A, T=8, maxq=4, k=A, v=A, bt=A, mb=4, sl=A, B=2, Hq=8, Hkv=2, D=128, bs=16, NB=64,
             maxlen=64, scale=0.1, window=20, sinks=4, kvdt=pa.PA_BF16, out=A, odt=pa.PA_BF16, plan=True)
    a.update(kw)
    plan = ctypes.c_void_p(None)
    pp = ctypes.byref(plan) if a["plan"] else None
    tail = (a["k"], a["v"], a["bt"], a["mb"], a["sl"], a["B"], a["Hq"], a["Hkv"], a["D"], a["bs"], a["NB"],
            a["maxlen"], a["scale"], a["window"], a["sinks"], a["kvdt"], a["out"], a["odt"], pp, None)
    st = (lib.pa_prefill_window(a["q"], a["qs"], a["T"], a["maxq"], *tail) if prefill
          else lib.pa_decode_window(a["q"], *tail))
    assert plan.value is None, "an argument error must not create a plan"
    return st


SHARED = [
    (dict(q=None), pa.PA_ERR_NULL), (dict(k=None), pa.PA_ERR_NULL), (dict(v=None), pa.PA_ERR_NULL),
    (dict(bt=None), pa.PA_ERR_NULL), (dict(sl=None), pa.PA_ERR_NULL), (dict(out=None), pa.PA_ERR_NULL),
    (dict(plan=False), pa.PA_ERR_NULL),
    (dict(window=0), pa.PA_ERR_SHAPE), (dict(window=-1), pa.PA_ERR_SHAPE),
    (dict(sinks=-1), pa.PA_ERR_SHAPE),
    (dict(kvdt=pa.PA_F32), pa.PA_ERR_DTYPE),
    (dict(odt=7), pa.PA_ERR_DTYPE),
    (dict(bs=8), pa.PA_ERR_BLOCK_SIZE),
    (dict(B=-1), pa.PA_ERR_SHAPE), (dict(B=8193), pa.PA_ERR_SHAPE),
    (dict(Hq=6, Hkv=4), pa.PA_ERR_SHAPE), (dict(D=96), pa.PA_ERR_SHAPE),
    (dict(mb=0), pa.PA_ERR_SHAPE), (dict(maxlen=0), pa.PA_ERR_SHAPE), (dict(NB=0), pa.PA_ERR_SHAPE),
    (dict(scale=float("nan")), pa.PA_ERR_SHAPE), (dict(scale=float("inf")), pa.PA_ERR_SHAPE),
    (dict(q=A + 8), pa.PA_ERR_ALIGN), (dict(k=A + 2), pa.PA_ERR_ALIGN), (dict(out=A + 4), pa.PA_ERR_ALIGN),
]


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(B=8192, Hq=64, Hkv=64, mb=65536, maxlen=1 << 20, window=1 << 20), pa.PA_ERR_SHAPE),
])
def test_decode_window_refuses_bad_arguments(lib, kw, status):
    assert _call(lib, False, **kw) == status


@pytest.mark.parametrize("kw,status", SHARED + [
    (dict(qs=None), pa.PA_ERR_NULL),
    (dict(D=64), pa.PA_ERR_SHAPE),
    (dict(Hq=24, Hkv=8), pa.PA_ERR_SHAPE),
    (dict(Hq=256, Hkv=1), pa.PA_ERR_SHAPE),
    (dict(mb=16385), pa.PA_ERR_SHAPE),
    (dict(maxq=0), pa.PA_ERR_SHAPE), (dict(T=-1), pa.PA_ERR_SHAPE),
    (dict(scale=0.0), pa.PA_ERR_SHAPE), (dict(scale=-0.1), pa.PA_ERR_SHAPE),
    (dict(Hq=70000, Hkv=70000), pa.PA_ERR_SHAPE),
])
def test_prefill_window_refuses_bad_arguments(lib, kw, status):
    assert _call(lib, True, **kw) == status


def test_empty_calls_are_no_ops(lib):
    assert _call(lib, False, B=0) == pa.PA_OK
    assert _call(lib, True, B=0) == pa.PA_OK
    assert _call(lib, True, T=0) == pa.PA_OK


def test_binding_refuses_host_tensors():
    q = torch.zeros(2, 8, 128, dtype=torch.bfloat16)
    pool = torch.zeros(4, 2, 16, 128, dtype=torch.bfloat16)
    bt, sl = torch.zeros(2, 4, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    qs = torch.arange(3, dtype=torch.int32)
    plan = pa.Plan()
    with pytest.raises(ValueError, match="CUDA device"):
        pa.pa_decode_window(q, pool, pool, bt, sl, 0.1, 8, 2, q, 64, plan)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.pa_prefill_window(q, qs, pool, pool, bt, sl, 0.1, 8, 2, q, 1, 64, plan)
    assert plan.handle.value is None


def _view(first, last, W, S, bs):
    """The kernels' numbering of the visible pages, in whole numbers."""
    w0 = first - W + 1 if first >= W else 0
    skip = max(0, w0 // bs - -(-S // bs))
    return skip, last + 1 - skip * bs, w0 - skip * bs


@pytest.mark.parametrize("W", [1, 2, 4, 5, 8, 9, 17, 40, 80])
@pytest.mark.parametrize("S", [0, 1, 3, 4, 5, 9, 20, 100])
def test_the_numbering_of_visible_tokens(W, S):
    bs = 4
    for L in list(range(1, 30)) + [63, 64, 65, 90]:
        for n in (1, 2, 7):
            if n > L:
                continue
            first, last = L - n, L - 1
            skip, end, lo = _view(first, last, W, S, bs)
            sp = -(-S // bs)
            token = [v if v < sp * bs else v + skip * bs for v in range(end)]
            for p in range(first, last + 1):
                hi = p - skip * bs
                seen = [t for v, t in enumerate(token) if v <= hi and (v < S or v > hi - W)]
                assert seen == tokens_seen(p, W, S).tolist()
            union = set().union(*(tokens_seen(p, W, S).tolist() for p in range(first, last + 1)))
            # What is zeroed in the values is exactly what no row sees.
            assert [v for v, t in enumerate(token) if t not in union] == list(range(S, min(lo, end)))
            # Nothing outside the sequence is looked up, and no page twice.
            pages = [p if p < sp else p + skip for p in range(-(-end // bs))]
            assert len(set(pages)) == len(pages) and max(pages) == last // bs
            if n == 1:
                assert end <= W + S + 2 * bs
                assert set(pages) == {t // bs for t in union}
