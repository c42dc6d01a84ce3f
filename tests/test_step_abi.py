"""Step preparation on the host (no GPU): the calls refuse bad arguments before
any CUDA call, the scaled frequencies follow their definitions, and a rotation
holds the exact fraction of a turn of every pair."""

import ctypes
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from paged_kv_cache_202_gb300 import _build
from step_reference import inv_freq


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return pa.lib()


A = 0x10000  # a fake, 16-byte aligned device address: never dereferenced


def _step(lib, **kw):
    a = dict(cl=A, nl=A + 0x100, B=4, fb=A, nf=8, fc=A + 0x200, bt=A + 0x1000, mb=8, bs=16, NB=64,
             maxlen=128, sl=A + 0x300, qs=A + 0x400, pos=A + 0x500, slots=A + 0x600, T=8,
             left=A + 0x700)
    a.update(kw)
    return lib.pa_step_maps(a["cl"], a["nl"], a["B"], a["fb"], a["nf"], a["fc"], a["bt"], a["mb"],
                            a["bs"], a["NB"], a["maxlen"], a["sl"], a["qs"], a["pos"], a["slots"],
                            a["T"], a["left"], None, None)


@pytest.mark.parametrize("kw,status", [
    (dict(cl=None), pa.PA_ERR_NULL),
    (dict(nl=None), pa.PA_ERR_NULL),
    (dict(fb=None), pa.PA_ERR_NULL),
    (dict(fc=None), pa.PA_ERR_NULL),
    (dict(bt=None), pa.PA_ERR_NULL),
    (dict(sl=None), pa.PA_ERR_NULL),
    (dict(qs=None), pa.PA_ERR_NULL),
    (dict(pos=None), pa.PA_ERR_NULL),
    (dict(slots=None), pa.PA_ERR_NULL),
    (dict(left=None), pa.PA_ERR_NULL),
    (dict(bs=8), pa.PA_ERR_BLOCK_SIZE),
    (dict(B=-1), pa.PA_ERR_SHAPE),
    (dict(B=8193), pa.PA_ERR_SHAPE),
    (dict(mb=0), pa.PA_ERR_SHAPE),
    (dict(mb=1 << 28), pa.PA_ERR_SHAPE),        # table positions past 32 bits
    (dict(NB=0), pa.PA_ERR_SHAPE),
    (dict(maxlen=0), pa.PA_ERR_SHAPE),
    (dict(nf=-1), pa.PA_ERR_SHAPE),
    (dict(T=-1), pa.PA_ERR_SHAPE),
    (dict(sl=A), pa.PA_ERR_SHAPE),              # outputs over the inputs they are made from
    (dict(sl=A + 0x104), pa.PA_ERR_SHAPE),
    (dict(qs=A + 12), pa.PA_ERR_SHAPE),
    (dict(qs=A + 0x100 - 16), pa.PA_ERR_SHAPE),  # q_start has B + 1 entries
    (dict(left=A + 0x200), pa.PA_ERR_SHAPE),
    (dict(slots=A + 0x604), pa.PA_ERR_ALIGN),
    (dict(pos=A + 0x502), pa.PA_ERR_ALIGN),
    (dict(cl=A + 1), pa.PA_ERR_ALIGN),
])
def test_step_maps_refuses_bad_arguments(lib, kw, status):
    assert _step(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(qs=None), pa.PA_ERR_NULL),
    (dict(slots=None), pa.PA_ERR_NULL),
    (dict(left=A + 0x200), pa.PA_ERR_SHAPE),
    (dict(slots=A + 0x604), pa.PA_ERR_ALIGN),
])
def test_step_maps_of_no_requests_refuses_bad_arguments(lib, kw, status):
    a = dict(B=0, cl=None, nl=None, bt=None, sl=None)
    a.update(kw)
    assert _step(lib, **a) == status


def _spec(**kw):
    s = pa.Rope(64).struct
    for k, v in kw.items():
        setattr(s, k, v)
    return ctypes.byref(s)


def _rope(lib, append, **kw):
    a = dict(q=A, qs=4096, k=A, ks=1024, v=A, vs=1024, pos=A, slots=A, T=4, Hq=32, Hk=8, D=128,
             dt=pa.PA_BF16, qw=None, kw=None, eps=1e-6, rope=_spec(), qo=A, qos=4096, ko=A,
             kos=1024, kp=A, vp=A, bs=16, NB=4)
    a.update(kw)
    head = (a["q"], a["qs"], a["k"], a["ks"])
    mid = (a["T"], a["Hq"], a["Hk"], a["D"], a["dt"], a["qw"], a["kw"], a["eps"], a["rope"],
           a["qo"], a["qos"])
    if append:
        return lib.pa_qk_rope_append(*head, a["v"], a["vs"], a["pos"], a["slots"], *mid, a["kp"],
                                     a["vp"], a["bs"], a["NB"], None, None)
    return lib.pa_qk_rope(*head, a["pos"], *mid, a["ko"], a["kos"], None)


_SHARED = [
    (dict(q=None), pa.PA_ERR_NULL),
    (dict(k=None), pa.PA_ERR_NULL),
    (dict(pos=None), pa.PA_ERR_NULL),
    (dict(qo=None), pa.PA_ERR_NULL),
    (dict(dt=2), pa.PA_ERR_DTYPE),
    (dict(T=-1), pa.PA_ERR_SHAPE),
    (dict(D=96), pa.PA_ERR_SHAPE),
    (dict(Hq=0), pa.PA_ERR_SHAPE),
    (dict(Hk=0), pa.PA_ERR_SHAPE),
    (dict(Hq=1 << 20), pa.PA_ERR_SHAPE),
    (dict(qs=4095), pa.PA_ERR_SHAPE),            # less than a row
    (dict(qs=4100), pa.PA_ERR_SHAPE),            # not whole 16-byte units
    (dict(ks=1000), pa.PA_ERR_SHAPE),
    (dict(qos=100), pa.PA_ERR_SHAPE),
    (dict(eps=-1.0), pa.PA_ERR_SHAPE),
    (dict(eps=math.nan), pa.PA_ERR_SHAPE),
    (dict(D=64, qs=2048, ks=512, rope="128"), pa.PA_ERR_SHAPE),   # more rotated than there is
    (dict(rope="layout"), pa.PA_ERR_SHAPE),
    (dict(rope="rot"), pa.PA_ERR_SHAPE),
    (dict(rope="amp"), pa.PA_ERR_SHAPE),
    (dict(q=A + 8), pa.PA_ERR_ALIGN),
    (dict(k=A + 2), pa.PA_ERR_ALIGN),
    (dict(qo=A + 4), pa.PA_ERR_ALIGN),
    (dict(qw=A + 4), pa.PA_ERR_ALIGN),
    (dict(kw=A + 8), pa.PA_ERR_ALIGN),
    (dict(pos=A + 2), pa.PA_ERR_ALIGN),
]
_SPECS = {"128": dict(rot_dim=128), "layout": dict(layout=2), "rot": dict(rot_dim=24),
          "amp": dict(amplitude=math.inf)}


def _with_spec(kw):
    return {**kw, "rope": _spec(**_SPECS[kw["rope"]])} if "rope" in kw else kw


@pytest.mark.parametrize("kw,status", _SHARED + [
    (dict(ko=None), pa.PA_ERR_NULL),
    (dict(kos=8), pa.PA_ERR_SHAPE),
    (dict(ko=A + 8), pa.PA_ERR_ALIGN),
])
def test_qk_rope_refuses_bad_arguments(lib, kw, status):
    assert _rope(lib, False, **_with_spec(kw)) == status


@pytest.mark.parametrize("kw,status", _SHARED + [
    (dict(v=None), pa.PA_ERR_NULL),
    (dict(slots=None), pa.PA_ERR_NULL),
    (dict(kp=None), pa.PA_ERR_NULL),
    (dict(vp=None), pa.PA_ERR_NULL),
    (dict(bs=64), pa.PA_ERR_BLOCK_SIZE),
    (dict(NB=0), pa.PA_ERR_SHAPE),
    (dict(vs=1020), pa.PA_ERR_SHAPE),
    (dict(v=A + 8), pa.PA_ERR_ALIGN),
    (dict(kp=A + 8), pa.PA_ERR_ALIGN),
    (dict(vp=A + 8), pa.PA_ERR_ALIGN),
    (dict(slots=A + 4), pa.PA_ERR_ALIGN),
])
def test_qk_rope_append_refuses_bad_arguments(lib, kw, status):
    assert _rope(lib, True, **_with_spec(kw)) == status


@pytest.mark.parametrize("append", [False, True])
def test_no_rows_are_a_no_op(lib, append):
    assert _rope(lib, append, T=0) == pa.PA_OK


@pytest.mark.parametrize("kw", [
    dict(rot_dim=8), dict(rot_dim=24), dict(rot_dim=144), dict(rot_dim=64, base=1.0),
    dict(rot_dim=64, base=math.inf), dict(rot_dim=64, scaling=4), dict(rot_dim=64, layout=3),
    dict(rot_dim=64, scaling=pa.PA_ROPE_LINEAR, factor=0.5),
    dict(rot_dim=64, scaling=pa.PA_ROPE_PARTS, factor=2.0, orig_len=0.0),
    dict(rot_dim=64, scaling=pa.PA_ROPE_YARN, factor=2.0, orig_len=4096, low_turns=4.0, high_turns=4.0),
    dict(rot_dim=64, scaling=pa.PA_ROPE_YARN, factor=2.0, orig_len=4096, low_turns=0.0),
    dict(rot_dim=16, inv_freq=[math.nan] * 8), dict(rot_dim=16, inv_freq=[1.0] * 8, amplitude=math.inf),
])
def test_rope_refuses_bad_scalings(kw):
    with pytest.raises(pa.PagedAttentionError) as e:
        pa.Rope(**kw)
    assert e.value.status == pa.PA_ERR_SHAPE


def test_rope_refuses_a_wrong_number_of_frequencies():
    with pytest.raises(ValueError, match="expected 8"):
        pa.Rope(16, inv_freq=[1.0] * 7)


@pytest.mark.parametrize("rot", [16, 48, 64, 128])
@pytest.mark.parametrize("base", [10000.0, 500000.0])
@pytest.mark.parametrize("kw", [
    dict(scaling=pa.PA_ROPE_NONE),
    dict(scaling=pa.PA_ROPE_LINEAR, factor=4.0),
    dict(scaling=pa.PA_ROPE_PARTS, factor=8.0, orig_len=8192, low_turns=1.0, high_turns=4.0),
    dict(scaling=pa.PA_ROPE_YARN, factor=16.0, orig_len=4096),
    dict(scaling=pa.PA_ROPE_YARN, factor=1.0, orig_len=64),
])
def test_scaled_frequencies(rot, base, kw):
    r = pa.Rope(rot, base=base, **kw)
    f, amp = inv_freq(rot, base, kw["scaling"], kw.get("factor", 1.0), kw.get("orig_len", 0.0),
                      kw.get("low_turns", 1.0), kw.get("high_turns", 32.0))
    # pow and a few products of 64-bit values: a handful of roundings.
    np.testing.assert_allclose(r.inv_freq, f, rtol=16 * 2.0 ** -53)
    assert abs(r.amplitude - amp) <= 2.0 ** -24 * amp


def test_a_rotation_holds_the_fraction_of_a_turn():
    # 2 pi to 50 digits; the fraction may be off by the 64-bit roundings of
    # the quotient (2^-52 relative) and by the last of its 64 bits.
    two_pi = Fraction("6.2831853071795864769252867665590057683943387987502")
    f = [1.0, 1e-4, 0.5, 6.2, 7.0, 100.25, 3e-9, -0.25]
    r = pa.Rope(16, inv_freq=f)
    for x, got in zip(f, list(r.struct.turn)[:8]):
        turns = Fraction(x) / two_pi
        want = turns - math.floor(turns)
        off = abs(Fraction(got, 1 << 64) - want)
        off = min(off, 1 - off)
        assert off <= abs(turns) * Fraction(1, 1 << 52) + Fraction(1, 1 << 53)
    assert list(r.struct.turn)[8:] == [0] * 56


def test_binding_refuses_host_tensors_shapes_and_types():
    i32 = torch.int32
    n = torch.zeros(2, dtype=i32)
    one = torch.zeros(1, dtype=i32)
    bf = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pool = torch.zeros(4, 4, 16, 64, dtype=torch.bfloat16)
    slots = torch.zeros(2, dtype=torch.int64)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.pa_step_maps(n, n, n, one, torch.zeros(2, 4, dtype=i32), 16, 4, 64, n, torch.zeros(3, dtype=i32),
                        n, slots, one)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.pa_qk_rope(bf, bf, n, None, bf, bf)
    with pytest.raises(ValueError, match="CUDA device"):
        pa.pa_qk_rope_append(bf, bf, bf, n, slots, None, pool, pool, bf)
