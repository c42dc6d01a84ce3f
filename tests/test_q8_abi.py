"""The 8-bit cache's calls on the host (no GPU): bad arguments are refused before
any CUDA call, and the references of the GPU tests follow the format."""

import ctypes
import math

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
import q8_reference as ref
from paged_kv_cache_202_gb300 import _build


@pytest.fixture(scope="module", autouse=True)
def lib():
    _build.build()
    return pa.lib()


A = 0x10000  # a fake, 16-byte aligned device address: never dereferenced


def _write(lib, **kw):
    rope = pa.Rope(64).struct
    a = dict(q=A, qs=32 * 128, k=A, ks=8 * 128, v=A, vs=8 * 128, pos=A, st=A, bt=A, mb=8, sl=A, B=4, T=8, Hq=32,
             Hkv=8, D=128, dt=pa.PA_BF16, qw=None, kw=None, eps=1e-6, rope=ctypes.byref(rope), qo=A, qos=32 * 128,
             kp=A, vp=A, ksc=A, vsc=A, bs=16, NB=64, err=None)
    a.update(kw)
    return lib.pa_qk_rope_append_q8(*[a[n] for n in (
        "q", "qs", "k", "ks", "v", "vs", "pos", "st", "bt", "mb", "sl", "B", "T", "Hq", "Hkv", "D", "dt", "qw", "kw",
        "eps", "rope", "qo", "qos", "kp", "vp", "ksc", "vsc", "bs", "NB", "err")], None)


def _read(lib, **kw):
    a = dict(kp=A, vp=A, ksc=A, vsc=A, bt=A, mb=8, sl=A, st=A, B=4, T=8, Hkv=8, D=128, bs=16, NB=64, ko=A, vo=A,
             dt=pa.PA_BF16, err=None)
    a.update(kw)
    return lib.pa_read_kv_q8(*[a[n] for n in ("kp", "vp", "ksc", "vsc", "bt", "mb", "sl", "st", "B", "T", "Hkv", "D",
                                              "bs", "NB", "ko", "vo", "dt", "err")], None)


def _decode(lib, **kw):
    plan = ctypes.c_void_p(None)
    a = dict(q=A, kp=A, vp=A, ksc=A, vsc=A, bt=A, mb=8, sl=A, B=4, Hq=32, Hkv=8, D=128, bs=16, NB=64, maxlen=128,
             scale=0.1, out=A, od=pa.PA_BF16, plan=ctypes.byref(plan))
    a.update(kw)
    st = lib.pa_decode_q8(*[a[n] for n in ("q", "kp", "vp", "ksc", "vsc", "bt", "mb", "sl", "B", "Hq", "Hkv", "D",
                                           "bs", "NB", "maxlen", "scale", "out", "od", "plan")], None)
    assert plan.value is None   # a refused call makes no plan
    return st


def _prefill(lib, **kw):
    plan = ctypes.c_void_p(None)
    a = dict(q=A, st=A, T=8, mq=4, kp=A, vp=A, ksc=A, vsc=A, bt=A, mb=8, sl=A, B=4, Hq=32, Hkv=8, D=128, bs=16, NB=64,
             maxlen=128, scale=0.1, out=A, od=pa.PA_BF16, plan=ctypes.byref(plan))
    a.update(kw)
    st = lib.pa_prefill_q8(*[a[n] for n in ("q", "st", "T", "mq", "kp", "vp", "ksc", "vsc", "bt", "mb", "sl", "B",
                                            "Hq", "Hkv", "D", "bs", "NB", "maxlen", "scale", "out", "od", "plan")],
                           None)
    assert plan.value is None
    return st


N, SH, DT, BS, AL, OK = (pa.PA_ERR_NULL, pa.PA_ERR_SHAPE, pa.PA_ERR_DTYPE, pa.PA_ERR_BLOCK_SIZE, pa.PA_ERR_ALIGN,
                         pa.PA_OK)


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, N) for n in ("q", "k", "v", "pos", "st", "bt", "sl", "qo", "kp", "vp", "ksc", "vsc")],
    (dict(dt=pa.PA_F32), DT), (dict(dt=7), DT), (dict(bs=8), BS), (dict(bs=64), BS), (dict(B=-1), SH),
    (dict(B=8193), SH), (dict(T=-1), SH), (dict(mb=0), SH), (dict(mb=1 << 28), SH), (dict(NB=0), SH),
    (dict(NB=1 << 29), SH), (dict(D=96), SH), (dict(Hq=0), SH), (dict(Hkv=0), SH), (dict(eps=-1.0), SH),
    (dict(eps=math.nan), SH), (dict(qs=32 * 128 - 8), SH), (dict(vs=8 * 128 + 4), SH), (dict(vs=8), SH),
    (dict(D=64, rope=ctypes.byref(pa._RopeStruct(rot_dim=128, layout=0, amplitude=1.0))), SH),
    *[({n: A + 8}, AL) for n in ("q", "k", "v", "qo", "kp", "vp", "qw", "kw")],
    *[({n: A + 2}, AL) for n in ("pos", "st", "bt", "sl", "ksc", "vsc", "err")],
    (dict(T=0), OK), (dict(B=0), OK),
])
def test_write_refuses(lib, kw, status):
    assert _write(lib, **kw) == status


@pytest.mark.parametrize("kw,status", [
    *[({n: None}, N) for n in ("kp", "vp", "ksc", "vsc", "bt", "sl", "st", "ko", "vo")],
    (dict(dt=5), DT), (dict(bs=0), BS), (dict(B=-1), SH), (dict(B=8193), SH), (dict(T=-1), SH), (dict(mb=0), SH),
    (dict(NB=0), SH), (dict(D=32), SH), (dict(Hkv=0), SH), (dict(mb=1 << 28), SH),
    *[({n: A + 8}, AL) for n in ("kp", "vp", "ko", "vo")], *[({n: A + 1}, AL) for n in ("ksc", "vsc", "bt", "sl", "st",
                                                                                         "err")],
    (dict(T=0), OK), (dict(B=0), OK),
])
def test_read_refuses(lib, kw, status):
    assert _read(lib, **kw) == status


_BOTH = [
    *[({n: None}, N) for n in ("q", "kp", "vp", "ksc", "vsc", "bt", "sl", "out", "plan")],
    (dict(od=3), DT), (dict(bs=24), BS), (dict(B=-1), SH), (dict(B=8193), SH), (dict(Hq=12), SH), (dict(Hq=0), SH),
    (dict(Hkv=0), SH), (dict(D=80), SH), (dict(mb=0), SH), (dict(NB=0), SH), (dict(NB=1 << 29), SH),
    (dict(maxlen=0), SH), (dict(scale=math.nan), SH), (dict(scale=math.inf), SH),
    *[({n: A + 8}, AL) for n in ("q", "kp", "vp", "out")], *[({n: A + 2}, AL) for n in ("ksc", "vsc", "bt", "sl")],
    (dict(B=0), OK),
]


@pytest.mark.parametrize("kw,status", _BOTH + [(dict(B=8192, Hq=1 << 18, Hkv=1 << 18), SH)])
def test_decode_refuses(lib, kw, status):
    assert _decode(lib, **kw) == status


@pytest.mark.parametrize("kw,status", _BOTH + [
    (dict(st=None), N), (dict(st=A + 2), AL), (dict(T=-1), SH), (dict(mq=0), SH), (dict(D=64), SH),
    (dict(Hq=40, Hkv=8), SH), (dict(Hq=256, Hkv=1), SH), (dict(mb=16385), SH), (dict(scale=0.0), SH),
    (dict(scale=-1.0), SH), (dict(T=0), OK),
])
def test_prefill_refuses(lib, kw, status):
    assert _prefill(lib, **kw) == status


def test_decode_refuses_page_streams_past_32_bits(lib):
    """8192 sequences x 64 kv heads x 4095 pages: their number fits 32 bits, but not that and a warp's share."""
    assert _decode(lib, B=8192, Hq=64, Hkv=64, mb=4095, maxlen=4095 * 16) == SH


@pytest.mark.skipif(torch.cuda.is_available(), reason="a GPU would run the call on its fake addresses")
def test_prefill_of_few_queries_takes_streams_past_32_bits(lib):
    """The same bounds are within those of pa_prefill_q8, whatever max_q: not refused, and no GPU to run on."""
    for mq in (1, 4, 40):
        assert _prefill(lib, B=8192, Hq=64, Hkv=64, mb=4095, maxlen=4095 * 16, mq=mq, T=40) == pa.PA_ERR_CUDA


@pytest.mark.parametrize("D,dt,status", [(64, pa.PA_BF16, OK), (32, pa.PA_BF16, OK), (32, pa.PA_F32, SH),
                                         (16, pa.PA_BF16, SH)])
def test_block_copies_take_codes_as_bf16_of_half_the_width(lib, D, dt, status):
    for bs in (16, 32):
        assert lib.pa_copy_blocks(A, A, A, A, 0, 3, D, bs, 64, dt, None) == status


def test_binding_refuses_host_tensors():
    z = torch.zeros
    i32 = torch.int32
    pool, sc = z(4, 2, 16, 64, dtype=torch.uint8), z(4, 2)
    with pytest.raises(ValueError):
        pa.pa_decode_q8(z(2, 4, 64, dtype=torch.bfloat16), pool, pool, sc, sc, z(2, 2, dtype=i32), z(2, dtype=i32),
                        0.1, z(2, 4, 64), 32, pa.Plan())
    with pytest.raises(ValueError):
        pa.pa_read_kv_q8(pool, pool, sc, sc, z(2, 2, dtype=i32), z(2, dtype=i32), z(3, dtype=i32), z(5, 2, 64),
                         z(5, 2, 64))


def test_reference_format():
    t = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(t, ref.VALUES)
    x = np.random.default_rng(1).standard_normal(20000) * np.exp2(np.random.default_rng(2).uniform(-12, 6, 20000))
    x = np.clip(x, -448, 448).astype(np.float32)
    # Ties and the format's ends among them.
    mids = ((ref.VALUES[:0x7e] + ref.VALUES[1:0x7f]) / 2).astype(np.float32)
    x = np.concatenate([x, mids, -mids, ref.VALUES[:0x7f].astype(np.float32), [0.0, -0.0, 2.0 ** -10, 448.0]])
    x = x.astype(np.float32)
    np.testing.assert_array_equal(ref.nearest(x), torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8))
    assert ref.nearest([np.nan, np.inf]).tolist() == [0x7f, 0x7f]
    for a, s in ((0.0, 2.0 ** -64), (448.0, 1.0), (448.0001, 2.0), (3.5, 2.0 ** -7), (3.51, 2.0 ** -6)):
        assert ref.scale_for(a) == s
