"""GPU: the norm, rotation and cache write of rows against 64-bit references:
both pair layouts, every rotated size, both types, strided and in-place rows,
far and negative positions, values that are not finite, padding rows, slots
that are wrong, pools past 2^31 elements, captured calls and side streams.

Tolerances: the reference's bound on the 32-bit arithmetic (step_reference.
norm_rope) plus the one rounding of the stored value, half a step: 2^-8 of it
in bf16, 2^-24 in float32 (2^-134 and 2^-150 absolutely, below the normal range)."""

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from step_reference import norm_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


DT = {"bf16": torch.bfloat16, "f32": torch.float32}
STEP = {"bf16": (2.0 ** -8, 2.0 ** -134), "f32": (2.0 ** -24, 2.0 ** -150)}


def rows(shape, dtype, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(DT[dtype])


def f64(t):
    return t.detach().double().cpu().numpy()


def close(got, ref, bound, dtype, what):
    rel, tiny = STEP[dtype]
    g = f64(got)
    tol = bound * (1 + rel) + rel * np.abs(ref) + tiny
    bad = ~(np.abs(g - ref) <= tol)
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.nanmax(np.abs(g - ref) / tol):.2f} of the tolerance"


class Case:
    def __init__(self, T=5, Hq=4, Hk=2, D=128, rot=128, inter=False, dtype="bf16", norm=True, fused=True,
                 far=100000, seed=0, bs=16, spec=None, scale=1.0, weights=None):
        rng = np.random.default_rng(seed)
        self.__dict__.update(T=T, Hq=Hq, Hk=Hk, D=D, rot=rot, inter=inter, dtype=dtype, bs=bs)
        dt = DT[dtype]
        if fused:
            x = rows((T, Hq + 2 * Hk, D), dtype, seed, scale).cuda()
            self.q, self.k, self.v = x[:, :Hq], x[:, Hq:Hq + Hk], x[:, Hq + Hk:]
        else:
            self.q, self.k, self.v = (rows((T, h, D), dtype, seed + 5 * i, scale).cuda()
                                      for i, h in enumerate((Hq, Hk, Hk)))
        self.posh = rng.integers(-far // 8, far, size=T).astype(np.int32)
        self.pos = torch.from_numpy(self.posh).cuda()
        nq, nk = (norm, norm) if weights is None else weights
        self.qw = (1 + 0.3 * rows((D,), "f32", seed + 3)).to(dt).cuda() if nq else None
        self.kw = (1 + 0.3 * rows((D,), "f32", seed + 4)).to(dt).cuda() if nk else None
        self.rope = spec or (pa.Rope(rot, layout=int(inter)) if rot else None)
        self.q_out = torch.full((T, Hq, D), 7.5, dtype=dt, device="cuda")
        self.k_out = torch.full((T, Hk, D), 7.5, dtype=dt, device="cuda")
        self.NB = -(-T // bs) + 2
        order = rng.permutation(self.NB * bs)[:T].astype(np.int64)
        self.sloth = order
        self.slots = torch.from_numpy(order).cuda()
        self.k_pool = rows((self.NB, Hk, bs, D), dtype, seed + 8).cuda()
        self.v_pool = rows((self.NB, Hk, bs, D), dtype, seed + 9).cuda()

    def ref(self, x, w):
        r = self.rope
        return norm_rope(f64(x), self.posh, np.array(r.inv_freq) if r else None, r.amplitude if r else 1.0,
                         self.rot if r else 0, self.inter, None if w is None else f64(w))

    def rotate(self, q_out=None, k_out=None, **kw):
        pa.pa_qk_rope(self.q, self.k, self.pos, self.rope, self.q_out if q_out is None else q_out,
                      self.k_out if k_out is None else k_out, q_weight=self.qw, k_weight=self.kw, **kw)

    def append(self, **kw):
        pa.pa_qk_rope_append(self.q, self.k, self.v, self.pos, self.slots, self.rope, self.k_pool,
                             self.v_pool, self.q_out, q_weight=self.qw, k_weight=self.kw, **kw)

    def check_rows(self):
        close(self.q_out, *self.ref(self.q, self.qw), self.dtype, "q")
        close(self.k_out, *self.ref(self.k, self.kw), self.dtype, "k")

    def check_append(self, before, keep=None):
        keep = np.ones(self.T, dtype=bool) if keep is None else keep
        kp0, vp0 = before
        blk, off = self.slots[torch.from_numpy(keep).cuda()] // self.bs, self.slots[torch.from_numpy(keep).cuda()] % self.bs
        m = torch.from_numpy(keep).cuda()
        ref, bound = self.ref(self.k, self.kw)
        close(self.k_pool[blk, :, off], ref[keep], bound[keep], self.dtype, "k pool")
        raw = torch.int16 if self.dtype == "bf16" else torch.int32
        assert torch.equal(self.v_pool[blk, :, off].view(raw), self.v[m].contiguous().view(raw))
        kp, vp = self.k_pool.clone(), self.v_pool.clone()
        kp[blk, :, off], vp[blk, :, off] = kp0[blk, :, off], vp0[blk, :, off]
        assert torch.equal(kp.view(raw), kp0.view(raw)) and torch.equal(vp.view(raw), vp0.view(raw))
        qr, qb = self.ref(self.q, self.qw)
        close(self.q_out[m], qr[keep], qb[keep], self.dtype, "q")
        assert bool((self.q_out[~m] == 7.5).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 96), (128, 64), (128, 16), (128, 0), (64, 64),
                                   (64, 48), (64, 16), (64, 0)])
@pytest.mark.parametrize("norm", [False, True])
def test_rotation(dtype, inter, D, rot, norm):
    c = Case(T=7, D=D, rot=rot, inter=inter, dtype=dtype, norm=norm, seed=rot + D)
    c.rotate()
    c.check_rows()
    if not norm:   # what is not rotated keeps its bits
        assert torch.equal(c.q_out[..., rot:], c.q[..., rot:]) and torch.equal(c.k_out[..., rot:], c.k[..., rot:])


@pytest.mark.parametrize("T,Hq,Hk", [(1, 1, 1), (1, 32, 8), (2, 3, 1), (3, 5, 5), (64, 32, 8), (65, 7, 2),
                                     (1000, 8, 1), (5003, 4, 2), (20000, 1, 1), (1, 600, 300)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rows_and_heads(T, Hq, Hk, dtype):
    c = Case(T=T, Hq=Hq, Hk=Hk, dtype=dtype, seed=T, fused=T % 2 == 0)
    c.rotate()
    c.check_rows()
    before = c.k_pool.clone(), c.v_pool.clone()
    c.q_out.fill_(7.5)
    c.append()
    c.check_append(before)
    assert pa.pa_last_device_error(None) == 0


@pytest.mark.parametrize("weights", [(True, False), (False, True)])
def test_norm_of_one_side_only(weights):
    c = Case(T=9, weights=weights, seed=4, Hq=3, Hk=3)
    c.rotate()
    c.check_rows()


@pytest.mark.parametrize("spec", [
    dict(scaling=pa.PA_ROPE_LINEAR, factor=4.0),
    dict(scaling=pa.PA_ROPE_PARTS, factor=8.0, orig_len=8192, high_turns=4.0),
    dict(scaling=pa.PA_ROPE_YARN, factor=16.0, orig_len=4096),
    dict(inv_freq=[100.0 - 3 * i for i in range(32)], amplitude=-0.5),
])
def test_scaled_rotations(spec):
    c = Case(T=33, rot=64, spec=pa.Rope(64, **spec), dtype="f32", norm=False, far=1 << 20)
    c.rotate()
    c.check_rows()


def test_far_positions():
    c = Case(T=8, dtype="f32", norm=False)
    c.posh = np.array([0, 1, -1, 2 ** 31 - 1, -2 ** 31, 2 ** 30, 12345678, -99999999], dtype=np.int32)
    c.pos = torch.from_numpy(c.posh).cuda()
    c.rotate()
    c.check_rows()
    # Position 0 turns nothing: an exact copy.
    assert torch.equal(c.q_out[0], c.q[0])


def test_a_turn_and_back():
    # Positions p, then -p: the rows again. With u = 2^-24 and m = |x1| + |x2|,
    # the first turn is off by 8u m and its store by u m in each element, up to
    # 18u m when turned back; the second is off by 9u (|y1| + |y2|) <= 9 sqrt(2) u m.
    # The two angles are exact negatives of each other.
    c = Case(T=40, dtype="f32", norm=False)
    c.rotate()
    back_q, back_k = torch.empty_like(c.q_out), torch.empty_like(c.k_out)
    pa.pa_qk_rope(c.q_out, c.k_out, -c.pos, c.rope, back_q, back_k)
    m = (c.q.abs() + c.q.roll(64, -1).abs()).double()
    assert bool(((back_q - c.q).double().abs() <= 32 * m * 2.0 ** -24).all())


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("inter", [False, True])
def test_in_place(dtype, inter):
    c = Case(T=50, dtype=dtype, inter=inter, rot=64, seed=6)
    c.rotate()
    q, k = c.q.clone(), c.k.clone()
    v = c.v.clone()
    c.rotate(q_out=c.q, k_out=c.k)           # views of the fused rows
    assert torch.equal(c.q, c.q_out) and torch.equal(c.k, c.k_out) and torch.equal(c.v, v)
    c.q.copy_(q)
    c.k.copy_(k)
    c.check_rows()


@pytest.mark.parametrize("norm", [False, True])
def test_values_that_are_not_finite_stay_in_their_head(norm):
    c = Case(T=6, Hq=4, Hk=2, norm=norm, rot=64, dtype="f32")
    c.q[1, 2, 3] = float("nan")
    c.q[2, 0, 100] = float("inf")           # not rotated
    c.k[3, 1, 5] = float("-inf")
    c.rotate()
    fin = torch.isfinite(c.q_out)
    assert not bool(fin[1, 2, 3]) and not bool(fin[1, 2, 35])
    fin[1, 2], fin[2, 0] = True, True
    assert bool(fin.all())
    if not norm:
        assert bool(torch.isfinite(c.q_out[1, 2, :3]).all()) and bool(c.q_out[2, 0, 100] == float("inf"))
        rest = torch.cat([c.q_out[2, 0, :100], c.q_out[2, 0, 101:]])
        assert bool(torch.isfinite(rest).all())
    kf = torch.isfinite(c.k_out)
    kf[3, 1] = True
    assert bool(kf.all())


def test_zero_rows_and_tiny_rows_under_the_norm():
    c = Case(T=4, dtype="f32", scale=1.0)
    c.q[0] = 0
    c.q[1] *= 1e-18
    c.q[2] *= 1e15
    c.rotate()
    c.check_rows()
    assert bool((c.q_out[0] == 0).all())


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("bf16", 64), ("f32", 128), ("f32", 64)])
def test_append_padding_and_wrong_slots(bs, dtype, D):
    c = Case(T=41, Hq=6, Hk=3, D=D, rot=32, bs=bs, dtype=dtype, seed=bs + D)
    c.sloth = c.sloth.copy()
    c.sloth[[0, 7, 40]] = -1
    c.slots = torch.from_numpy(c.sloth).cuda()
    before = c.k_pool.clone(), c.v_pool.clone()
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    c.append(device_error=err)
    c.check_append(before, c.sloth >= 0)
    assert int(err) == 0
    c.sloth[[1, 2]] = [c.NB * bs, -2]
    c.sloth[3] = 2 ** 40
    c.slots = torch.from_numpy(c.sloth).cuda()
    c.k_pool.copy_(before[0])
    c.v_pool.copy_(before[1])
    c.q_out.fill_(7.5)
    c.append(device_error=err)
    c.check_append(before, (c.sloth >= 0) & (c.sloth < c.NB * bs))
    assert int(err) == pa.PA_DEVERR_TABLE
    c.append()
    assert pa.pa_last_device_error(None) == pa.PA_DEVERR_TABLE


def test_the_bits_of_values_pass_through():
    c = Case(T=16, Hq=2, Hk=2)
    raw = torch.arange(16 * 2 * 128, device="cuda").to(torch.int16) * 17 - 30000   # NaN payloads among them
    c.v = raw.view(torch.bfloat16).view(16, 2, 128)
    c.append()
    blk, off = c.slots // 16, c.slots % 16
    assert torch.equal(c.v_pool[blk, :, off].view(torch.int16), c.v.view(torch.int16))


def test_a_pool_past_32_bits():
    # 2^31 elements end at block 2^31 / (8 * 32 * 128) = 65536: the last blocks lie behind.
    NB, Hk, bs, D = 65600, 8, 32, 128
    c = Case(T=12, Hq=8, Hk=Hk, D=D, bs=bs)
    c.NB = NB
    c.k_pool = torch.zeros(NB, Hk, bs, D, dtype=torch.bfloat16, device="cuda")
    c.v_pool = torch.zeros(NB, Hk, bs, D, dtype=torch.bfloat16, device="cuda")
    c.sloth = np.array([NB * bs - 1 - 37 * i for i in range(12)], dtype=np.int64)
    c.slots = torch.from_numpy(c.sloth).cuda()
    c.append()
    blk, off = c.slots // bs, c.slots % bs
    ref, bound = c.ref(c.k, c.kw)
    close(c.k_pool[blk, :, off], ref, bound, "bf16", "k pool")
    assert torch.equal(c.v_pool[blk, :, off], c.v)
    assert int((c.v_pool != 0).any(-1).sum()) == 12 * Hk


def test_side_stream_and_graph_replay():
    c = Case(T=70, Hq=8, Hk=2, seed=3)
    before = c.k_pool.clone(), c.v_pool.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    c.append(stream=side)
    torch.cuda.synchronize()
    c.check_append(before)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.append()
    other = Case(T=70, Hq=8, Hk=2, seed=5)
    c.q.copy_(other.q)
    c.k.copy_(other.k)
    c.v.copy_(other.v)
    c.pos.copy_(other.pos)
    c.posh = other.posh
    c.k_pool.copy_(before[0])
    c.v_pool.copy_(before[1])
    g.replay()
    torch.cuda.synchronize()
    c.check_append(before)


def test_the_same_call_gives_the_same_bits():
    c = Case(T=3000, Hq=8, Hk=2)
    c.rotate()
    a = c.q_out.clone(), c.k_out.clone()
    c.rotate()
    assert torch.equal(a[0], c.q_out) and torch.equal(a[1], c.k_out)


def test_binding_refuses_shapes_types_and_strides():
    c = Case(T=4, Hq=4, Hk=2)
    for kw, e in ((dict(q_out=c.k_out), ValueError), (dict(q_out=c.q_out.float()), TypeError),
                  (dict(k_out=c.k_out.transpose(1, 2).contiguous().transpose(1, 2)), ValueError)):
        with pytest.raises(e):
            c.rotate(**kw)
    c.pos = c.pos.long()
    with pytest.raises(TypeError):
        c.rotate()
    c.pos = c.pos.int()
    c.slots = c.slots.int()
    with pytest.raises(TypeError):
        c.append()
    c.slots = c.slots.long()[:2]
    with pytest.raises(ValueError):
        c.append()
    c = Case(T=4, Hq=4, Hk=2, D=64, rot=64)
    c.rope = pa.Rope(128)
    with pytest.raises(pa.PagedAttentionError):
        c.rotate()
    c = Case(T=0)
    c.rotate()
    c.append()
    torch.cuda.synchronize()
