"""Calls of the 8-bit cache at the edges of what they take."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
import q8_reference as ref

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _q(T, Hq, D, seed):
    return torch.randn(T, Hq, D, generator=torch.Generator("cuda").manual_seed(seed), device="cuda").to(torch.bfloat16)


@pytest.fixture
def plan():
    p = pa.Plan()
    yield p
    p.free()


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 32)])
@pytest.mark.parametrize("lens", [[0, 0, 0], [-1, 400, 0], [301, 302, 1 << 30]], ids=str)
def test_decode_of_invalid_sequences_alone(lens, D, bs, plan):
    """No sequence has a page: zero rows and the error bit, and the plan's next call is right."""
    c = ref.Cache([300, 300, 300], 2, D, bs, seed=1)
    q = _q(3, 8, D, 2)
    want, tol = ref.attention(c, q, [1] * 3, 0.1)
    for _ in range(2):
        out = torch.full((3, 8, D), 3.0, device="cuda")
        pa.pa_decode_q8(q, *c.args, c.dtables, _i32(lens), 0.1, out, 300, plan)
        assert pa.pa_last_device_error(plan) == pa.PA_DEVERR_SEQ_LEN
        assert bool((out == 0).all())
        pa.pa_decode_q8(q, *c.args, c.dtables, c.dlens, 0.1, out, 300, plan)
        assert pa.pa_last_device_error(plan) == 0
        ref.check(out, want, tol)


def test_few_queries_of_invalid_or_idle_sequences_alone(plan):
    """The same on the decode's tiles: idle requests leave the padded rows, invalid ones get zeros."""
    c = ref.Cache([300, 40], 2, 128, 16, seed=3)
    q = _q(6, 8, 128, 4)
    want, tol = ref.attention(c, q[:4], [3, 1], 0.1)
    for start, lens, bit, left in (([0, 0, 0], [300, 40], 0, 0), ([0, 0, 0], [0, 0], 0, 0),
                                   ([0, 3, 4], [2, 0], pa.PA_DEVERR_SEQ_LEN, 4)):
        out = torch.full((6, 8, 128), 3.0, device="cuda")
        pa.pa_prefill_q8(q, _i32(start), *c.args, c.dtables, _i32(lens), 0.1, out, 3, 300, plan)
        assert pa.pa_last_device_error(plan) == bit
        assert bool((out[:left] == 0).all()) and bool((out[left:] == 3).all())
        pa.pa_prefill_q8(q, _i32([0, 3, 4]), *c.args, c.dtables, c.dlens, 0.1, out, 3, 300, plan)
        assert pa.pa_last_device_error(plan) == 0
        ref.check(out[:4], want, tol)
        assert bool((out[4:] == 3).all())


def test_few_queries_within_wide_bounds(plan):
    """8192 requests of up to 65535 tokens by the call's bounds, a few of them with queries: too many
    pages for the decode's tiles, not for the call."""
    B, Hkv, MB = 8192, 64, 4096
    lens, new = [300, 1, 40], [2, 1, 2]
    c = ref.Cache(lens, Hkv, 128, 16, seed=5)
    at = [0, 5000, B - 1]
    tables = torch.full((B, MB), -1, dtype=torch.int32, device="cuda")
    seq, n = torch.zeros(B, dtype=torch.int32), torch.zeros(B, dtype=torch.int32)
    for b, L, k, row in zip(at, lens, new, c.tables):
        tables[b, :c.MB] = torch.from_numpy(row).cuda()
        seq[b], n[b] = L, k
    start = torch.cat([torch.zeros(1, dtype=torch.int32), torch.cumsum(n, 0, dtype=torch.int32)]).cuda()
    q = _q(sum(new), Hkv, 128, 6)
    out = torch.full(q.shape, math.nan, device="cuda")
    pa.pa_prefill_q8(q, start, *c.args, tables, seq.cuda(), 0.1, out, 2, MB * 16, plan)
    assert pa.pa_last_device_error(plan) == 0
    ref.check(out, *ref.attention(c, q, new, 0.1))


def test_no_sequences(plan):
    """B = 0 with padded rows is a no-op in all four calls."""
    c = ref.Cache([40], 2, 128, 16, seed=7)
    before = [t.view(torch.uint8).clone() for t in c.args]
    T, none, tables = 5, _i32([]), torch.empty(0, c.MB, dtype=torch.int32, device="cuda")
    q, k, v = _q(T, 8, 128, 1), _q(T, 2, 128, 2), _q(T, 2, 128, 3)
    out, kr, vr = torch.full_like(q, 3.0), torch.full_like(k, 3.0), torch.full_like(v, 3.0)
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    pa.pa_qk_rope_append_q8(q, k, v, _i32([0] * T), _i32([0]), tables, none, None, *c.args, out, device_error=err)
    pa.pa_read_kv_q8(*c.args, tables, none, _i32([0]), kr, vr, device_error=err)
    pa.pa_prefill_q8(q, _i32([0]), *c.args, tables, none, 0.1, out, 1, 40, plan)
    pa.pa_decode_q8(q[:0], *c.args, tables, none, 0.1, out[:0], 40, plan)
    assert int(err) == 0 and all(bool((t == 3).all()) for t in (out, kr, vr))
    for t, b in zip(c.args, before):
        assert torch.equal(t.view(torch.uint8), b)


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 32)])
def test_write_over_scales_that_are_no_powers_of_two(D, bs):
    """A caller's larger scale stays, and every code is within half a step and 2^-22 of x (or of the earlier
    token's value), also where x / scale is within 2^-24 of the middle of two codes; a smaller one grows to
    a power of two."""
    nb, Hkv = 60, 4
    rng = np.random.default_rng(10)
    x = torch.from_numpy(rng.uniform(1, 2, (nb, Hkv))).to(torch.bfloat16).double().numpy()
    middle = rng.integers(8, 16, (nb, Hkv)) + 0.5   # of two neighbouring codes
    scales = (x / middle).astype(np.float32)
    scales[:, 1] *= np.float32(2.0 ** -12)          # too small for the new token
    powers = 2.0 ** rng.integers(-12, 1, (nb, Hkv, D))
    powers[..., 0] = 1
    rows = x[..., None] * powers * rng.choice([-1.0, 1.0], (nb, Hkv, D))
    c = ref.Cache([2] * nb, Hkv, D, bs, seed=8, slack=0)
    blk = c.tables[:, 0]
    for s, codes in zip(c.scales, c.codes):   # an earlier token in every block
        s[blk] = scales
        codes[blk, :, 0] = ref.nearest(rng.uniform(-448, 448, (nb, Hkv, D)))
    c.upload()
    new = torch.from_numpy(rows).to(torch.bfloat16).cuda()
    pa.pa_qk_rope_append_q8(new, new, new, _i32([0] * nb), _i32(range(nb + 1)), c.dtables, c.dlens, None, *c.args,
                            torch.empty_like(new))
    need = np.vectorize(ref.scale_for)(np.abs(rows).max(-1))
    assert bool((need[:, 1] > scales[:, 1]).all()) and bool((np.delete(need <= scales, 1, 1)).all())
    for pool, scale, codes in zip(c.args[:2], c.args[2:], c.codes):
        s = scale.cpu().numpy()[blk]
        np.testing.assert_array_equal(s, np.maximum(scales, need).astype(np.float32))
        got = ref.VALUES[pool.view(torch.uint8).cpu().numpy()[blk]]
        old = ref.VALUES[codes[blk][:, :, 0]] * scales[..., None].astype(np.float64)
        s = s.astype(np.float64)[..., None]
        for i, y in ((0, old), (1, rows)):
            assert np.all(np.abs(got[:, :, i] * s - y) <= ref.half_step(y / s * (1 + 2.0 ** -22)) * s + 2.0 ** -22 * np.abs(y))
        keep = [h for h in range(Hkv) if h != 1]
        np.testing.assert_array_equal(got[:, keep, 0], ref.VALUES[codes[blk]][:, keep, 0])
        assert bool(np.isnan(got[:, :, 2:]).all())


@pytest.mark.parametrize("D,bs", [(128, 16), (64, 32)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_rounds_as_documented(D, bs, dtype):
    """Code times scale to float32, and that to bf16, bit for bit, for products within 2^-24 of the middle
    of two bf16 numbers too (what rounding once would change)."""
    nb, Hkv = 50, 6
    rng = np.random.default_rng(11)
    c = ref.Cache([bs] * nb, Hkv, D, bs, seed=12, slack=0)
    # Scales whose products with the codes of mantissa 9, 11, 13 or 15 come next to j + 1/2 for 8 bits j.
    m = rng.choice([9, 11, 13, 15], (2, nb, Hkv))
    f = np.rint((2 * rng.integers(128, 256, (2, nb, Hkv)) + 1) * 2.0 ** 18 / m) * 2.0 ** rng.integers(-40, -20, (2, nb, Hkv))
    for i in range(2):
        c.scales[i][c.tables[:, 0]] = f[i].astype(np.float32)
    c.upload()
    outs = [torch.full((nb * bs, Hkv, D), math.nan, dtype=dtype, device="cuda") for _ in range(2)]
    pa.pa_read_kv_q8(*c.args, c.dtables, c.dlens, _i32(range(0, (nb + 1) * bs, bs)), *outs)
    for i, out in enumerate(outs):
        y = torch.cat([c.dense(b)[i].transpose(0, 1) for b in range(nb)])   # exact in 64 bits
        assert int((y != y.float().double()).sum()) > 1000
        assert torch.equal(out, y.float().to(dtype))


@pytest.mark.parametrize("kernel,tile", [(pa.PA_PREFILL_AUTO, 64), (pa.PA_PREFILL_ONE_TILE, 32),
                                         (pa.PA_PREFILL_TWO_TILE, 64)])
@pytest.mark.parametrize("at", [0, 31, 300, 479])
def test_how_far_a_value_that_is_no_number_shows(kernel, tile, at, plan):
    """In its own element of the rows that see it, at most of the same tile's (or pair's) other rows, and
    nowhere else."""
    L, n, g = 500, 480, 4
    c = ref.Cache([L], 2, 128, 16, seed=15)
    q = _q(n, 2 * g, 128, 16)
    want, tol = ref.attention(c, q, [n], 0.1)
    tok = L - n + at
    c.v_pool.view(torch.uint8)[int(c.tables[0, tok // 16]), 1, tok % 16, 5] = 0x7f
    pa.pa_debug_set_prefill_kernel(kernel)
    try:
        out = torch.zeros(q.shape, device="cuda")
        pa.pa_prefill_q8(q, _i32([0, n]), *c.args, c.dtables, c.dlens, 0.1, out, n, L, plan)
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)
    assert bool(torch.isnan(out[at:, g:, 5]).all())
    out[at // tile * tile:, g:, 5] = want[at // tile * tile:, g:, 5].float()
    ref.check(out, want, tol)


@pytest.mark.parametrize("kernel,new", [(pa.PA_PREFILL_TWO_TILE, [3000, 1100]), (pa.PA_PREFILL_ONE_TILE, [1000, 96]),
                                        (pa.PA_PREFILL_AUTO, [16, 40])])
def test_prompts_repeat_bit_for_bit(kernel, new, plan):
    """The score product of a chunk is issued behind the value product that reads the weights in the same
    tensor memory, without a wait between them: any overtaking would show as other bits."""
    lens = [4000, 1100]
    c = ref.Cache(lens, 8, 128, 16, seed=17)
    q = _q(sum(new), 32, 128, 18)
    want, tol = ref.attention(c, q, new, 0.1)
    start = _i32([0, new[0], sum(new)])
    first = None
    pa.pa_debug_set_prefill_kernel(kernel)
    try:
        for i in range(40):
            out = torch.full(q.shape, math.nan, device="cuda")
            pa.pa_prefill_q8(q, start, *c.args, c.dtables, c.dlens, 0.1, out, max(new), max(lens), plan)
            if first is None:
                first = out
                ref.check(out, want, tol)
            assert torch.equal(out, first), i
    finally:
        pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)


@pytest.mark.parametrize("Hkv,D,bs", [(3, 64, 16), (2, 64, 32), (1, 128, 16)])
def test_blocks_copied_with_their_scales(Hkv, D, bs, plan):
    """Copy on write of a fork's blocks, as bf16 of half the width: the same codes, and the same rows."""
    c = ref.Cache([200, 90], Hkv, D, bs, seed=19, slack=20)
    used = c.tables[0, :-(-200 // bs)]
    free = [x for x in range(c.NB) if x not in set(c.tables[c.tables >= 0].tolist())][:len(used)]
    src, dst = _i32(used[:len(free)]), _i32(free)
    before = [t.view(torch.uint8).clone() for t in c.args[:2]]
    pa.pa_copy_blocks(*[p.view(torch.uint8).view(torch.bfloat16) for p in c.args[:2]], src, dst)
    for s in c.args[2:]:
        s[dst.long()] = s[src.long()]
    for p, b in zip(c.args[:2], before):
        want = b.clone()
        want[dst.long()] = b[src.long()]
        assert torch.equal(p.view(torch.uint8), want)
    fork = c.dtables.clone()
    fork[0, :len(free)] = dst
    q = _q(2, 4 * Hkv, D, 20)
    outs = [pa.pa_decode_q8(q, *c.args, t, c.dlens, 0.1, torch.zeros_like(q), 200, plan) for t in (c.dtables, fork)]
    assert torch.equal(*outs)


@pytest.mark.parametrize("scale", [-0.1, 0.0, -3.0])
@pytest.mark.parametrize("Hq,Hkv,D", [(8, 2, 128), (17, 1, 64), (34, 2, 128)])
def test_decode_of_any_score_scale(scale, Hq, Hkv, D, plan):
    """Score scales that turn the order round, and none; heads that make slices of unequal size."""
    lens = [700, 3, 33, 5000]
    c = ref.Cache(lens, Hkv, D, 16, seed=21)
    q = _q(4, Hq, D, 22)
    # (The tolerance goes by the scale's magnitude.)
    want, _ = ref.attention(c, q, [1] * 4, scale)
    _, tol = ref.attention(c, -q if scale < 0 else q, [1] * 4, abs(scale))
    out = torch.full((4, Hq, D), math.nan, device="cuda")
    pa.pa_decode_q8(q, *c.args, c.dtables, c.dlens, scale, out, 5000, plan)
    assert pa.pa_last_device_error(plan) == 0
    ref.check(out, want, tol)
