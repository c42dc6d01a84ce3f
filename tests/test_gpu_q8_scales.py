"""Attention over an 8-bit cache whose value scales take the whole range that the write
makes, 2^-64 to 2^120, in any mix, and scales outside it."""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
import q8_reference as ref

pytestmark = pytest.mark.gpu


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _q(T, Hq, D, seed, sigma=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(T, Hq, D, generator=g, device="cuda") * sigma).to(torch.bfloat16)


@pytest.fixture
def plan():
    p = pa.Plan()
    yield p
    p.free()


@pytest.fixture(params=[pa.PA_PREFILL_AUTO, pa.PA_PREFILL_ONE_TILE, pa.PA_PREFILL_TWO_TILE],
                ids=["auto", "one tile", "two tiles"])
def kernel(request):
    pa.pa_debug_set_prefill_kernel(request.param)
    yield request.param
    pa.pa_debug_set_prefill_kernel(pa.PA_PREFILL_AUTO)


def _decode(c, q, plan, dtype=torch.float32):
    out = torch.full(q.shape, math.nan, dtype=dtype, device="cuda")
    return pa.pa_decode_q8(q, *c.args, c.dtables, c.dlens, q.shape[2] ** -0.5, out, max(c.lens), plan)


def _prefill(c, q, new, plan, dtype=torch.float32):
    out = torch.full(q.shape, math.nan, dtype=dtype, device="cuda")
    start = _i32(np.concatenate([[0], np.cumsum(new)]).astype(int))
    return pa.pa_prefill_q8(q, start, *c.args, c.dtables, c.dlens, q.shape[2] ** -0.5, out, max(new), max(c.lens), plan)


def _attention(c, q, new):
    """The reference's rows, and its tolerance with what weights below 2^-32 of the row's largest lose. A
    weight w = p_t vs_t is rounded as w / W 2^7 or more to f16, W the largest, so what lies in its subnormal
    numbers is off by at most half of their step 2^-24: 2^-32 W, times the token's code."""
    scale = q.shape[2] ** -0.5
    want, tol = ref.attention(c, q, new, scale)
    T, Hq, D = q.shape
    row = 0
    for b, n in enumerate(new):
        L, blk = c.lens[b], c.tables[b, :-(-c.lens[b] // c.bs)]
        k, v = c.dense(b)
        vs = torch.from_numpy(np.repeat(c.scales[1][blk].astype(np.float64), c.bs, 0)[:L].T.copy()).to(q.device)
        x = q[row:row + n].double().view(n, c.Hkv, -1, D)
        s = torch.einsum("nhgd,htd->nhgt", x, k) * scale
        vis = torch.arange(L, device=q.device)[None, :] <= torch.arange(L - n, L, device=q.device)[:, None]
        p = torch.softmax(s.masked_fill(~vis[:, None, None, :], -math.inf), -1)
        most = (p * vs[None, :, None, :]).amax(-1)
        codes = (v.abs() / vs[..., None]).sum(1)
        tol[row:row + n] += (2.0 ** -32 * most[..., None] * codes[None, :, None, :]).reshape(n, Hq, D)
        row += n
    return want, tol


# Exponents of the value scales of a sequence's blocks, by block: the largest is 2^119, as
# 448 x 2^120 is past float32.
MIXES = {
    "any": lambda rng, n: rng.integers(-64, 120, n),
    "least": lambda rng, n: np.full(n, -64),
    "largest": lambda rng, n: np.full(n, 119),
    "large and small": lambda rng, n: rng.choice([-64, 119], n),
    "small first": lambda rng, n: np.where(np.arange(n) < (n + 1) // 2, -64, 119),
    "small last": lambda rng, n: np.where(np.arange(n) < (n + 1) // 2, 119, -64),
    "far and not so far": lambda rng, n: rng.choice([30, -20, -49, -51, -64], n),
    "ordinary and one small": lambda rng, n: np.where(np.arange(n) == n // 3, -64, rng.integers(-9, 20, n)),
}


def _cache(mix, lens, Hkv, D, bs, zeros=False):
    c = ref.Cache(lens, Hkv, D, bs, seed=len(lens) + D + bs)
    rng = np.random.default_rng(3)
    for b, L in enumerate(lens):
        n = -(-L // bs)
        for h in range(Hkv):
            c.scales[1][c.tables[b, :n], h] = np.exp2(MIXES[mix](rng, n).astype(np.float64)).astype(np.float32)
    if zeros:   # the values of the smallest scales are zeros, as the write has them
        low = (c.scales[1] == np.float32(2.0 ** -64))[:, :, None, None] & ~np.isnan(ref.VALUES[c.codes[1]])
        c.codes[1][low] = 0
    c.upload()
    return c


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("sigma", [1.0, 12.0])
@pytest.mark.parametrize("Hq,Hkv,D,bs", [(8, 2, 128, 16), (5, 5, 64, 32), (16, 1, 128, 32), (24, 2, 64, 16)])
def test_decode(mix, sigma, Hq, Hkv, D, bs, plan):
    """The last: sequences cut over many warps and joined by the merge."""
    for lens in ([1, 40, 333], [5000, 64]):
        for zeros in (False, True):
            c = _cache(mix, lens, Hkv, D, bs, zeros)
            q = _q(len(lens), Hq, D, 5, sigma)
            want, tol = _attention(c, q, [1] * len(lens))
            ref.check(_decode(c, q, plan), want, tol)
            ref.check(_decode(c, q, plan, torch.bfloat16), want, tol)


@pytest.mark.parametrize("mix", MIXES)
@pytest.mark.parametrize("sigma", [1.0, 12.0])
@pytest.mark.parametrize("Hq,Hkv,bs", [(8, 2, 16), (16, 1, 32)])
def test_prefill(kernel, mix, sigma, Hq, Hkv, bs, plan):
    """Few queries, many, and a long sequence whose keys are cut over several blocks."""
    for lens, new in (([300, 77, 16], [2, 1, 2]), ([300, 77, 700], [40, 3, 200]), ([9000], [40])):
        for zeros in (False, True):
            c = _cache(mix, lens, Hkv, 128, bs, zeros)
            q = _q(sum(new), Hq, 128, 6, sigma)
            want, tol = _attention(c, q, new)
            ref.check(_prefill(c, q, new, plan), want, tol)


def test_zero_blocks_beside_large_values(plan):
    """Equal scores: half of the tokens zeros, half 2^70, the mean between them."""
    c = ref.Cache([64], 1, 128, 16, seed=7)
    blk = c.tables[0, :4]
    c.codes[0][blk] = 0
    c.codes[1][blk[:2]], c.codes[1][blk[2:]] = 0, ref.nearest(256.0)
    c.scales[1][blk[:2]], c.scales[1][blk[2:]] = 2.0 ** -64, 2.0 ** 62
    c.upload()
    q = _q(40, 4, 128, 8)
    for out in (_decode(c, q[:1], plan), _prefill(c, q, [40], plan)[-1]):
        assert bool(((out.double() / 2.0 ** 69 - 1).abs() < 2.0 ** -11).all())


@pytest.mark.parametrize("power", [-60, -100, -115, -125, -131])
@pytest.mark.parametrize("D", [64, 128])
def test_tiny_queries(kernel, power, D, plan):
    """Query rows of any size keep their bits (below 2^-126 bf16's own subnormal ones) where large keys make
    scores of them."""
    k = min(-power - 7.0, 119.0)
    lens, new = [300, 77, 700], [40, 3, 100]
    c = ref.Cache(lens, 2, D, 16, seed=13, k_exp=(k - 1, k))
    q = (_q(sum(new), 8, D, 14).float() * 2.0 ** power).to(torch.bfloat16)
    assert float(q.abs().max()) > 0
    want, tol = ref.attention(c, q[:3], [1] * 3, D ** -0.5)
    ref.check(_decode(c, q[:3], plan), want, tol)
    if D == 128:
        for n in (new, [2, 1, 2]):
            want, tol = ref.attention(c, q[:sum(n)], n, D ** -0.5)
            ref.check(_prefill(c, q[:sum(n)], n, plan), want, tol)


BAD = [(1, x) for x in (2.0 ** -65, 1e-37, 1e-40, 0.0, -1.0, 2.0 ** 121, math.inf, math.nan)] + \
      [(0, x) for x in (0.0, -1.0, math.inf, math.nan)]


@pytest.mark.parametrize("which,scale", BAD)
def test_scales_that_are_none_show(kernel, which, scale, plan):
    """A block with such a scale makes the rows that see it NaN, and those of other sequences and heads
    are right."""
    for lens, new in (([300, 90, 40], [2, 1, 2]), ([300, 90, 40], [100, 40, 1]), ([6000, 90], [40, 1])):
        c = ref.Cache(lens, 2, 128, 16, seed=9)
        q = _q(sum(new), 8, 128, 10)
        want, tol = ref.attention(c, q, new, 128 ** -0.5)
        dwant, dtol = ref.attention(c, q[:len(lens)], [1] * len(lens), 128 ** -0.5)
        c.scales[which][c.tables[0, 7], 1] = np.float32(scale)
        c.upload()
        out = _prefill(c, q, new, plan)
        assert bool(torch.isnan(out[:new[0], 4:]).all())
        ref.check(out[new[0]:], want[new[0]:], tol[new[0]:])
        ref.check(out[:, :4], want[:, :4], tol[:, :4])
        out = _decode(c, q[:len(lens)], plan)
        assert bool(torch.isnan(out[0, 4:]).all())
        ref.check(out[1:], dwant[1:], dtol[1:])
        ref.check(out[:, :4], dwant[:, :4], dtol[:, :4])
