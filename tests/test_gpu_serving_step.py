"""GPU: the serving-step calls together, as an engine runs them for a layer with
per-head norms, scaled rotary positions and a sliding window: step maps ->
norm, rotation and cache write -> windowed attention, for prompts, mixed steps
and single tokens, with blocks behind the window given back and handed out
again. The outputs are compared with a 64-bit model that keeps the whole
history of every request and knows neither blocks nor tables."""

import numpy as np
import pytest
import torch

import paged_kv_cache_202_gb300 as pa
from step_reference import norm_rope
from window_reference import tokens_seen, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    import __graft_entry__
    __graft_entry__.build()


I32 = torch.int32


def bf(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def expect(q, ks, vs, p, scale, W, S, D, prefill):
    """Attention of one query over the request's kept keys and values, and how far off it may be."""
    t = tokens_seen(p, W, S)
    Hkv = ks.shape[1]
    k, v = ks[t], vs[t]
    qg = q.reshape(Hkv, -1, D)
    s = np.einsum("hgd,nhd->hgn", qg, k) * scale
    mag = (np.einsum("hgd,nhd->hgn", np.abs(qg), np.abs(k)) * scale).max(-1)
    w = np.exp(s - s.max(-1, keepdims=True))
    w /= w.sum(-1, keepdims=True)
    out = np.einsum("hgn,nhd->hgd", w, v).reshape(-1, D)
    wv = np.einsum("hgn,nhd->hgd", w, np.abs(v)).reshape(-1, D)
    return out, tolerance(out, wv, mag.reshape(-1, 1), D, 8 if prefill else 16, True)


@pytest.mark.parametrize("bs", [16, 32])
@pytest.mark.parametrize("layout", [pa.PA_ROPE_HALF, pa.PA_ROPE_INTERLEAVED])
def test_steps_of_a_layer(bs, layout):
    B, Hq, Hkv, D, W, S, NB, MB = 5, 8, 2, 128, 40, 5, 40, 16
    rng = np.random.default_rng(bs + layout)
    rope = pa.Rope(64, layout=layout, scaling=pa.PA_ROPE_YARN, factor=4.0, orig_len=64)
    qw, kw = bf(1 + 0.2 * rng.standard_normal(D)), bf(1 + 0.2 * rng.standard_normal(D))
    kp = torch.full((NB, Hkv, bs, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    vp = torch.full_like(kp, float("nan"))
    free = list(rng.permutation(NB))
    table = np.full((B, MB), -1, dtype=np.int32)
    cache = np.zeros(B, dtype=np.int32)
    hist_k, hist_v = [np.zeros((0, Hkv, D)) for _ in range(B)], [np.zeros((0, Hkv, D)) for _ in range(B)]
    d = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda()  # noqa: E731
    steps = [[70, 33, 1, 90, 16], [1, 1, 40, 1, 0], [1] * 5, [1] * 5, [3, 20, 1, 5, 60], [1] * 5, [1] * 5]
    scale = D ** -0.5
    with pa.Plan() as plan:
        for step, new in enumerate(steps):
            new = np.array(new, dtype=np.int32)
            T = int(new.sum())
            rows = T + 3                      # a batch padded past its rows
            x = bf(rng.standard_normal((rows, Hq + 2 * Hkv, D))).cuda()
            x[T:] = float("nan")
            q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
            dt = d(table)
            o = {n: torch.zeros(m, dtype=I32, device="cuda") for n, m in (("seq", B), ("start", B + 1), ("pos", rows), ("left", 1))}
            slots = torch.zeros(rows, dtype=torch.int64, device="cuda")
            err = torch.zeros(1, dtype=I32, device="cuda")
            q_out = torch.full((rows, Hq, D), 7.5, dtype=torch.bfloat16, device="cuda")
            pa.pa_step_maps(d(cache), d(new), d(np.array(free, dtype=np.int32)), torch.tensor([len(free)], dtype=I32, device="cuda"),
                            dt, bs, NB, MB * bs, o["seq"], o["start"], o["pos"], slots, o["left"], device_error=err)
            pa.pa_qk_rope_append(q, k, v, o["pos"], slots, rope, kp, vp, q_out, q_weight=qw.cuda(),
                                 k_weight=kw.cuda(), eps=1e-5, device_error=err)
            out = torch.full((T, Hq, D), 7.5, dtype=torch.bfloat16, device="cuda")
            single = bool((new == 1).all())
            if single:
                pa.pa_decode_window(q_out[:T], kp, vp, dt, o["seq"], scale, W, S, out, MB * bs, plan)
            else:
                pa.pa_prefill_window(q_out[:T], o["start"], kp, vp, dt, o["seq"], scale, W, S, out,
                                     int(new.max()), MB * bs, plan)
            assert pa.pa_last_device_error(plan) == 0 and int(err) == 0
            assert bool((q_out[T:] == 7.5).all())
            # The model: keys and values as the pools must hold them (the
            # cache write is checked by its own tests; here its rows are read
            # back through the new tables).
            table = dt.cpu().numpy()
            free = free[:int(o["left"])]
            pos, hx = o["pos"].cpu().numpy()[:T], x[:T].double().cpu().numpy()
            qr, qb = norm_rope(hx[:, :Hq], pos, np.array(rope.inv_freq), rope.amplitude, 64, layout, qw.double().numpy(), 1e-5)
            kr, kb = norm_rope(hx[:, Hq:Hq + Hkv], pos, np.array(rope.inv_freq), rope.amplitude, 64, layout, kw.double().numpy(), 1e-5)
            got_q = q_out[:T].double().cpu().numpy()
            assert (np.abs(got_q - qr) <= qb * 1.01 + 2.0 ** -8 * np.abs(qr)).all()
            blk = slots[:T] // bs
            got_k = kp[blk, :, slots[:T] % bs].double().cpu().numpy()
            assert (np.abs(got_k - kr) <= kb * 1.01 + 2.0 ** -8 * np.abs(kr)).all()
            t, got = 0, out.double().cpu().numpy()
            for b in range(B):
                n = int(new[b])
                hist_k[b] = np.concatenate([hist_k[b], got_k[t:t + n]])
                hist_v[b] = np.concatenate([hist_v[b], hx[t:t + n, Hq + Hkv:]])
                for i in range(n):
                    ref, tol = expect(got_q[t + i], hist_k[b], hist_v[b], int(cache[b]) + i, scale, W, S, D, not single)
                    assert (np.abs(got[t + i] - ref) <= tol).all(), (step, b, i)
                t += n
            cache = cache + new
            # Blocks wholly behind the window of the next query go back, and
            # whatever they hold is no one's any more.
            for b in range(B):
                for p in range(-(-S // bs), max(0, int(cache[b]) + 1 - W) // bs):
                    if table[b, p] >= 0:
                        free.append(int(table[b, p]))
                        kp[table[b, p]] = float("nan")
                        vp[table[b, p]] = float("inf")
                        table[b, p] = -1
    assert len(free) + int((table >= 0).sum()) == NB
