"""Attention mass and eviction on the GPU against the float64 oracle, and the
two with attention as a serving loop uses them.

Bar for mass: relative 1e-4 of each sum of positive weights.  A weight is
2^x with x from a dot product of 64 exact bf16 products summed in fp32; even if
every addition truncates (2^-23) its error is at most 64 * 2^-23 * scale *
sum|q k|, with sum|q k| below 80 for these normal inputs 7.7e-5 in the
exponent; the hardware exponential adds 2^-22, the sum of at most 700 * 16
weights in a few chains (order below 2^-24 * 700) 4e-5 in the worst case and
far less in practice.  The pieces do not reach their worst cases together.
Eviction copies: it is compared bit for bit.
"""

import numpy as np
import pytest
import torch

import gqa_attention_learned_gb300 as sa
from bounded_inputs import DEV, Paged, bf16, np64
from oracle import bounded
from tolerances import assert_lse_close, assert_out_close

pytestmark = pytest.mark.gpu
RTOL = 1e-4


def _mass_close(got, want):
    np.testing.assert_allclose(np64(got), want, rtol=RTOL, atol=1e-30)


# -------------------------------------------------------------------- mass
@pytest.mark.parametrize("heads", [(64, 8), (4, 1), (8, 8), (10, 2), (32, 2), (24, 1)])
def test_decode_mass(heads):
    lens = [0, 1, 15, 16, 17, 130, 700, 1025, 2100]
    c = Paged(lens, *heads)
    q = bf16(c.rng, len(lens), heads[0], 64)
    _, lse = sa.decode(q.to(DEV), *c.paged(), c.sinks.to(DEV), c.scale, c.max_kv)
    stride = c.max_kv + 5
    start = torch.from_numpy(c.rng.random((len(lens), heads[1], stride)).astype(np.float32))
    start[0] = 0
    mass = start.to(DEV)
    k, _, table, kv = c.paged()
    ret = sa.decode_mass(q.to(DEV), k, table, kv, lse, c.scale, c.max_kv, mass)
    assert ret is mass
    want = np64(start)
    for b, n in enumerate(lens):
        want[b, :, :n] += bounded.mass_rows(np64(q[b:b + 1]), np64(c.k[b]), [n - 1], np64(lse[b:b + 1]), c.scale)
        assert torch.equal(mass[b, :, n:].cpu(), start[b, :, n:])
    _mass_close(mass, want)


@pytest.mark.parametrize("heads", [(64, 8), (4, 1), (8, 8), (10, 2), (32, 2), (128, 1)])
@pytest.mark.parametrize("q_lens,prefix", [([1, 17, 140], [0, 0, 0]), ([1, 5, 33, 2], [0, 400, 259, 128]),
                                           ([64, 3], [130, 700])])
def test_prefill_mass(heads, q_lens, prefix):
    c = Paged([a + b for a, b in zip(q_lens, prefix)], *heads, seed=7)
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    q = bf16(c.rng, cu[-1], heads[0], 64)
    cu_gpu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    _, lse = sa.prefill_paged(q.to(DEV), cu_gpu, *c.paged(), c.sinks.to(DEV), c.scale, max(q_lens), c.max_kv)
    k, _, table, kv = c.paged()
    mass = torch.zeros(len(q_lens), heads[1], c.max_kv + 3, device=DEV)
    want = np.zeros(mass.shape)
    for b, n in enumerate(c.lens):
        rows = slice(cu[b], cu[b + 1])
        want[b, :, :n] = bounded.mass_rows(np64(q[rows]), np64(c.k[b]), range(prefix[b], n), np64(lse[rows]), c.scale)
    for times in (1, 2):                                  # a second call adds the same again
        sa.prefill_mass(q.to(DEV), cu_gpu, k, table, kv, lse, c.scale, max(q_lens), c.max_kv, mass)
        _mass_close(mass, times * want)


@pytest.mark.parametrize("heads,lens", [((8, 1), [1111, 2300, 40]), ((32, 1), [700, 9, 1500]), ((4, 1), [2205])])
def test_prefill_mass_of_long_prompts(heads, lens):
    # prompts long enough that a cluster of CTAs shares each key's rows
    hq, hkv = heads
    c = Paged(lens, hq, hkv, seed=3)
    cu = np.concatenate([[0], np.cumsum(lens)])
    q = bf16(c.rng, cu[-1], hq, 64)
    k, v, table, kv = c.paged()
    cu_gpu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    _, lse = sa.prefill_paged(q.to(DEV), cu_gpu, k, v, table, kv, c.sinks.to(DEV), c.scale, max(lens), c.max_kv)
    bad = [b for b, n in enumerate(lens) if n == 40]
    for b in bad:
        kv[b] = -7                                        # out of range: among the long ones
    mass = torch.zeros(len(lens), hkv, c.max_kv, device=DEV)
    sa.prefill_mass(q.to(DEV), cu_gpu, k, table, kv, lse, c.scale, max(lens), c.max_kv, mass)
    for b, n in enumerate(lens):
        if b in bad:
            assert torch.isnan(mass[b]).all()
            continue
        s = np.einsum("ihd,jd->hij", np64(q[cu[b]:cu[b + 1]]), np64(c.k[b][:, 0])) * c.scale
        w = np.exp(s - np64(lse[cu[b]:cu[b + 1]]).T[:, :, None])
        w[:, np.arange(n)[:, None] < np.arange(n)] = 0
        _mass_close(mass[b, 0, :n], w.sum((0, 1)))
        assert (mass[b, :, n:] == 0).all()


def test_prefill_mass_of_many_prompts():
    # enough (request, KV head) units that none is shared
    lens = [300 + 7 * (b % 5) for b in range(60)]
    c = Paged(lens, 64, 8, seed=4)
    cu = np.concatenate([[0], np.cumsum(lens)])
    q = bf16(c.rng, cu[-1], 64, 64)
    k, v, table, kv = c.paged()
    cu_gpu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    _, lse = sa.prefill_paged(q.to(DEV), cu_gpu, k, v, table, kv, c.sinks.to(DEV), c.scale, max(lens), c.max_kv)
    mass = torch.zeros(60, 8, c.max_kv, device=DEV)
    sa.prefill_mass(q.to(DEV), cu_gpu, k, table, kv, lse, c.scale, max(lens), c.max_kv, mass)
    for b in (0, 13, 59):
        n = lens[b]
        s = np.einsum("ighd,jgd->ghij", np64(q[cu[b]:cu[b + 1]]).reshape(n, 8, 8, 64), np64(c.k[b])) * c.scale
        w = np.exp(s - np64(lse[cu[b]:cu[b + 1]]).T.reshape(8, 8, n, 1))
        w[..., np.arange(n)[:, None] < np.arange(n)] = 0
        _mass_close(mass[b, :, :n], w.sum((1, 2)))


def test_mass_is_the_same_bits_every_time_and_in_a_graph():
    c = Paged([700, 333], 64, 8)
    q, q1 = bf16(c.rng, 300, 64, 64).to(DEV), bf16(c.rng, 2, 64, 64).to(DEV)
    cu = torch.tensor([0, 200, 300], dtype=torch.int32, device=DEV)
    k, v, table, kv = c.paged()
    sinks = c.sinks.to(DEV)

    def run():
        mass = torch.zeros(2, 8, 700, device=DEV)
        _, lse = sa.prefill_paged(q, cu, k, v, table, kv, sinks, c.scale, 200, 700)
        sa.prefill_mass(q, cu, k, table, kv, lse, c.scale, 200, 700, mass)
        _, lse = sa.decode(q1, k, v, table, kv, sinks, c.scale, 700, num_splits=1)
        return sa.decode_mass(q1, k, table, kv, lse, c.scale, 700, mass)

    want = run()
    for _ in range(3):
        assert torch.equal(run(), want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = run()
    for _ in range(2):
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want)


def test_mass_of_rows_without_weight_and_of_bad_requests():
    c = Paged([40, 40, 40, 40], 4, 1)
    q = bf16(c.rng, 4, 4, 64).to(DEV)
    k, v, table, kv = c.paged()
    _, lse = sa.decode(q, k, v, table, kv, c.sinks.to(DEV), c.scale, 40)
    lse[0] = -np.inf                                      # adds nothing
    kv[1] = 41                                            # past the bound: the whole row
    table[2, 1] = c.pages                                 # one page: its keys
    cu = torch.arange(5, dtype=torch.int32, device=DEV)
    for prefill in (False, True):
        mass = torch.ones(4, 1, 48, device=DEV)
        if prefill:
            sa.prefill_mass(q, cu, k, table, kv, lse, c.scale, 1, 40, mass)
        else:
            sa.decode_mass(q, k, table, kv, lse, c.scale, 40, mass)
        assert (mass[0] == 1).all()
        assert torch.isnan(mass[1]).all()
        assert torch.isnan(mass[2, 0, 16:32]).all()
        assert torch.isfinite(mass[2, 0, :16]).all() and torch.isfinite(mass[2, 0, 32:]).all()
        assert torch.isfinite(mass[3]).all() and (mass[3, 0, 40:] == 1).all()


def test_mass_with_zero_and_negative_scale():
    c = Paged([150], 4, 1)
    q = bf16(c.rng, 9, 4, 64)
    cu = torch.tensor([0, 9], dtype=torch.int32, device=DEV)
    k, _, table, kv = c.paged()
    for scale in (0.0, -0.125):
        _, lse = bounded.window_rows(np64(q), np64(c.k[0]), np64(c.v[0]), range(141, 150), np64(c.sinks), scale, 150)
        lse32 = torch.from_numpy(lse.astype(np.float32))
        want = bounded.mass_rows(np64(q), np64(c.k[0]), range(141, 150), np64(lse32), scale)
        mass = torch.zeros(1, 1, 150, device=DEV)
        sa.prefill_mass(q.to(DEV), cu, k, table, kv, lse32.to(DEV), scale, 9, 150, mass)
        _mass_close(mass[0], want)


# ---------------------------------------------------------------- eviction
def _evict_ref(c, mass, budget, first, recent):
    """kept [B][Hkv] lists."""
    return [[bounded.keep(np64(mass[b, g]), n, budget, first, recent) for g in range(c.hkv)]
            for b, n in enumerate(c.lens)]


def _check(c, kept_ref, kept, new_lens, budget, dst_table, k_cache, v_cache, old_k, old_v,
           mass_out, old_mass, dst_mass_before):
    want_k, want_v, want_m = old_k.clone(), old_v.clone(), dst_mass_before.clone()
    for b, n in enumerate(c.lens):
        count = min(n, budget)
        assert int(new_lens[b]) == count
        for g in range(c.hkv):
            row = kept_ref[b][g]
            assert kept[b, g, :count].tolist() == row
            assert (kept[b, g, count:] == -1).all()
            for r, j in enumerate(row):
                s, d = int(c.table[b, j // 16]), int(dst_table[b, r // 16])
                want_k[d, g, r % 16] = old_k[s, g, j % 16]
                want_v[d, g, r % 16] = old_v[s, g, j % 16]
                want_m[b, g, r] = old_mass[b, g, j]
            want_m[b, g, count:min(n, want_m.shape[2])] = 0
    assert torch.equal(k_cache.cpu().view(torch.int16), want_k.view(torch.int16))
    assert torch.equal(v_cache.cpu().view(torch.int16), want_v.view(torch.int16))
    assert torch.equal(mass_out.cpu().view(torch.int32), want_m.view(torch.int32))


def _weights(rng, kind, *shape):
    if kind == "ties":
        return rng.integers(0, 4, shape).astype(np.float32)
    m = np.exp(2 * rng.standard_normal(shape) - 3).astype(np.float32)
    if kind == "odd":
        m[..., ::7] = np.nan
        m[..., 3::11] = np.inf
        m[..., 5::13] = -0.0
        m[..., 6::17] = -np.inf
        m[..., 8::19] = 1e-42
    return m


@pytest.mark.parametrize("kind", ["normal", "ties", "odd"])
@pytest.mark.parametrize("budget,first,recent", [(1, 0, 0), (1, 1, 0), (16, 4, 5), (17, 0, 17), (33, 16, 16),
                                                 (100, 0, 1), (256, 4, 64), (5000, 4, 7)])
@pytest.mark.parametrize("in_place", [True, False])
def test_evict(kind, budget, first, recent, in_place):
    lens = [0, 1, 16, 17, 100, 257, 1500]
    per = -(-min(budget, 1500) // 16)
    c = Paged(lens, 2, 2, seed=budget, spare=per * len(lens) + 2)
    stride = 1500 + 9
    mass = torch.from_numpy(_weights(c.rng, kind, len(lens), 2, stride))
    ref = _evict_ref(c, mass, budget, first, recent)
    k, v, table, kv = c.paged()
    m = mass.to(DEV)
    kw = dict(first_tokens=first, recent=recent)
    dst, dst_mass, before = c.table, m, mass
    if not in_place:
        dst = c.free[:per * len(lens)].view(len(lens), per).contiguous()
        before = torch.from_numpy(c.rng.random((len(lens), 2, min(budget, 1500) + 3)).astype(np.float32))
        dst_mass = before.to(DEV)
        kw.update(dst_page_table=dst.to(DEV), dst_mass=dst_mass)
    new, kept = sa.evict(k, v, table, kv, m, budget, 1500, **kw)
    torch.cuda.synchronize()
    _check(c, ref, kept.cpu(), new.cpu(), budget, dst, k, v, c.k_cache, c.v_cache, dst_mass, mass, before)
    if not in_place:
        assert torch.equal(m.cpu().view(torch.int32), mass.view(torch.int32))


@pytest.mark.parametrize("in_place", [True, False])
def test_evict_long(in_place):
    # several tiles of everything, a length that fills no tile
    c = Paged([20011, 4096, 9], 1, 1, seed=5, spare=3 * 257)
    mass = torch.from_numpy(_weights(c.rng, "normal", 3, 1, 20011))
    ref = _evict_ref(c, mass, 4099, 4, 100)
    k, v, table, kv = c.paged()
    m = mass.to(DEV)
    dst, dst_mass, before, kw = c.table, m, mass, {}
    if not in_place:
        dst = c.free[:3 * 257].view(3, 257).contiguous()
        before = torch.zeros(3, 1, 4099)
        dst_mass = before.to(DEV)
        kw = dict(dst_page_table=dst.to(DEV), dst_mass=dst_mass)
    new, kept = sa.evict(k, v, table, kv, m, 4099, 20011, first_tokens=4, recent=100, **kw)
    torch.cuda.synchronize()
    _check(c, ref, kept.cpu(), new.cpu(), 4099, dst, k, v, c.k_cache, c.v_cache, dst_mass, mass, before)


def test_evict_one_long_row_among_many():
    # so many rows that none is shared, one of them longer than a CTA holds
    lens = [30001] + [5] * 160
    c = Paged(lens, 1, 1, seed=6)
    for kind in ("normal", "ties"):
        mass = torch.from_numpy(_weights(c.rng, kind, len(lens), 1, 30001))
        ref = _evict_ref(c, mass, 4099, 4, 100)
        k, v, table, kv = c.paged()
        m = mass.to(DEV)
        new, kept = sa.evict(k, v, table, kv, m, 4099, 30001, first_tokens=4, recent=100)
        torch.cuda.synchronize()
        _check(c, ref, kept.cpu(), new.cpu(), 4099, c.table, k, v, c.k_cache, c.v_cache, m, mass, mass)


def test_evict_leaves_bad_requests_alone():
    c = Paged([100, 100, 100, 100, 100], 1, 1)
    mass = torch.from_numpy(_weights(c.rng, "normal", 5, 1, 100)).to(DEV)
    k, v, table, kv = c.paged()
    kv[0] = -1
    kv[1] = 101                                           # past the bound
    table[2, 6] = c.pages                                 # a page that holds a key
    dst = table.clone()
    dst[2:, :] = table[2:, :]
    dst[3, 1] = -7                                        # a destination outside the pool
    before = (k.clone(), v.clone(), mass.clone())
    new, kept = sa.evict(k, v, table, kv, mass, 32, 100, dst_page_table=dst)
    torch.cuda.synchronize()
    assert new.tolist() == [-1, -1, -1, -1, 32]
    assert (kept[:4] == -1).all()
    ids = [int(i) for i in c.table[:4].flatten() if 0 <= i < c.pages]
    for now, was in zip((k, v), before):
        assert torch.equal(now[ids].view(torch.int16), was[ids].view(torch.int16))
    assert torch.equal(mass[:4], before[2][:4])


def test_nothing_to_weigh_or_evict():
    c = Paged([0, 0], 4, 1)
    k, v, table, kv = c.paged()
    q = bf16(c.rng, 2, 4, 64).to(DEV)
    lse = torch.zeros(2, 4, device=DEV)
    mass = torch.zeros(2, 1, 0, device=DEV)
    sa.decode_mass(q, k, table, kv, lse, c.scale, 0, mass)
    sa.prefill_mass(q, torch.tensor([0, 1, 2], dtype=torch.int32, device=DEV), k, table, kv, lse, c.scale, 1, 0, mass)
    new, kept = sa.evict(k, v, table, kv, mass, 8, 0)
    assert new.tolist() == [0, 0] and (kept == -1).all()


def test_evict_from_a_graph_and_on_two_streams():
    # a captured eviction replays on new weights and lengths; two evictions of
    # different requests run side by side
    cs = [Paged([900, 40, 333], 2, 2, seed=s) for s in (1, 2)]
    sides = [torch.cuda.Stream() for _ in cs]
    runs = []
    for c, side in zip(cs, sides):
        k, v, table, kv = c.paged()
        mass = torch.zeros(3, 2, 900, device=DEV)
        new, kept = torch.empty_like(kv), torch.empty(3, 2, 100, dtype=torch.int32, device=DEV)

        def call(k=k, v=v, table=table, kv=kv, mass=mass, new=new, kept=kept):
            sa.evict(k, v, table, kv, mass, 100, 900, first_tokens=3, recent=20, new_kv_lens=new, kept=kept)

        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            call()                                        # weights 0: ties, then put everything back
        side.synchronize()
        k.copy_(c.k_cache), v.copy_(c.v_cache)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
        runs.append((c, g, side, k, v, mass, new, kept))
    for rep in range(2):
        weights = []
        for c, g, side, k, v, mass, new, kept in runs:
            w = torch.from_numpy(_weights(c.rng, "normal", 3, 2, 900))
            weights.append(w)
            k.copy_(c.k_cache), v.copy_(c.v_cache), mass.copy_(w)
        torch.cuda.synchronize()
        for c, g, side, *_ in runs:
            with torch.cuda.stream(side):
                g.replay()
        torch.cuda.synchronize()
        for w, (c, g, side, k, v, mass, new, kept) in zip(weights, runs):
            _check(c, _evict_ref(c, w, 100, 3, 20), kept.cpu(), new.cpu(), 100, c.table, k, v, c.k_cache,
                   c.v_cache, mass, w, w)


# ------------------------------------------------------------ all together
def test_a_serving_loop_with_eviction():
    # prompt -> its weights -> cut to a budget -> new tokens that attend to
    # what was kept, add their weight and are cut again
    lens, hq, hkv, budget = [300, 150, 40], 16, 2, 64
    c = Paged([n + 40 for n in lens], hq, hkv)            # room for new tokens
    k, v, table, _ = c.paged()
    kv = torch.tensor(lens, dtype=torch.int32, device=DEV)
    sinks, cap = c.sinks.to(DEV), 340
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device=DEV)
    q = bf16(c.rng, sum(lens), hq, 64)
    _, lse = sa.prefill_paged(q.to(DEV), cu, k, v, table, kv, sinks, c.scale, 300, cap)
    mass = torch.zeros(3, hkv, cap, device=DEV)
    sa.prefill_mass(q.to(DEV), cu, k, table, kv, lse, c.scale, 300, cap, mass)

    held = [[np64(c.k[b][:n]), np64(c.v[b][:n])] for b, n in enumerate(lens)]   # [n, Hkv, 64] each

    def cut(kv):
        n_before = kv.tolist()
        new, kept = sa.evict(k, v, table, kv, mass, budget, cap, first_tokens=2, recent=8)
        for b, n in enumerate(n_before):
            count = min(n, budget)
            idx = kept[b, :, :count].cpu().numpy()
            for t in range(2):
                held[b][t] = np.stack([held[b][t][idx[g], g] for g in range(hkv)], 1)
        return new

    kv = cut(kv)
    for step in range(20):
        # one new token each: its key and value go to the next slot
        new_k, new_v, q1 = (bf16(c.rng, 3, h, 64) for h in (hkv, hkv, hq))
        pos = kv.long()
        page = table.long().gather(1, (pos // 16)[:, None])[:, 0]
        k[page, :, pos % 16] = new_k.to(DEV)
        v[page, :, pos % 16] = new_v.to(DEV)
        kv = kv + 1
        for b in range(3):
            for t, x in enumerate((new_k, new_v)):
                held[b][t] = np.concatenate([held[b][t], np64(x[b:b + 1])])
        out, lse = sa.decode(q1.to(DEV), k, v, table, kv, sinks, c.scale, cap)
        before = mass.clone()
        sa.decode_mass(q1.to(DEV), k, table, kv, lse, c.scale, cap, mass)
        for b in range(3):
            n = held[b][0].shape[0]
            ro, rl = bounded.window_rows(np64(q1[b:b + 1]), held[b][0], held[b][1], [n - 1], np64(c.sinks),
                                         c.scale, n)
            assert_out_close(out[b:b + 1], ro)
            assert_lse_close(lse[b:b + 1], rl)
            add = bounded.mass_rows(np64(q1[b:b + 1]), held[b][0], [n - 1], np64(lse[b:b + 1]), c.scale)
            np.testing.assert_allclose(np64(mass[b, :, :n]), np64(before[b, :, :n]) + add, rtol=RTOL, atol=1e-30)
            assert (mass[b, :, n:] == 0).all()            # evicted places start from nothing
        if step % 6 == 5:
            kv = cut(kv)


def test_a_decode_step_of_both_kinds_of_layer_chained_programmatically():
    # windowed layer, full layer with weights, eviction, decode again: every
    # launch may start under the one before it
    c = Paged([500, 260, 90, 33], 64, 8, spare=40)
    sinks, q = c.sinks.to(DEV), bf16(c.rng, 4, 64, 64).to(DEV)

    def step(programmatic):
        k, v, table, kv = c.paged()
        mass = torch.zeros(4, 8, 500, device=DEV)
        a, _ = sa.decode_window(q, k, v, table, kv, sinks, c.scale, 500, 128, 4, programmatic=programmatic)
        b, lse = sa.decode(a, k, v, table, kv, sinks, c.scale, 500, programmatic=programmatic)
        sa.decode_mass(a, k, table, kv, lse, c.scale, 500, mass)
        new, kept = sa.evict(k, v, table, kv, mass, 64, 500, first_tokens=4, recent=16)
        # evict wrote the lengths just before: this one has to be an ordinary launch
        o, l = sa.decode(b, k, v, table, new, sinks, c.scale, 64, programmatic=False)
        torch.cuda.synchronize()
        return a, b, lse, mass, new, kept, o, l

    for x, y in zip(step(False), step(True)):
        assert torch.equal(x, y)


# ------------------------------------------------------ many requests, few rows
def test_prefill_mass_of_many_requests_with_few_rows():
    # a decode batch with draft tokens: more requests than a warp looks up at
    # once, some without rows, one refused, several key pairs each, so that a
    # CTA's share crosses requests and heads
    rng = np.random.default_rng(11)
    q_lens = [int(n) for n in rng.integers(0, 5, 75)]
    q_lens[31], q_lens[32], q_lens[40] = 0, 0, 3
    prefix = [int(n) for n in rng.integers(0, 900, 75)]
    prefix[7], prefix[64] = 1500, 1031
    c = Paged([a + b for a, b in zip(q_lens, prefix)], 16, 2, seed=12)
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    q = bf16(c.rng, cu[-1], 16, 64)
    cu_gpu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    k, v, table, kv = c.paged()
    _, lse = sa.prefill_paged(q.to(DEV), cu_gpu, k, v, table, kv, c.sinks.to(DEV), c.scale, 4, c.max_kv)
    kv[40] = -3
    mass = torch.zeros(75, 2, c.max_kv, device=DEV)
    for times in (1, 2):
        sa.prefill_mass(q.to(DEV), cu_gpu, k, table, kv, lse, c.scale, 4, c.max_kv, mass)
        for b, n in enumerate(c.lens):
            if b == 40:
                assert torch.isnan(mass[b]).all()
                continue
            rows = slice(cu[b], cu[b + 1])
            want = bounded.mass_rows(np64(q[rows]), np64(c.k[b]), range(prefix[b], n), np64(lse[rows]), c.scale)
            _mass_close(mass[b, :, :n], times * want)
            assert (mass[b, :, n:] == 0).all()


@pytest.mark.parametrize("first,recent", [(100, 900), (0, 1000), (1000, 0)])
def test_evict_long_rows_by_place_alone(first, recent):
    # the first and the recent keys fill the budget: no weight is looked at, and
    # the CTAs that share a row meet only to number what they keep
    c = Paged([30000, 999, 16001, 1001], 2, 2, seed=13)
    mass = torch.from_numpy(_weights(c.rng, "odd", 4, 2, 30000))
    ref = _evict_ref(c, mass, 1000, first, recent)
    for _ in range(3):
        k, v, table, kv = c.paged()
        m = mass.to(DEV)
        new, kept = sa.evict(k, v, table, kv, m, 1000, 30000, first_tokens=first, recent=recent)
        torch.cuda.synchronize()
        _check(c, ref, kept.cpu(), new.cpu(), 1000, c.table, k, v, c.k_cache, c.v_cache, m, mass, mass)


# --------------------------------------------------------- what a row does not see
@pytest.mark.parametrize("tokens,row", [(200, 100), (200, 130), (2300, 777)])
def test_a_row_without_an_lse_spoils_only_the_keys_that_it_sees(tokens, row):
    c = Paged([tokens], 8, 1, seed=14)
    q = bf16(c.rng, tokens, 8, 64)
    k, v, table, kv = c.paged()
    cu = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    _, lse = sa.prefill_paged(q.to(DEV), cu, k, v, table, kv, c.sinks.to(DEV), c.scale, tokens, tokens)
    want = torch.zeros(1, 1, tokens, device=DEV)
    sa.prefill_mass(q.to(DEV), cu, k, table, kv, lse, c.scale, tokens, tokens, want)
    lse[row, 3] = float("nan")
    mass = torch.zeros(1, 1, tokens, device=DEV)
    sa.prefill_mass(q.to(DEV), cu, k, table, kv, lse, c.scale, tokens, tokens, mass)
    assert torch.isnan(mass[0, 0, :row + 1]).all()
    assert torch.equal(mass[0, 0, row + 1:], want[0, 0, row + 1:])


def test_mass_of_bounds_of_zero():
    # lengths past a bound of 0 are out of range as past any other
    c = Paged([5, 0, 3], 4, 1)
    q = bf16(c.rng, 3, 4, 64).to(DEV)
    k, _, table, kv = c.paged()
    lse = torch.zeros(3, 4, device=DEV)
    cu = torch.tensor([0, 2, 2, 3], dtype=torch.int32, device=DEV)
    for call in (lambda m: sa.decode_mass(q, k, table, kv, lse, c.scale, 0, m),
                 lambda m: sa.prefill_mass(q, cu, k, table, kv, lse, c.scale, 2, 0, m),
                 lambda m: sa.prefill_mass(q, cu, k, table, kv, lse, c.scale, 300, 0, m),
                 lambda m: sa.prefill_mass(q, cu, k, table, kv, lse, c.scale, 0, 5, m)):
        mass = torch.ones(3, 1, 9, device=DEV)
        call(mass)
        assert torch.isnan(mass[[0, 2]]).all()
        assert (mass[1] == 1).all()


@pytest.mark.parametrize("heads", [(10, 2), (4, 1), (24, 1), (5, 1), (36, 2), (8, 1)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_infinite_keys_weigh_nothing_where_every_score_is_minus_infinity(heads, sign):
    # key 20 holds an infinity, its score is -inf for every head: exp(-inf) = 0,
    # for any number of heads
    hq, hkv = heads
    c = Paged([40], hq, hkv)
    k, v, table, kv = c.paged()
    k[table[0, 1].long(), :, 4, 9] = sign * float("inf")
    q = bf16(c.rng, 2, hq, 64)
    q[..., 9] = -sign
    q = q.to(DEV)
    cu = torch.tensor([0, 2], dtype=torch.int32, device=DEV)
    lse = torch.full((2, hq), 3.0, device=DEV)
    for call in (lambda m: sa.decode_mass(q[:1], k, table, kv, lse[:1], c.scale, 40, m),
                 lambda m: sa.prefill_mass(q, cu, k, table, kv, lse, c.scale, 2, 40, m)):
        mass = torch.ones(1, hkv, 40, device=DEV)
        call(mass)
        assert (mass[0, :, 20] == 1).all()
        assert torch.isfinite(mass).all()


# ------------------------------------------------------------- the largest sizes
def test_lengths_and_budgets_up_to_the_largest_int():
    # rows of 2^31 - 1 entries: a length that fits them but not its page table is out of
    # range, and what is written over a whole row ends at its end
    top = 2**31 - 1
    c = Paged([5], 4, 1)
    k, v, table, kv = c.paged()
    q, lse = bf16(c.rng, 1, 4, 64).to(DEV), torch.zeros(1, 4, device=DEV)
    cu = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    mass = torch.empty(1, 1, top, device=DEV)
    for length in (top, top - 7, -1):
        kv[0] = length
        for call in (lambda: sa.decode_mass(q, k, table, kv, lse, c.scale, top, mass),
                     lambda: sa.prefill_mass(q, cu, k, table, kv, lse, c.scale, 1, top, mass)):
            mass.zero_()
            call()
            for at in (slice(0, 4096), slice(top // 2, top // 2 + 4096), slice(top - 4096, top)):
                assert torch.isnan(mass[0, 0, at]).all()
        before = (k.clone(), v.clone())
        new, kept = sa.evict(k, v, table, kv, mass, 4, top)
        assert new.tolist() == [-1] and (kept == -1).all()
        assert torch.equal(k.view(torch.int16), before[0].view(torch.int16))
        assert torch.equal(v.view(torch.int16), before[1].view(torch.int16))
    kv[0] = 5
    kept = torch.zeros(1, 1, top, dtype=torch.int32, device=DEV)
    new, _ = sa.evict(k, v, table, kv, mass, top, top, kept=kept)
    assert new.tolist() == [5] and kept[0, 0, :5].tolist() == [0, 1, 2, 3, 4]
    for at in (slice(5, 4096), slice(top // 2, top // 2 + 4096), slice(top - 4096, top)):
        assert (kept[0, 0, at] == -1).all()


def test_the_calls_allocate_nothing_when_handed_their_outputs():
    c = Paged([700, 300], 16, 2, spare=20)
    q, q1, sinks = bf16(c.rng, 60, 16, 64).to(DEV), bf16(c.rng, 2, 16, 64).to(DEV), c.sinks.to(DEV)
    k, v, table, kv = c.paged()
    cu = torch.tensor([0, 40, 60], dtype=torch.int32, device=DEV)
    out, lse, out1, lse1 = (torch.empty_like(x) for x in (q, q[..., 0].float(), q1, q1[..., 0].float()))
    kk, vv = (x[0][:60].to(DEV) for x in (c.k, c.v))
    mass = torch.zeros(2, 2, 700, device=DEV)
    new, kept = torch.empty_like(kv), torch.empty(2, 2, 650, dtype=torch.int32, device=DEV)
    splits, need = sa.decode_window_plan(2, 16, 2, 700, 600, 4, 5)
    assert splits > 1
    ws = torch.zeros(need, dtype=torch.uint8, device=DEV)

    def run():
        sa.decode_window(q1, k, v, table, kv, sinks, c.scale, 700, 600, 4, num_splits=5, out=out1, lse=lse1, workspace=ws)
        for window in (20, 500):
            sa.prefill_window(q, kk, vv, cu, sinks, c.scale, 40, window, out=out, lse=lse)
            sa.prefill_paged_window(q, cu, k, v, table, kv, sinks, c.scale, 40, 700, window, out=out, lse=lse)
        sa.prefill_mass(q, cu, k, table, kv, lse, c.scale, 40, 700, mass)
        sa.decode_mass(q1, k, table, kv, lse1, c.scale, 700, mass)
        sa.evict(k, v, table, kv, mass, 650, 700, new_kv_lens=new, kept=kept)

    def held():
        torch.cuda.synchronize()
        return torch.cuda.memory_stats()["allocation.all.allocated"], torch.cuda.mem_get_info()[0]

    run()                                                 # kernels are loaded on their first launch
    before = held()
    for _ in range(3):
        run()
    assert held() == before
