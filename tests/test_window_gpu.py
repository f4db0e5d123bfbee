"""Windowed attention on the GPU against the float64 oracle: one token,
ragged prefill, prefill on a paged prefix.

Bars: those of the other attention kernels (tolerances.py).  They hold here
too: the kernels round the same things (weights to bf16 for the product with
V, the output once to bf16), and a window only takes keys away.
"""

import numpy as np
import pytest
import torch

import gqa_attention_learned_gb300 as sa
from bounded_inputs import DEV, Paged, bf16, np64
from oracle import bounded
from tolerances import assert_lse_close, assert_out_close

pytestmark = pytest.mark.gpu

HEADS = [(64, 8), (4, 1), (8, 8), (10, 2), (32, 2), (24, 1)]
WINDOWS = [(1, 0), (2, 1), (16, 0), (17, 5), (128, 4), (130, 33), (1000, 0), (40, 64)]
LENS = [0, 1, 2, 15, 16, 17, 31, 33, 128, 129, 144, 145, 300, 301]


def _decode_ref(c, q, window, first):
    outs, lses = [], []
    for b, n in enumerate(c.lens):
        o, l = bounded.window_rows(np64(q[b:b + 1]), np64(c.k[b]), np64(c.v[b]), [n - 1],
                                   np64(c.sinks), c.scale, window, first)
        outs.append(o[0])
        lses.append(l[0])
    return np.stack(outs), np.stack(lses)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("window,first", WINDOWS)
def test_decode_window(heads, window, first):
    c = Paged(LENS, *heads, seed=window)
    q = bf16(c.rng, len(LENS), heads[0], 64)
    ro, rl = _decode_ref(c, q, window, first)
    for b, n in enumerate(c.lens):
        c.hide(b, bounded.visible(n - 1, n, window, first))
    args = (q.to(DEV), *c.paged(), c.sinks.to(DEV), c.scale, c.max_kv, window, first)
    for splits in (0, 1, 3):
        out, lse = sa.decode_window(*args, num_splits=splits)
        assert_out_close(out, ro)
        assert_lse_close(lse, rl)
    again, lse2 = sa.decode_window(*args, num_splits=3, programmatic=True)
    assert torch.equal(again, out) and torch.equal(lse2, lse)


@pytest.mark.parametrize("heads,batch", [((64, 8), 64), ((48, 4), 130)])
@pytest.mark.parametrize("window,first", [(40, 3), (130, 0)])
def test_decode_window_of_many_requests(heads, batch, window, first):
    # more CTAs than the GPU holds with two pages in flight per warp
    lens = [int(n) for n in np.random.default_rng(batch).integers(0, 400, batch)]
    c = Paged(lens, *heads, seed=window)
    q = bf16(c.rng, batch, heads[0], 64)
    ro, rl = _decode_ref(c, q, window, first)
    for b, n in enumerate(c.lens):
        c.hide(b, bounded.visible(n - 1, n, window, first))
    k, v, table, kv_lens = c.paged()
    args = (q.to(DEV), k, v, table, kv_lens, c.sinks.to(DEV), c.scale, c.max_kv, window, first)
    out, lse = sa.decode_window(*args)
    assert_out_close(out, ro)
    assert_lse_close(lse, rl)
    b = int(np.argmax(lens))                             # a visible page outside the pool
    table[b, (lens[b] - 1) // 16] = c.pages
    bad, bad_lse = sa.decode_window(*args)
    assert torch.isnan(bad[b]).all() and torch.isnan(bad_lse[b]).all()
    rest = torch.arange(batch, device=DEV) != b
    assert torch.equal(bad[rest], out[rest]) and torch.equal(bad_lse[rest], lse[rest])


def test_a_window_without_bound_is_decode():
    c = Paged([300, 17, 1], 64, 8)
    q = bf16(c.rng, 3, 64, 64).to(DEV)
    args = (q, *c.paged(), c.sinks.to(DEV), c.scale, c.max_kv)
    for splits in (1, 4):
        a = sa.decode(*args, num_splits=splits)
        b = sa.decode_window(*args, 2**40, num_splits=splits)
        assert_out_close(b[0], np64(a[0]))
        assert_lse_close(b[1], np64(a[1]))


@pytest.mark.parametrize("window,first", [(20, 3), (2**40, 0), (20, 2**40), (2**40, 2**40)])
def test_lengths_without_bound(window, first):
    # bounds past any int mean none; nothing else changes
    c = Paged([300, 17], 8, 2)
    paged, sinks = c.paged(), c.sinks.to(DEV)
    q = bf16(c.rng, 140, 8, 64).to(DEV)
    cu = torch.tensor([0, 130, 140], dtype=torch.int32, device=DEV)
    none = 2**40
    ours = (min(window, 300), min(first, 300))
    for free, bound in (
            (sa.decode_window(q[:2], *paged, sinks, c.scale, none, window, first),
             sa.decode_window(q[:2], *paged, sinks, c.scale, 300, *ours)),
            (sa.prefill_paged_window(q, cu, *paged, sinks, c.scale, none, none, window, first),
             sa.prefill_paged_window(q, cu, *paged, sinks, c.scale, 130, 300, *ours)),
            (sa.prefill_window(q, *(x[0][:140].to(DEV) for x in (c.k, c.v)), cu, sinks, c.scale, none, window,
                               first),
             sa.prefill_window(q, *(x[0][:140].to(DEV) for x in (c.k, c.v)), cu, sinks, c.scale, 130, *ours))):
        assert torch.isfinite(bound[0]).all()
        assert_out_close(free[0], np64(bound[0]))
        assert_lse_close(free[1], np64(bound[1]))


@pytest.mark.parametrize("window", [40, 260])
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
def test_keys_that_are_not_finite_spoil_the_rows_that_see_them(window, what):
    # key 20: the output and the lse of a row that sees it are NaN (an infinite
    # score is one too: inf - inf), in one chunk or several
    c = Paged([300], 4, 1)
    k, v, table, lens = c.paged()
    k[table[0, 1].long(), 0, 4, 0] = what
    sinks = c.sinks.to(DEV)
    q = bf16(c.rng, 300, 4, 64).abs().to(DEV)            # no score of -inf
    seen = torch.tensor(np.stack([bounded.visible(i, 300, window, 0) for i in range(300)])[:, 20], device=DEV)
    cu = torch.tensor([0, 300], dtype=torch.int32, device=DEV)
    out, lse = sa.prefill_paged_window(q, cu, k, v, table, lens, sinks, c.scale, 300, 300, window)
    assert torch.isnan(lse[seen]).all() and torch.isfinite(lse[~seen]).all()
    assert torch.isnan(out[seen]).all() and torch.isfinite(out[~seen]).all()
    for splits in (1, 5):
        out, lse = sa.decode_window(q[:1], k, v, table, lens, sinks, c.scale, 300, 300, num_splits=splits)
        assert torch.isnan(out).all() and torch.isnan(lse).all()
        out, lse = sa.decode_window(q[:1], k, v, table, lens, sinks, c.scale, 300, 200, num_splits=splits)
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()


def test_decode_window_masked_heads_and_zero_scale():
    # a sink of -inf on some heads; a request that sees nothing; scale 0 and below
    c = Paged([40, 0, 200], 8, 2)
    c.sinks[::2] = -np.inf
    q = bf16(c.rng, 3, 8, 64)
    for scale in (0.0, -0.125):
        c.scale = scale
        ro, rl = _decode_ref(c, q, 9, 2)
        out, lse = sa.decode_window(q.to(DEV), *c.paged(), c.sinks.to(DEV), scale, c.max_kv, 9, 2)
        assert_out_close(out, ro)
        assert_lse_close(lse, rl)


def test_decode_window_out_of_range_requests_give_nan():
    c = Paged([20, 300, 20, 64], 4, 1)
    q = bf16(c.rng, 4, 4, 64).to(DEV)
    k, v, table, lens = c.paged()
    lens[0] = -1
    lens[1] = 301                                       # past max_kv_len
    table[2, 1] = c.pages                               # a visible page outside the pool
    out, lse = sa.decode_window(q, k, v, table, lens, c.sinks.to(DEV), c.scale, 300, 8)
    assert torch.isnan(out[:3]).all() and torch.isnan(lse[:3]).all()
    assert torch.isfinite(out[3]).all()


def _prefill_ref(c_or_kv, q, cu, shift, sinks, scale, window, first):
    k, v = c_or_kv
    outs, lses = [], []
    for b in range(len(cu) - 1):
        rows = range(cu[b], cu[b + 1])
        o, l = bounded.window_rows(np64(q[cu[b]:cu[b + 1]]), np64(k[b]), np64(v[b]),
                                   [shift[b] + i for i in range(len(rows))], sinks, scale, window, first)
        outs.append(o)
        lses.append(l)
    return np.concatenate(outs), np.concatenate(lses)


@pytest.mark.parametrize("heads", [(64, 8), (4, 1), (8, 8), (10, 2), (32, 2)])
@pytest.mark.parametrize("window,first", [(1, 0), (17, 5), (128, 0), (130, 33), (1000, 0), (40, 64)])
def test_prefill_window_ragged(heads, window, first):
    hq, hkv = heads
    rng = np.random.default_rng(window)
    lens = [1, 17, 300, 0, 129]
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = bf16(rng, cu[-1], hq, 64), bf16(rng, cu[-1], hkv, 64), bf16(rng, cu[-1], hkv, 64)
    sinks = torch.from_numpy(rng.standard_normal(hq).astype(np.float32))
    parts = [slice(cu[b], cu[b + 1]) for b in range(len(lens))]
    ro, rl = _prefill_ref(([k[p] for p in parts], [v[p] for p in parts]), q, cu, [0] * len(lens),
                          np64(sinks), 0.125, window, first)
    out, lse = sa.prefill_window(q.to(DEV), k.to(DEV), v.to(DEV),
                                 torch.tensor(cu, dtype=torch.int32, device=DEV), sinks.to(DEV), 0.125,
                                 300, window, first)
    assert_out_close(out, ro)
    assert_lse_close(lse, rl)


@pytest.mark.parametrize("heads", [(64, 8), (4, 1), (6, 2)])
@pytest.mark.parametrize("window,first", [(1, 0), (17, 5), (128, 4), (130, 33), (1000, 0), (40, 64), (300, 150)])
def test_prefill_paged_window(heads, window, first):
    # new tokens on prefixes of every alignment; what no row sees is NaN or has no page
    q_lens, prefix = [1, 5, 140, 33, 16], [0, 400, 259, 31, 512]
    c = Paged([a + b for a, b in zip(q_lens, prefix)], *heads, seed=first)
    cu = np.concatenate([[0], np.cumsum(q_lens)])
    q = bf16(c.rng, cu[-1], heads[0], 64)
    ro, rl = _prefill_ref((c.k, c.v), q, cu, prefix, np64(c.sinks), c.scale, window, first)
    for b, n in enumerate(c.lens):
        seen = np.zeros(n, bool)
        for p in range(prefix[b], n):
            seen |= bounded.visible(p, n, window, first)
        c.hide(b, seen)
    out, lse = sa.prefill_paged_window(q.to(DEV), torch.tensor(cu, dtype=torch.int32, device=DEV),
                                       *c.paged(), c.sinks.to(DEV), c.scale, max(q_lens), c.max_kv,
                                       window, first)
    assert_out_close(out, ro)
    assert_lse_close(lse, rl)


def test_prefill_window_zero_and_negative_scale():
    rng = np.random.default_rng(3)
    q, k, v = bf16(rng, 200, 4, 64), bf16(rng, 200, 1, 64), bf16(rng, 200, 1, 64)
    sinks = torch.tensor([0.5, -np.inf, 3.0, -1.0])
    cu = torch.tensor([0, 200], dtype=torch.int32, device=DEV)
    for scale in (0.0, -0.125):
        ro, rl = bounded.window_rows(np64(q), np64(k), np64(v), range(200), np64(sinks), scale, 30, 3)
        out, lse = sa.prefill_window(q.to(DEV), k.to(DEV), v.to(DEV), cu, sinks.to(DEV), scale, 200, 30, 3)
        assert_out_close(out, ro)
        assert_lse_close(lse, rl)


def test_prefill_window_leaves_other_rows_alone_and_flags_bad_ones():
    # rows behind the last sequence stay as they were; a sequence longer than
    # the bound gives NaN; cu_seqlens past the rows give NaN up to their end
    rng = np.random.default_rng(4)
    q, k, v = (bf16(rng, 100, h, 64).to(DEV) for h in (4, 1, 1))
    sinks = torch.zeros(4, device=DEV)
    out = torch.full_like(q, 7.0)
    lse = torch.full((100, 4), 7.0, device=DEV)
    sa.prefill_window(q, k, v, torch.tensor([0, 20, 60], dtype=torch.int32, device=DEV), sinks, 0.125,
                      30, 8, out=out, lse=lse)
    assert torch.isfinite(out[:20]).all()
    assert torch.isnan(out[20:60]).all() and torch.isnan(lse[20:60]).all()
    assert (out[60:] == 7).all() and (lse[60:] == 7).all()
    sa.prefill_window(q, k, v, torch.tensor([0, 90, 120], dtype=torch.int32, device=DEV), sinks, 0.125,
                      90, 8, out=out, lse=lse)
    assert torch.isfinite(out[:90]).all() and torch.isnan(out[90:]).all()


def test_long_windows_leave_other_rows_alone_and_flag_bad_ones():
    # the same where a tile's keys do not fit at once
    rng = np.random.default_rng(5)
    q, k, v = (bf16(rng, 700, h, 64).to(DEV) for h in (4, 1, 1))
    sinks = torch.zeros(4, device=DEV)
    for cu, bad, good in (([0, 300, 600], [], [(0, 600)]), ([0, 250, 600], [(250, 600)], [(0, 250)]),
                          ([0, 290, 580, 900], [(580, 700)], [(0, 580)])):
        out = torch.full_like(q, 7.0)
        lse = torch.full((700, 4), 7.0, device=DEV)
        sa.prefill_window(q, k, v, torch.tensor(cu, dtype=torch.int32, device=DEV), sinks, 0.125, 300, 280,
                          out=out, lse=lse)
        touched = torch.zeros(700, dtype=torch.bool, device=DEV)
        for a, z in good:
            touched[a:z] = True
            assert torch.isfinite(out[a:z]).all() and not (out[a:z] == 7).all(-1).any()
        for a, z in bad:
            touched[a:z] = True
            assert torch.isnan(out[a:z]).all() and torch.isnan(lse[a:z]).all()
        assert (out[~touched] == 7).all() and (lse[~touched] == 7).all()


@pytest.mark.parametrize("window", [20, 280])
def test_prefill_window_of_many_requests(window):
    # 100 requests, some without tokens, one longer than the bound, one of cu_seqlens
    # that falls back: its neighbours' rows stay right
    rng = np.random.default_rng(6)
    lens = [int(n) for n in rng.integers(0, 40, 100)]
    lens[40] = 290                                       # the kernel for long windows needs long requests
    lens[41] = 0
    lens[70] = 310
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1])
    q, k, v = bf16(rng, total, 16, 64), bf16(rng, total, 1, 64), bf16(rng, total, 1, 64)
    sinks = torch.from_numpy(rng.standard_normal(16).astype(np.float32))
    parts = [slice(cu[b], cu[b + 1]) for b in range(100)]
    ro, rl = _prefill_ref(([k[p] for p in parts], [v[p] for p in parts]), q, cu, [0] * 100,
                          np64(sinks), 0.125, window, 3)
    out, lse = sa.prefill_window(q.to(DEV), k.to(DEV), v.to(DEV),
                                 torch.tensor(cu, dtype=torch.int32, device=DEV), sinks.to(DEV), 0.125,
                                 300, window, 3)
    good = np.ones(total, bool)
    good[parts[70]] = False
    assert torch.isnan(out[parts[70]]).all() and torch.isnan(lse[parts[70]]).all()
    assert_out_close(out[good], ro[good])
    assert_lse_close(lse[good], rl[good])
    # entry 51 before entry 50: request 50 has no rows, request 51 is out of order
    back = cu.copy()
    back[51] = cu[50] - 5
    out, lse = sa.prefill_window(q.to(DEV), k.to(DEV), v.to(DEV),
                                 torch.tensor(back, dtype=torch.int32, device=DEV), sinks.to(DEV), 0.125,
                                 300, window, 3)
    assert torch.isnan(out[cu[50]:cu[52]]).all()
    good[cu[50] - 5:cu[52]] = False
    assert_out_close(out[good], ro[good])
    assert_lse_close(lse[good], rl[good])


@pytest.mark.parametrize("window", [20, 280])
def test_prefill_window_of_requests_alike(window):
    # tiles of equal requests; one longer than the bound, one past the rows
    rng = np.random.default_rng(8)
    q, k, v = (bf16(rng, 1500, h, 64) for h in (4, 1, 1))
    sinks = torch.zeros(4)
    cu = [0, 290, 580, 870, 1160, 1500]
    parts = [slice(a, b) for a, b in zip(cu, cu[1:])]
    ro, rl = _prefill_ref(([k[p] for p in parts], [v[p] for p in parts]), q, cu, [0] * 5, np64(sinks), 0.125,
                          window, 0)
    for bound, ends in ((340, 1500), (300, 1500), (340, 1600)):
        at = cu[:5] + [ends]
        out, lse = sa.prefill_window(q.to(DEV), k.to(DEV), v.to(DEV),
                                     torch.tensor(at, dtype=torch.int32, device=DEV), sinks.to(DEV), 0.125,
                                     bound, window)
        good = 1500 if bound >= 340 and ends == 1500 else 1160
        assert_out_close(out[:good], ro[:good])
        assert_lse_close(lse[:good], rl[:good])
        assert torch.isnan(out[good:]).all() and torch.isnan(lse[good:]).all()


@pytest.mark.parametrize("window", [100, 400])
@pytest.mark.parametrize("batch,longest", [(90, 300), (300, 60)])
def test_prefill_window_of_a_request_does_not_depend_on_the_batch(window, batch, longest):
    # more tiles than the persistent CTAs look up at a time, more requests than are
    # numbered through
    rng = np.random.default_rng(7)
    lens = [int(n) for n in rng.integers(0, longest, batch)]
    lens[5] = 450
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1])
    gen = torch.Generator(DEV).manual_seed(0)
    q, k, v = (torch.randn(total, h, 64, generator=gen, device=DEV).bfloat16() for h in (64, 1, 1))
    sinks = torch.zeros(64, device=DEV)

    def ints(x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    out, lse = sa.prefill_window(q, k, v, ints(cu), sinks, 0.125, 450, window)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for b in (0, 5, 31, 32, 50, 63, 64, batch - 2, batch - 1):
        at = slice(cu[b], cu[b + 1])
        if lens[b]:
            # the same bound on lengths: the same kernel
            a, c = sa.prefill_window(q[at].contiguous(), k[at].contiguous(), v[at].contiguous(),
                                     ints([0, lens[b]]), sinks, 0.125, 450, window)
            assert torch.equal(out[at], a) and torch.equal(lse[at], c)


def test_windowed_calls_without_lse_and_without_keys():
    c = Paged([0, 0], 4, 1)
    q = bf16(c.rng, 2, 4, 64).to(DEV)
    k, v, table, lens = c.paged()
    out, lse = sa.decode_window(q, k, v, table, lens, c.sinks.to(DEV), c.scale, 0, 5, 3)
    assert (out == 0).all()
    assert_lse_close(lse, np.broadcast_to(np64(c.sinks), (2, 4)))
    c = Paged([500], 4, 1)
    q = bf16(c.rng, 500, 4, 64).to(DEV)
    cu = torch.tensor([0, 500], dtype=torch.int32, device=DEV)
    kv = c.paged()
    for window in (20, 400):
        args = (q, cu, *kv, c.sinks.to(DEV), c.scale, 500, 500, window, 2)
        a, none = sa.prefill_paged_window(*args, want_lse=False)
        b, _ = sa.prefill_paged_window(*args)
        assert none is None and torch.equal(a, b)
    q1 = q[:1].contiguous()
    a, none = sa.decode_window(q1, *kv, c.sinks.to(DEV), c.scale, 500, 20, want_lse=False)
    b, _ = sa.decode_window(q1, *kv, c.sinks.to(DEV), c.scale, 500, 20)
    assert none is None and torch.equal(a, b)


def test_prefill_paged_window_bad_page_and_short_cache():
    c = Paged([200, 50, 90], 4, 1)
    cu = torch.tensor([0, 100, 160, 200], dtype=torch.int32, device=DEV)
    q = bf16(c.rng, 200, 4, 64).to(DEV)
    k, v, table, lens = c.paged()
    table[0, 12] = -5                                    # keys 192..199: seen by the last rows
    out, lse = sa.prefill_paged_window(q, cu, k, v, table, lens, c.sinks.to(DEV), c.scale, 100, 200, 16)
    assert torch.isnan(out[99]).all() and torch.isnan(lse[99]).all()
    assert torch.isfinite(out[0]).all()
    assert torch.isnan(out[100:160]).all()               # 60 new tokens, 50 keys
    assert torch.isfinite(out[160:]).all()


def test_windowed_forms_agree_and_replay_from_a_graph():
    # decode of the last token = the last row of the paged and ragged prefill
    c = Paged([333], 64, 8)
    q = bf16(c.rng, 333, 64, 64).to(DEV)
    cu = torch.tensor([0, 333], dtype=torch.int32, device=DEV)
    paged, sinks = c.paged(), c.sinks.to(DEV)
    k, v = c.k[0].to(DEV), c.v[0].to(DEV)

    def run():
        a = sa.prefill_window(q, k, v, cu, sinks, c.scale, 333, 100, 7)
        b = sa.prefill_paged_window(q, cu, *paged, sinks, c.scale, 333, 333, 100, 7)
        d = sa.decode_window(q[-1:].contiguous(), *paged, sinks, c.scale, 333, 100, 7)
        return a, b, d

    a, b, d = run()
    assert_out_close(b[0], np64(a[0]))
    assert_lse_close(b[1], np64(a[1]))
    assert_out_close(d[0], np64(a[0][-1:]))
    assert_lse_close(d[1], np64(a[1][-1:]))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ga, gb, gd = run()
    q.copy_(bf16(np.random.default_rng(9), 333, 64, 64))
    g.replay()
    torch.cuda.synchronize()
    for x, y in zip((ga, gb, gd), run()):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])


def test_another_stream_orders_its_own_workspace():
    c = Paged([2000, 1999], 64, 8)
    q = bf16(c.rng, 2, 64, 64).to(DEV)
    args = (q, *c.paged(), c.sinks.to(DEV), c.scale, 2000, 1500, 4)
    want = sa.decode_window(*args, num_splits=8)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = [sa.decode_window(*args, num_splits=8, stream=side) for _ in range(4)]
    side.synchronize()
    for o, l in got:
        assert torch.equal(o, want[0]) and torch.equal(l, want[1])


# ------------------------------------------------- few tiles per persistent CTA
@pytest.mark.parametrize("heads,window,first", [((16, 2), 30, 3), ((16, 2), 100, 40), ((4, 1), 100, 0), ((10, 2), 7, 1)])
@pytest.mark.parametrize("tokens", [1, 40, 330, 1300])
def test_short_windows_with_few_tiles_per_cta(heads, window, first, tokens):
    # a CTA's first tiles and its last entries follow one another without a
    # stage to wait for: 0, 1, 2 tiles per CTA and some more
    hq, hkv = heads
    c = Paged([tokens], hq, hkv, seed=tokens)
    q = bf16(c.rng, tokens, hq, 64)
    ro, rl = bounded.window_rows(np64(q), np64(c.k[0]), np64(c.v[0]), range(tokens), np64(c.sinks), c.scale,
                                 window, first)
    cu = torch.tensor([0, tokens], dtype=torch.int32, device=DEV)
    for _ in range(3):
        out, lse = sa.prefill_paged_window(q.to(DEV), cu, *c.paged(), c.sinks.to(DEV), c.scale, tokens, tokens,
                                           window, first)
        assert_out_close(out, ro)
        assert_lse_close(lse, rl)


# -------------------------------------------------------------------- odd sinks
@pytest.mark.parametrize("what", [float("nan"), float("inf")])
@pytest.mark.parametrize("others", [None, 90.0, -float("inf")])
def test_sinks_that_are_no_logit_spoil_their_heads(what, others):
    # NaN and +inf: output and lse of the head are NaN, in one chunk or several,
    # whatever the row sees and whether the other heads' running maxima move (below a
    # sink of 90 they do not); the other heads are not touched
    def sinks(c):
        good = c.sinks if others is None else torch.full_like(c.sinks, others)
        bad = good.clone()
        bad[2], bad[7] = what, what
        return good.to(DEV), bad.to(DEV)

    fine = torch.tensor([h not in (2, 7) for h in range(8)], device=DEV)

    def check(got, want):
        assert torch.isnan(got[0][:, ~fine]).all() and torch.isnan(got[1][:, ~fine]).all()
        assert torch.equal(got[0][:, fine], want[0][:, fine]) and torch.equal(got[1][:, fine], want[1][:, fine])

    for hkv in (1, 2):                                   # groups of 8 and of 4
        c = Paged([300, 0, 20], 8, hkv)
        q = bf16(c.rng, 3, 8, 64).to(DEV)
        want, got = ([sa.decode_window(q, *c.paged(), s, c.scale, 300, 200, 3, num_splits=n) for n in (1, 5)]
                     for s in sinks(c))
        for x, y in zip(got, want):
            check(x, y)
        c = Paged([450], 8, hkv)
        q = bf16(c.rng, 450, 8, 64).to(DEV)
        cu = torch.tensor([0, 450], dtype=torch.int32, device=DEV)
        want, got = ([sa.prefill_paged_window(q, cu, *c.paged(), s, c.scale, 450, 450, w) for w in (20, 400)]
                     for s in sinks(c))
        for x, y in zip(got, want):
            check(x, y)


# ---------------------------------------------------------- one workspace for all
def test_one_workspace_serves_windowed_plans_of_every_shape():
    # zero-filled once: plans keep their counters where others keep partial results,
    # so every call has to leave all of that at zero
    cases = []
    for batch, hq, hkv, window, splits in ((8, 64, 8, 1500, 4), (28, 64, 8, 1500, 3), (8, 64, 8, 1500, 4),
                                           (64, 8, 8, 700, 5), (3, 128, 1, 900, 7), (9, 64, 8, 1500, 0),
                                           (1, 4, 1, 2000, 9), (28, 64, 8, 1500, 3), (700, 8, 8, 64, 2),
                                           (28, 64, 8, 1500, 3)):
        rng = np.random.default_rng(batch)
        c = Paged([int(n) for n in rng.integers(600, 2000, batch)] if batch < 100 else [70] * batch, hq, hkv,
                  seed=batch)
        q = bf16(c.rng, batch, hq, 64).to(DEV)
        cases.append(((q, *c.paged(), c.sinks.to(DEV), c.scale, 2000, window, 5), splits))
    sizes = [sa.decode_window_plan(a[0].shape[0], a[0].shape[1], a[1].shape[1], 2000, a[8], 5, s)
             for a, s in cases]
    assert min(s for s, _ in sizes) > 1
    shared = torch.zeros(max(b for _, b in sizes), dtype=torch.uint8, device=DEV)
    for args, splits in cases:
        want = sa.decode_window(*args, num_splits=splits)
        out = torch.full_like(want[0], 7.0)
        lse = torch.full_like(want[1], 7.0)
        sa.decode_window(*args, num_splits=splits, workspace=shared, out=out, lse=lse)
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.parametrize("window", [20, 400])
def test_requests_longer_than_a_bound_of_zero_give_nan(window):
    c = Paged([40, 450], 4, 1)
    q = bf16(c.rng, 10, 4, 64).to(DEV)
    cu = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    sinks = c.sinks.to(DEV)
    k, v = (x[0][:10].to(DEV) for x in (c.k, c.v))
    for call in (lambda **kw: sa.prefill_paged_window(q, cu, *c.paged(), sinks, c.scale, 0, 450, window, **kw),
                 lambda **kw: sa.prefill_paged_window(q, cu, *c.paged(), sinks, c.scale, 4, 0, window, **kw),
                 lambda **kw: sa.prefill_window(q, k, v, cu, sinks, c.scale, 0, window, **kw)):
        out, lse = torch.full_like(q, 7.0), torch.full((10, 4), 7.0, device=DEV)
        call(out=out, lse=lse)
        assert torch.isnan(out[:8]).all() and torch.isnan(lse[:8]).all()
        assert (out[8:] == 7).all() and (lse[8:] == 7).all()


# ----------------------------------------------------------------- loose bounds
@pytest.mark.parametrize("heads,window,requests", [((64, 8), 20, 2), ((64, 8), 20, 150), ((64, 8), 400, 150),
                                                   ((128, 1), 20, 40), ((6, 2), 100, 200)])
def test_prefill_window_bounds_need_not_be_tight(heads, window, requests):
    # lengths far below the bounds, and no bounds: the same rows, whatever the
    # number of requests and of tiles that none of them has; requests that are refused
    # stay refused, rows behind the last request stay as they are
    hq, hkv = heads
    rng = np.random.default_rng(requests)
    lens = [int(n) for n in rng.integers(0, 30, requests)]
    lens[0], lens[1] = 40, 130
    prefix = [int(n) for n in rng.integers(0, 60, requests)]
    prefix[1] = 500
    bad = requests // 2 if requests > 2 else None
    c = Paged([a + b for a, b in zip(lens, prefix)], hq, hkv, seed=window)
    cu = np.concatenate([[0], np.cumsum(lens)])
    total = int(cu[-1])
    q = bf16(c.rng, total + 9, hq, 64).to(DEV)
    cu = torch.tensor(cu, dtype=torch.int32, device=DEV)
    sinks, paged = c.sinks.to(DEV), c.paged()
    k, v = (torch.cat(x)[:total + 9].to(DEV).contiguous() for x in (c.k, c.v))
    if bad:
        paged[3][bad] = -1
    parts = [slice(a, b) for a, b in zip(cu.tolist(), cu.tolist()[1:])]
    nan = torch.zeros(total, dtype=torch.bool)
    if bad:
        nan[parts[bad]] = True
    held = ((c.k, c.v, prefix), ([k[p] for p in parts], [v[p] for p in parts], [0] * requests))
    refs = [_prefill_ref(kv[:2], q[:total], cu.tolist(), kv[2], np64(c.sinks), c.scale, window, 3) for kv in held]
    # Rows that see few keys: weights p and the output are rounded to bf16, each off by at
    # most 2^-8 of its value, so out = sum p v is off by at most 2^-8 (sum p |v| + |out|), and
    # sum p <= 1 bounds the first sum by the largest |v| of the request; 5% on top for the
    # second order (2^-8) and fp32 (scores of 64 products are off by less than 1e-4).
    bars = []
    for (_, vs, _), (ref, _) in zip(held, refs):
        top = [np.abs(np64(x)).max(0) if len(x) else np.zeros((hkv, 64)) for x in vs]
        top = np.concatenate([np.broadcast_to(t, (n, hkv, 64)) for t, n in zip(top, lens)])
        bars.append(1.05 * 2.0**-8 * (np.repeat(top, hq // hkv, 1) + np.abs(ref)))
    out, lse = torch.empty_like(q), torch.empty(total + 9, hq, device=DEV)
    for ragged, bounds in ((0, (130, c.max_kv)), (0, (5000, c.max_kv)), (0, (2**40, c.max_kv)), (0, (2**40, 2**40)),
                           (1, (130,)), (1, (700,)), (1, (131072,)), (1, (2**40,))):
        out.fill_(7)
        lse.fill_(7)
        if ragged:
            sa.prefill_window(q, k, v, cu, sinks, c.scale, *bounds, window, 3, out=out, lse=lse)
        else:
            sa.prefill_paged_window(q, cu, *paged, sinks, c.scale, *bounds, window, 3, out=out, lse=lse)
        refused = nan if not ragged else torch.zeros_like(nan)
        assert torch.isnan(out[:total][refused]).all() and torch.isnan(lse[:total][refused]).all()
        fine = (~refused).numpy()
        assert (np.abs(np64(out[:total])[fine] - refs[ragged][0][fine]) <= bars[ragged][fine]).all()
        assert_lse_close(lse[:total][~refused], refs[ragged][1][fine])
        assert (out[total:] == 7).all() and (lse[total:] == 7).all()
