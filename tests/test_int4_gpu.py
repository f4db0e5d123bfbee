"""Operators on a paged cache held in 4 bits, on the GPU, against float64 references
(tests/int4_inputs.py says where the bars come from)."""

import numpy as np
import pytest
import torch

import gqa_attention_learned_gb300 as sa
from gqa_attention_learned_gb300 import workloads
from int4_inputs import DEV, Packed, assert_rows, np64, rows
from oracle import int4
from oracle import prologue as pro

pytestmark = pytest.mark.gpu

HEADS = [(64, 8), (4, 1), (8, 8), (10, 2), (32, 2), (24, 1), (40, 1)]


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# -------------------------------------------------------------------- prologue
def _rotated(x, cos, sin, interleaved):
    """fp32 steps of the rotation, one rounding each; x [T, H, 64]."""
    a, b = pro.pair_index(64, "interleaved" if interleaved else "half")
    y = np.empty_like(x)
    with np.errstate(all="ignore"):
        y[..., a] = x[..., a] * cos[:, None] - x[..., b] * sin[:, None]
        y[..., b] = x[..., b] * cos[:, None] + x[..., a] * sin[:, None]
    return y


@pytest.mark.parametrize("heads", [(64, 8), (3, 1), (5, 5), (2, 2)])
@pytest.mark.parametrize("tokens,interleaved,bias", [(1, 0, True), (3, 1, True), (77, 0, False), (4103, 1, True)])
def test_prologue_codes_are_the_formats(heads, tokens, interleaved, bias):
    hq, hkv = heads
    if tokens > 1000 and hq > 5:
        hq, hkv = 4, 2
    rng = np.random.default_rng(tokens)
    width = (hq + 2 * hkv) * 64
    qkv = torch.from_numpy(rng.standard_normal((tokens, width)).astype(np.float32) * 3).bfloat16()
    b = torch.from_numpy(rng.standard_normal(width).astype(np.float32)).bfloat16() if bias else None
    pages = -(-tokens // 16) + 3
    slots = rng.permutation(pages * 16)[:tokens].astype(np.int32)
    pos = rng.integers(0, 5000, tokens).astype(np.int32)
    cache = rng.integers(0, 256, (pages, hkv, int4.BLOCK)).astype(np.uint8)
    want = cache.copy()
    rope = sa.rope_table(*sa.yarn_table(), 5000, device=DEV)
    tab = rope.cpu().numpy()[pos]
    x = qkv.float().numpy().reshape(tokens, -1, 64)
    if bias:
        x = x + b.float().numpy().reshape(-1, 64)
    qk = _rotated(x[:, :hq + hkv], tab[:, :32], tab[:, 32:], interleaved)
    skip = np.zeros(tokens, bool)
    if tokens > 2:                                       # no slot: nothing written
        slots[1], slots[2] = -1, pages * 16
        skip[1:3] = True
    int4.write(want, slots[~skip], qk[~skip, hq:], x[~skip, hq + hkv:])
    got = torch.from_numpy(cache).to(DEV)
    q = sa.qkv_prologue_int4(qkv.to(DEV), None if b is None else b.to(DEV), ints(pos), ints(slots), rope, got, hq,
                             hkv, rope_style=sa.ROPE_INTERLEAVED if interleaved else sa.ROPE_HALF)
    assert torch.equal(q.cpu(), torch.from_numpy(qk[:, :hq]).bfloat16())
    assert np.array_equal(got.cpu().numpy(), want)       # the other bytes among them


def test_prologue_odd_rows():
    # zeros, constants, one-sided, tiny, huge, not finite; positions outside of the table
    hkv = 2
    kinds = [lambda r: 0 * r, lambda r: 0 * r + 3, lambda r: -abs(r), lambda r: r * 1e-39, lambda r: r * 5e37,
             lambda r: r * 3e38, lambda r: np.where(np.arange(64) == 7, np.nan, r),
             lambda r: np.where(np.arange(64) == 63, np.inf, r), lambda r: np.where(np.arange(64) == 0, -np.inf, r),
             lambda r: r * 2.0**-120]
    rng = np.random.default_rng(0)
    t = len(kinds)
    qkv = np.stack([np.stack([f(np.clip(rng.standard_normal(64), -1, 1)) for _ in range(5 * 1)]) for f in kinds])
    qkv = torch.from_numpy(qkv.astype(np.float32)).bfloat16().reshape(t, 5 * 64)
    rope = torch.cat([torch.ones(4, 32), torch.zeros(4, 32)], 1).to(DEV)      # no rotation
    cache = sa.int4_cache(1, hkv, DEV)
    pos = ints([0, 1, 2, 3, 0, 0, 0, 0, 0, 0])
    q = sa.qkv_prologue_int4(qkv.to(DEV), None, pos, ints(list(range(t))), rope, cache, 1, hkv)
    k, v = (np64(x) for x in sa.gather_int4(cache, ints(list(range(t)))))
    x = qkv.float().numpy().reshape(t, 5, 64)
    with np.errstate(all="ignore"):
        turned = _rotated(x, np.ones((t, 32), np.float32), np.zeros((t, 32), np.float32), 0)
    np.testing.assert_array_equal(k, int4.round_trip(turned[:, 1:3]))
    np.testing.assert_array_equal(v, int4.round_trip(x[:, 3:]))
    assert np.isnan(k[5:9]).all() and np.isnan(v[6:9]).all() and not np.isnan(k[:5]).any()
    for p in (-1, 4, 2**31 - 1):
        q = sa.qkv_prologue_int4(qkv[:1].to(DEV) + 1, None, ints([p]), ints([3]), rope, cache, 1, hkv)
        k, v = sa.gather_int4(cache, ints([3]))
        assert torch.isnan(q).all() and torch.isnan(k).all()
        np.testing.assert_array_equal(np64(v), int4.round_trip(np.ones((1, hkv, 64))))


# ---------------------------------------------------------------------- gather
@pytest.mark.parametrize("hkv", [1, 3, 8])
def test_gather(hkv):
    c = Packed([1, 40, 33], hkv, hkv)
    cache = torch.from_numpy(c.cache).to(DEV)
    pick = np.concatenate(c.slots)[::-1].copy()
    k, v = sa.gather_int4(cache, ints(pick))
    np.testing.assert_array_equal(np64(k), np.concatenate(c.k)[::-1])
    np.testing.assert_array_equal(np64(v), np.concatenate(c.v)[::-1])
    odd = ints([-1, c.pages * 16, int(pick[0]), 2**31 - 1, -2**31])
    k, v = sa.gather_int4(cache, odd)
    for x, want in ((k, c.k), (v, c.v)):
        assert torch.isnan(x[[0, 1, 3, 4]]).all()
        np.testing.assert_array_equal(np64(x[2]), np.concatenate(want)[-1])
    k, v = sa.gather_int4(cache, ints([]))
    assert k.shape == v.shape == (0, hkv, 64)


# ---------------------------------------------------------------------- decode
def _decode_want(c, q):
    parts = [rows(np64(q[b:b + 1]), c.k[b], c.v[b], np.ones((1, n), bool), c.sinks, c.scale)
             for b, n in enumerate(c.lens)]
    return [np.concatenate(p) for p in zip(*parts)]


LENS = [0, 1, 2, 15, 16, 17, 31, 33, 47, 48, 64, 65, 128, 129, 300, 511, 700]


@pytest.mark.parametrize("heads", HEADS)
def test_decode(heads):
    c = Packed(LENS, *heads, seed=heads[0])
    q = c.q(len(LENS))
    want = _decode_want(c, q)
    args = (q.to(DEV), *c.gpu())
    first = sa.decode_int4(*args, c.max_kv)
    assert_rows(first, want)
    for kw in (dict(programmatic=True), dict(want_lse=False)):
        out, lse = sa.decode_int4(*args, c.max_kv, **kw)
        assert torch.equal(out, first[0]) and (lse is None or torch.equal(lse, first[1]))
    for bound in (5000, 2**40):                          # bounds need not be tight
        assert_rows(sa.decode_int4(*args, bound), want)


@pytest.mark.parametrize("lens", [[5000], [2500, 1, 2501], [40] * 600, [1] * 700 + [3000], [0] * 300, [0, 0, 90, 0] * 80])
def test_decode_shares(lens):
    # long units over many CTAs; units shorter than a share; more requests than the
    # scan has threads; empty ones between them
    c = Packed(lens, 8, 1, seed=len(lens))
    q = c.q(len(lens))
    args = (q.to(DEV), *c.gpu())
    first = sa.decode_int4(*args, c.max_kv)
    assert_rows(first, _decode_want(c, q))
    again = sa.decode_int4(*args, c.max_kv)
    assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])


def test_decode_large_scores_and_scales():
    # keys of large and of tiny rows, negative and zero scale, maxima that move late
    c = Packed([200, 90], 16, 2, seed=3, k_gain=1.0)
    for b in range(2):
        gain = np.exp(np.linspace(-4, 2, c.lens[b]))[:, None, None]
        k = c.rng.standard_normal((c.lens[b], 2, 64)) * gain
        c.put(c.slots[b], k, c.v[b])
        c.k[b], c.v[b] = int4.round_trip(k), int4.round_trip(c.v[b])
    q = c.q(2)
    cache, table, lens, sinks, _ = c.gpu()
    for scale in (0.125, -0.125, 0.0):
        c.scale = scale
        # rows of up to 4 e^2: eight times the scores that the bars are made for
        got = sa.decode_int4(q.to(DEV), cache, table, lens, sinks, scale, 200)
        out, lse, weight = _decode_want(c, q)
        bar = 1.05 * 2.0**-8 * (weight + np.abs(out)) + 2.0**-10 * weight + 2.0**-15
        assert (np.abs(np64(got[0]) - out) <= bar).all()
        assert (np.abs(np64(got[1]) - lse) <= 2.0**-10).all()


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
def test_odd_sinks(what):
    c = Packed([300, 0, 20], 8, 2)
    c.sinks[[2, 7]] = what
    q = c.q(3)
    got = sa.decode_int4(q.to(DEV), *c.gpu(), c.max_kv)
    fine = np.array([h not in (2, 7) for h in range(8)]) | (what == -np.inf)
    want = _decode_want(c, q)
    assert_rows([x[:, torch.from_numpy(fine).to(DEV)] for x in got], [x[:, fine] for x in want])
    if what != -np.inf:
        assert torch.isnan(got[0][:, [2, 7]]).all() and torch.isnan(got[1][:, [2, 7]]).all()


def test_requests_out_of_range_are_nan():
    c = Packed([40, 300, 17, 200], 16, 2, width_extra=0)
    q = c.q(4)
    want = _decode_want(c, q)
    cache, table, lens, sinks, scale = c.gpu()
    ok = np.arange(4) != 1
    for change in ("len", "table", "page", "negative page", "bound"):
        t, n, bound = table.clone(), lens.clone(), 300
        if change == "len":
            n[1] = -1
        elif change == "table":
            n[1] = 16 * table.shape[1] + 1
            bound = 5000
        elif change == "page":
            t[1, 18] = c.pages
        elif change == "negative page":
            t[1, 0] = -1
        else:
            bound = 299
        out, lse = sa.decode_int4(q.to(DEV), cache, t, n, sinks, scale, bound)
        assert torch.isnan(out[1]).all() and torch.isnan(lse[1]).all(), change
        assert_rows([out[ok], lse[ok]], [x[ok] for x in want], change)


def test_rows_that_are_not_finite_spoil_those_who_see_them():
    c = Packed([50, 50, 50], 8, 2)
    q = c.q(3)
    want = _decode_want(c, q)
    k, v = np.concatenate([a[None, 20] for a in c.k]), np.concatenate([a[None, 20] for a in c.v])
    k[1, 0], v[2, 1] = np.nan, np.nan
    c.put(np.array([s[20] for s in c.slots]), k, v)
    out, lse = sa.decode_int4(q.to(DEV), *c.gpu(), 50)
    assert_rows([out[0], lse[0]], [x[0] for x in want])
    assert torch.isnan(out[1, :4]).all() and torch.isnan(lse[1, :4]).all()
    assert torch.isnan(out[2, 4:]).all() and torch.isfinite(lse[2]).all()
    assert_rows([out[1, 4:], lse[1, 4:]], [x[1, 4:] for x in want])
    assert_rows([out[2, :4], lse[2, :4]], [x[2, :4] for x in want])


# ---------------------------------------------------------------- verification
def _verify_want(c, q, masks):
    parts = []
    for b, n in enumerate(c.lens):
        t = q.shape[1]
        seen = np.zeros((t, n), bool)
        for i in range(t):
            seen[i, :n - t] = True
            bits = (1 << i + 1) - 1 if masks is None else int(masks[b, i]) % (1 << 64)
            for u in range(t):
                seen[i, n - t + u] = bits >> u & 1
        parts.append(rows(np64(q[b]), c.k[b], c.v[b], seen, c.sinks, c.scale))
    return [np.stack(p) for p in zip(*parts)]


@pytest.mark.parametrize("heads", [(64, 8), (4, 1), (10, 2), (32, 2), (8, 8)])
@pytest.mark.parametrize("q_len", [1, 2, 3, 8, 17, 64])
@pytest.mark.parametrize("tree", [False, True])
def test_verify(heads, q_len, tree):
    if heads[0] * q_len > 600:
        heads = (heads[0] // heads[1], 1)
    lens = [q_len, q_len + 1, q_len + 15, q_len + 16, q_len + 40, 150 + q_len]
    c = Packed(lens, *heads, seed=q_len)
    q = c.q(len(lens), q_len)
    masks = workloads.random_tree_masks(c.rng, len(lens), q_len) if tree else None
    if tree and q_len > 2:
        masks[0, 1] = 0                                  # a row that sees no key at all
        masks[4, 2] = 0
    got = sa.verify_int4(q.to(DEV), *c.gpu(), c.max_kv, tree_mask=None if masks is None else masks.to(DEV))
    assert_rows(got, _verify_want(c, q, None if masks is None else masks.numpy()))


def test_hidden_drafts_may_be_anything():
    c = Packed([30, 30, 30], 8, 1)
    q = c.q(3, 4)
    masks = torch.tensor([[0b0001, 0b0011, 0b0100, 0b1100]] * 3)
    want = _verify_want(c, q, masks.numpy())
    k, v = np.stack([a[27] for a in c.k]), np.stack([a[27] for a in c.v])
    k[1], v[2] = np.nan, np.inf                          # draft 1: seen by row 1 alone
    c.put(np.array([s[27] for s in c.slots]), k, v)
    out, lse = sa.verify_int4(q.to(DEV), *c.gpu(), 30, tree_mask=masks.to(DEV))
    assert torch.isnan(out[1:, 1]).all() and torch.isnan(lse[1, 1]).all()
    rest = [0, 2, 3]
    assert_rows([out[:, rest], lse[:, rest]], [x[:, rest] for x in want])


def test_verify_shorter_than_its_tokens_is_nan():
    c = Packed([2, 3, 40], 8, 2)
    q = c.q(3, 3)
    out, lse = sa.verify_int4(q.to(DEV), *c.gpu(), 40)
    assert torch.isnan(out[0]).all() and torch.isnan(lse[0]).all() and torch.isfinite(out[1:]).all()


# --------------------------------------------------------------------- prefill
def _prefill_want(c, q, q_lens):
    parts, at = [], 0
    for b, (t, n) in enumerate(zip(q_lens, c.lens)):
        seen = np.arange(n)[None] <= n - t + np.arange(t)[:, None]
        parts.append(rows(np64(q[at:at + t]), c.k[b], c.v[b], seen, c.sinks, c.scale))
        at += t
    return [np.concatenate(p) for p in zip(*parts)]


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("q_lens,prefix", [([1, 40, 17], [0, 0, 0]), ([5, 1, 0, 33], [300, 16, 50, 127]),
                                           ([130, 3], [1, 260])])
def test_prefill(heads, q_lens, prefix):
    if heads[0] > 40 and sum(q_lens) > 100:
        heads = (16, 2)
    c = Packed([a + b for a, b in zip(q_lens, prefix)], *heads, seed=sum(q_lens))
    total = sum(q_lens)
    q = c.q(total + 5)
    cu = ints(np.concatenate([[0], np.cumsum(q_lens)]))
    cache, table, lens, sinks, scale = c.gpu()
    want = _prefill_want(c, q, q_lens)
    for bounds in ((max(q_lens), c.max_kv), (4000, 9000), (2**40, 2**40)):
        out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
        sa.prefill_paged_int4(q.to(DEV), cu, cache, table, lens, sinks, scale, *bounds, out=out, lse=lse)
        assert_rows([out[:total], lse[:total]], want)
        assert (out[total:] == 7).all() and (lse[total:] == 7).all()     # rows of nobody stay


def test_prefill_requests_out_of_range_are_nan():
    q_lens = [20, 30, 40]
    c = Packed([50, 30, 90], 8, 2, width_extra=0)
    q = c.q(90)
    want = _prefill_want(c, q, q_lens)
    cache, table, lens, sinks, scale = c.gpu()
    fine = np.r_[0:20, 50:90]
    for change in ("len", "page", "bound", "rows"):
        t, n, cu, bounds = table.clone(), lens.clone(), ints([0, 20, 50, 90]), (40, 90)
        rest, bad = fine, np.r_[20:50]
        if change == "len":
            n[1] = 29
        elif change == "page":
            t[1, 1] = c.pages + 7
        elif change == "bound":
            bounds, rest, bad = (30, 90), np.r_[0:50], np.r_[50:90]
        else:
            cu[3], rest, bad = 91, np.r_[0:50], np.r_[50:90]
        out, lse = sa.prefill_paged_int4(q.to(DEV), cu, cache, t, n, sinks, scale, *bounds)
        assert torch.isnan(out[bad]).all() and torch.isnan(lse[bad]).all(), change
        assert_rows([out[rest], lse[rest]], [x[rest] for x in want], change)
    out = torch.full_like(q.to(DEV), 7.0)
    sa.prefill_paged_int4(q.to(DEV), ints([0, 20, 50, 90]), cache, table, lens, sinks, scale, 0, 90, out=out)
    assert torch.isnan(out).all()


# ---------------------------------------------------------------- used together
def _serve(c, hq, hkv, steps, workspace, stream=None):
    """A prompt in two chunks, then tokens one by one, then a verification of three,
    each appended to the cache first.  Returns everything that the calls returned."""
    got = []
    for name, (qkv, pos, slots, kv_lens, cu) in steps.items():
        q = sa.qkv_prologue_int4(qkv, c["bias"], pos, slots, c["rope"], c["cache"], hq, hkv, stream=stream)
        paged = (c["cache"], c["table"], kv_lens, c["sinks"], 0.125)
        kw = dict(workspace=workspace, stream=stream)
        if cu is not None:
            got += sa.prefill_paged_int4(q, cu, *paged, 200, 400, **kw)
        elif name.startswith("verify"):
            got += sa.verify_int4(q.view(2, 3, hq, 64), *paged, 400, programmatic=True, **kw)
        else:
            got += sa.decode_int4(q, *paged, 400, programmatic=True, **kw)
    got += sa.gather_int4(c["cache"], steps["chunk 1"][2], stream=stream)
    return got


def test_a_session_eager_captured_and_on_another_stream():
    hq, hkv = 16, 2
    rng = np.random.default_rng(5)
    chunks = [("chunk 0", [100, 60]), ("chunk 1", [77, 31])] + [(f"token {i}", [1, 1]) for i in range(3)] + [("verify", [3, 3])]
    pages = rng.permutation(60)
    table = ints(np.stack([pages[:25], pages[25:50]]))
    c = dict(bias=torch.randn(20 * 64, device=DEV).bfloat16(), rope=sa.rope_table(*sa.yarn_table(), 400, device=DEV),
             cache=sa.int4_cache(60, hkv, DEV), table=table, sinks=torch.randn(hq, device=DEV))
    have, steps, past, oracle_q = [0, 0], {}, [], []
    for name, new in chunks:
        pos = np.concatenate([np.arange(h, h + n) for h, n in zip(have, new)])
        req = np.repeat([0, 1], new)
        slots = np.array([int(pages[25 * r + p // 16]) * 16 + p % 16 for r, p in zip(req, pos)])
        have = [h + n for h, n in zip(have, new)]
        qkv = torch.from_numpy(rng.standard_normal((len(pos), 20 * 64)).astype(np.float32)).bfloat16().to(DEV)
        steps[name] = (qkv, ints(pos), ints(slots), ints(have), ints([0, new[0], sum(new)]) if "chunk" in name else None)
        past.append((list(have), new))
    w = torch.zeros(sa.int4_workspace_bytes(), dtype=torch.uint8, device=DEV)
    want = _serve(c, hq, hkv, steps, w)
    torch.cuda.synchronize()

    # against float64 attention over what the cache stands for after each step
    for i, (name, step) in enumerate(steps.items()):
        q = sa.qkv_prologue_int4(step[0], c["bias"], step[1], step[2], c["rope"], c["cache"], hq, hkv)
        out, lse = (x.reshape(-1, *x.shape[2:]) if name == "verify" else x for x in want[2 * i:2 * i + 2])
        at = 0
        for b in range(2):
            n, t = past[i][0][b], past[i][1][b]
            every = np.array([int(pages[25 * b + p // 16]) * 16 + p % 16 for p in range(n)])
            k, v = (np64(x) for x in sa.gather_int4(c["cache"], ints(every)))
            seen = np.arange(n)[None] <= n - t + np.arange(t)[:, None]
            ref = rows(np64(q[at:at + t]), k, v, seen, np64(c["sinks"]), 0.125)
            # q and k rows carry the rotation's factor 1.35 each and a bias of their own
            # size: scores four times those that the bars are made for
            bar = 1.05 * 2.0**-8 * (ref[2] + np.abs(ref[0])) + 2.0**-11 * ref[2] + 2.0**-15
            assert (np.abs(np64(out[at:at + t]) - ref[0]) <= bar).all(), name
            assert (np.abs(np64(lse[at:at + t]) - ref[1]) <= 2.0**-11).all(), name
            at += t

    def same(got):
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)

    side = torch.cuda.Stream()
    c["cache"].fill_(255)
    torch.cuda.synchronize()
    same(_serve(c, hq, hkv, steps, None, stream=side))
    graph = torch.cuda.CUDAGraph()
    c["cache"].fill_(255)
    with torch.cuda.graph(graph):
        got = _serve(c, hq, hkv, steps, w)
    for _ in range(3):
        c["cache"].fill_(255)
        for x in got:
            x.fill_(3)
        graph.replay()
        same(got)


def test_a_packed_cache_is_a_bf16_cache_of_its_values():
    # the operators of the bf16 cache on the values: within the roundings of both
    c = Packed([100, 333, 16, 1], 64, 8)
    q = c.q(4)
    cache, table, lens, sinks, scale = c.gpu()
    k, v = (torch.from_numpy(np.nan_to_num(x)).bfloat16().to(DEV) for x in c.values())
    a = sa.decode(q.to(DEV), k, v, table, lens, sinks, scale, 333)
    b = sa.decode_int4(q.to(DEV), cache, table, lens, sinks, scale, 333)
    _, _, weight = _decode_want(c, q)
    bar = 2.1 * 2.0**-8 * (weight + np.abs(np64(a[0]))) + 2.0**-12 * weight + 2.0**-14
    assert (np.abs(np64(a[0]) - np64(b[0])) <= bar).all()
    assert (np64(a[1]) - np64(b[1])).max() <= 2.0**-12


def test_one_workspace_serves_every_call():
    # of any form, batch and heads, and those of the bf16 cache in between
    shared = torch.zeros(max(sa.int4_workspace_bytes(), 64 << 20), dtype=torch.uint8, device=DEV)
    for seed, (lens, heads, q_len) in enumerate([([4000, 17], (64, 8), 1), ([900] * 9, (10, 2), 4), ([50] * 300, (8, 8), 1),
                                                 ([6000], (4, 1), 2), ([300, 3000], (32, 2), 8), ([4000, 17], (64, 8), 1)]):
        rng = np.random.default_rng(seed)
        pages = sum(-(-n // 16) for n in lens)
        cache = sa.int4_cache(pages, heads[1], DEV)
        ids, table, slots = iter(rng.permutation(pages)), np.zeros((len(lens), -(-max(lens) // 16)), np.int32), []
        for b, n in enumerate(lens):
            for i in range(-(-n // 16)):
                table[b, i] = next(ids)
            slots += [table[b, p // 16] * 16 + p % 16 for p in range(n)]
        gen = torch.Generator(DEV).manual_seed(seed)
        qkv = torch.randn(len(slots), (heads[0] + 2 * heads[1]) * 64, generator=gen, device=DEV).bfloat16()
        sa.qkv_prologue_int4(qkv, None, ints([0] * len(slots)), ints(slots), sa.rope_table([0.0] * 32, 1.0, 1, DEV), cache, *heads)
        q = torch.randn(len(lens), q_len, heads[0], 64, generator=gen, device=DEV).bfloat16()
        rest = (ints(table), ints(lens), torch.zeros(heads[0], device=DEV), 0.125, max(lens))
        k, v = (torch.zeros(pages, heads[1], 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        for _ in range(2):
            want = sa.verify_int4(q, cache, *rest)
            out, lse = torch.full_like(want[0], 7.0), torch.full_like(want[1], 7.0)
            sa.verify_int4(q, cache, *rest, workspace=shared, out=out, lse=lse)
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])
            cu = ints([q_len * i for i in range(len(lens) + 1)])
            flat = q.view(-1, heads[0], 64)
            want = sa.prefill_paged_int4(flat, cu, cache, *rest[:4], q_len, max(lens))
            got = sa.prefill_paged_int4(flat, cu, cache, *rest[:4], q_len, max(lens), workspace=shared)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
            want = sa.verify(q, k, v, *rest, num_splits=5)
            got = sa.verify(q, k, v, *rest, num_splits=5, workspace=shared)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_with_nothing_to_do():
    c = Packed([20], 8, 2)
    cache, table, lens, sinks, scale = c.gpu()
    empty = torch.zeros(0, 8, 64, dtype=torch.bfloat16, device=DEV)
    out, lse = sa.decode_int4(empty, cache, table[:0], lens[:0], sinks, scale, 20)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    out, lse = sa.prefill_paged_int4(empty, ints([0, 0]), cache, table, lens, sinks, scale, 4, 20)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)


def test_workspaces_that_do_not_fit_are_refused():
    c = Packed([20], 8, 2)
    q = c.q(1).to(DEV)
    need = sa.int4_workspace_bytes()
    with pytest.raises(sa.SinkAttnError) as e:
        sa.decode_int4(q, *c.gpu(), 20, workspace=torch.zeros(need - 1, dtype=torch.uint8, device=DEV))
    assert e.value.status == sa.WORKSPACE_TOO_SMALL
    with pytest.raises(sa.SinkAttnError) as e:
        sa.decode_int4(q, *c.gpu(), 20, workspace=torch.zeros(need + 16, dtype=torch.uint8, device=DEV)[16:])
    assert e.value.status == sa.INVALID_ARGUMENT


# ------------------------------------------- both attention kernels, odd arguments
@pytest.mark.parametrize("bound", [12, 500])             # few rows; tensor cores
def test_sequences_that_fall_back_are_nan(bound):
    c = Packed([40, 40, 40, 40], 8, 2)
    q = c.q(24)
    cache, table, lens, sinks, scale = c.gpu()
    # request 1 ends before it starts, request 2 starts before request 1 does
    out, lse = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV), torch.full(q.shape[:2], 7.0, device=DEV)
    sa.prefill_paged_int4(q.to(DEV), ints([10, 20, 3, 8, 10]), cache, table, lens, sinks, scale, bound, 40, out=out,
                          lse=lse)
    for b, a, e in ((0, 10, 20), (3, 8, 10)):
        seen = np.arange(40)[None] <= 40 - (e - a) + np.arange(e - a)[:, None]
        assert_rows([out[a:e], lse[a:e]], rows(np64(q[a:e]), c.k[b], c.v[b], seen, c.sinks, c.scale))
    assert torch.isnan(out[3:8]).all() and torch.isnan(lse[3:8]).all()
    rest = [0, 1, 2, 20, 21, 22, 23]
    assert (out[rest] == 7).all() and (lse[rest] == 7).all()


@pytest.mark.parametrize("q_len", [4, 40])               # 16 rows; 160 rows: tensor cores
def test_hidden_drafts_of_either_kernel_may_be_anything(q_len):
    n = 130 + q_len
    c = Packed([n, n, n], 4, 1)
    q = c.q(3, q_len)
    masks = workloads.random_tree_masks(c.rng, 3, q_len) & ~(1 << 2)
    masks[:, 2] |= 1 << 2                                # draft 2 is seen by its own row alone
    k, v = np.stack([a[132] for a in c.k]), np.stack([a[132] for a in c.v])
    c.k[0][132], c.v[0][132] = int4.round_trip(k[0]), int4.round_trip(v[0])      # quantised once more
    want = _verify_want(c, q, masks.numpy())
    k[1], v[2] = np.nan, np.inf
    c.put(np.array([s[132] for s in c.slots]), k, v)
    out, lse = sa.verify_int4(q.to(DEV), *c.gpu(), n, tree_mask=masks.to(DEV))
    assert torch.isnan(out[1:, 2]).all() and torch.isnan(lse[1, 2]).all()
    rest = [i for i in range(q_len) if i != 2]
    assert_rows([out[:, rest], lse[:, rest]], [x[:, rest] for x in want])
    assert_rows([out[0], lse[0]], [x[0] for x in want])


@pytest.mark.parametrize("what", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("q_lens", [[3, 7], [90, 300]])  # few rows; tensor cores
def test_odd_sinks_and_rows_of_prompts(q_lens, what):
    c = Packed(q_lens, 8, 2, seed=3)
    q = c.q(sum(q_lens))
    c.sinks[1] = what
    cu = ints([0, q_lens[0], sum(q_lens)])
    want = _prefill_want(c, q, q_lens) if what == -float("inf") else None
    c.sinks[1] = 0.0
    plain = _prefill_want(c, q, q_lens)
    c.sinks[1] = what
    args = c.gpu()
    out, lse = sa.prefill_paged_int4(q.to(DEV), cu, *args, max(q_lens), max(q_lens))
    other = [h for h in range(8) if h != 1]
    assert_rows([out[:, other], lse[:, other]], [x[:, other] for x in plain])
    if want is not None:
        assert_rows([out[:, 1], lse[:, 1]], [x[:, 1] for x in want])
    else:
        assert torch.isnan(out[:, 1]).all() and torch.isnan(lse[:, 1]).all()
    # a value row that is not finite: those before it do not see it
    k, v = np.array(c.k[1][2][None]), np.array(c.v[1][2][None])
    c.k[1][2], c.v[1][2] = int4.round_trip(k[0]), int4.round_trip(v[0])          # quantised once more
    c.sinks[1] = 0.0
    plain = _prefill_want(c, q, q_lens)
    v[0, 1] = np.nan
    c.put(np.array([c.slots[1][2]]), k, v)
    out2, lse2 = sa.prefill_paged_int4(q.to(DEV), cu, c.gpu()[0], *args[1:], max(q_lens), max(q_lens))
    start = q_lens[0] + 2
    assert torch.isnan(out2[start:, 4:]).all()
    assert_rows([out2[:start, 4:], lse2[:start, 4:]], [x[:start, 4:] for x in plain])
    assert_rows([out2[:, other[:3]], lse2[:, other[:3]]], [x[:, other[:3]] for x in plain])


# ------------------------------------------------- keys in parts (many rows, long caches)
def _parts_case(seed=5):
    # 48 rows per KV head; 1 .. 40 key tiles, one request of a single page
    q_lens, prefix = [6, 6, 1, 6, 3], [5003, 1500, 2100, 0, 770]
    c = Packed([a + b for a, b in zip(q_lens, prefix)], 16, 2, seed=seed)
    return c, q_lens, c.q(sum(q_lens)), ints(np.concatenate([[0], np.cumsum(q_lens)]))


def test_parts_of_long_caches():
    c, q_lens, q, cu = _parts_case()
    want = _prefill_want(c, q, q_lens)
    ws = torch.zeros(sa.int4_workspace_bytes(), dtype=torch.uint8, device=DEV)
    first = None
    for bounds in ((6, c.max_kv), (60, 9000), (2**40, 2**40)):
        got = sa.prefill_paged_int4(q.to(DEV), cu, *c.gpu(), *bounds, workspace=ws)
        assert_rows(got, want, str(bounds))
        assert not ws[:16384].any()                      # ready for the next call
        again = sa.prefill_paged_int4(q.to(DEV), cu, *c.gpu(), *bounds, workspace=ws)
        assert all(torch.equal(a, b) for a, b in zip(got, again))
        first = first or got


@pytest.mark.parametrize("tree", [False, True])
@pytest.mark.parametrize("heads", [(16, 2), (12, 1), (40, 1), (8, 8)])
def test_parts_of_verifications(heads, tree):
    q_len = 64 if heads == (8, 8) else 9
    lens = [3000, 600, q_len, 1100 + q_len]
    c = Packed(lens, *heads, seed=11)
    q = c.q(4, q_len)
    c.sinks[0] = -np.inf
    masks = workloads.random_tree_masks(c.rng, 4, q_len) if tree else None
    got = sa.verify_int4(q.to(DEV), *c.gpu(), c.max_kv, tree_mask=None if masks is None else masks.to(DEV))
    assert_rows(got, _verify_want(c, q, None if masks is None else masks.numpy()))


def test_parts_with_bad_pages_values_and_lengths():
    c, q_lens, q, cu = _parts_case(6)
    want = _prefill_want(c, q, q_lens)
    cache, table, lens, sinks, scale = c.gpu()
    ws = torch.zeros(sa.int4_workspace_bytes(), dtype=torch.uint8, device=DEV)
    for change in ("first page", "middle page", "last page", "length"):
        t, n = table.clone(), lens.clone()
        if change == "length":
            n[0] = -3
        else:
            t[0, {"first page": 0, "middle page": 150, "last page": 312}[change]] = c.pages
        out, lse = sa.prefill_paged_int4(q.to(DEV), cu, cache, t, n, sinks, scale, 6, c.max_kv, workspace=ws)
        assert torch.isnan(out[:6]).all() and torch.isnan(lse[:6]).all(), change
        assert_rows([out[6:], lse[6:]], [x[6:] for x in want], change)
        assert not ws[:16384].any()
    k, v = np.array(c.k[0][2500][None]), np.array(c.v[0][2500][None])
    v[0, 1] = np.inf
    c.put(np.array([c.slots[0][2500]]), k, v)
    out, lse = sa.prefill_paged_int4(q.to(DEV), cu, *c.gpu(), 6, c.max_kv, workspace=ws)
    assert torch.isnan(out[:6, 8:]).all() and torch.isfinite(out[:6, :8]).all()
    assert_rows([out[6:], lse[6:]], [x[6:] for x in want])


def test_parts_captured_and_among_overlapping_sequences():
    c, q_lens, q, cu = _parts_case(7)
    want = _prefill_want(c, q, q_lens)
    ws = torch.zeros(sa.int4_workspace_bytes(), dtype=torch.uint8, device=DEV)
    args, q_dev = c.gpu(), q.to(DEV)
    graph = torch.cuda.CUDAGraph()
    sa.prefill_paged_int4(q_dev, cu, *args, 6, c.max_kv, workspace=ws)
    with torch.cuda.graph(graph):
        got = sa.prefill_paged_int4(q_dev, cu, *args, 6, c.max_kv, workspace=ws)
    for _ in range(3):
        graph.replay()
    assert_rows(got, want)
    # sequences that overlap hold more rows than there are: rows may be anyone's, the
    # workspace is as it was, and the next call is right
    many = torch.tensor([0, 22, 0, 0, 22, 0, 0, 22, 0, 0, 22], dtype=torch.int32, device=DEV)
    wide = [args[1].repeat(2, 1), args[2].repeat(2)]
    sa.prefill_paged_int4(q_dev, many, args[0], *wide, *args[3:], 40, c.max_kv, workspace=ws)
    assert not ws[:16384].any()
    assert_rows(sa.prefill_paged_int4(q_dev, cu, *args, 6, c.max_kv, workspace=ws), want)


@pytest.mark.parametrize("q_len", [3, 9, 63, 64])
def test_bits_past_the_drafts_mean_nothing(q_len):
    n = 700 + q_len
    c = Packed([n, q_len, n + 20], 4, 1, seed=q_len)
    q = c.q(3, q_len)
    masks = workloads.random_tree_masks(c.rng, 3, q_len)
    want = _verify_want(c, q, masks.numpy())
    past = -(1 << q_len) if q_len < 64 else 0
    got = sa.verify_int4(q.to(DEV), *c.gpu(), c.max_kv, tree_mask=(masks | past).to(DEV))
    assert_rows(got, want)


def test_the_same_rows_again_and_slots_shared_between_requests():
    # two requests over the same pages, a page twice in one request
    c = Packed([64, 64], 8, 2)
    q = c.q(2)
    cache, table, lens, sinks, scale = c.gpu()
    table[1] = table[0]
    table[1, 2] = table[0, 1]
    order = np.r_[0:32, 16:32, 48:64]
    want = [rows(np64(q[b:b + 1]), c.k[0][o], c.v[0][o], np.ones((1, 64), bool), c.sinks, c.scale)
            for b, o in enumerate((np.arange(64), order))]
    got = sa.decode_int4(q.to(DEV), cache, table, lens, sinks, scale, 64)
    assert_rows(got, [np.concatenate(p) for p in zip(*want)])
    k, v = sa.gather_int4(cache, ints([int(c.slots[0][5])] * 3 + [-1, 16 * c.pages]))
    assert torch.equal(k[0], k[2]) and torch.equal(v[1], v[2]) and torch.isnan(k[3:]).all() and torch.isnan(v[3:]).all()
    assert (np64(k[0]) == c.k[0][5]).all()


def test_pages_past_four_gigabytes():
    q_lens = [70, 3, 1]
    c = Packed([700, 90, 33], 16, 8, spare=0)
    q, q1 = c.q(sum(q_lens)).to(DEV), c.q(3).to(DEV)
    cache, table, lens, sinks, scale = c.gpu()
    pages = 2**32 // (8 * sa.INT4_BLOCK_BYTES) + 5000
    large = torch.empty(pages, 8, sa.INT4_BLOCK_BYTES, dtype=torch.uint8, device=DEV)
    large[-c.pages:] = cache
    far = torch.where(table >= 0, table + (pages - c.pages), table)
    cu = ints(np.concatenate([[0], np.cumsum(q_lens)]))
    slots = ints(c.slots[0][:50])

    def everything(cache, table, first):
        got = list(sa.decode_int4(q1, cache, table, lens, sinks, scale, 700))
        got += sa.verify_int4(q[:6].view(3, 2, 16, 64), cache, table, lens, sinks, scale, 700)
        got += sa.prefill_paged_int4(q, cu, cache, table, lens, sinks, scale, 70, 700)
        got += sa.gather_int4(cache, slots + 16 * first)
        qkv = q[:8].reshape(8, -1).repeat(1, 2)          # 16 + 2 * 8 heads
        got += [sa.qkv_prologue_int4(qkv, None, ints(range(8)), slots[:8] + 16 * first,
                                     torch.ones(8, 64, device=DEV), cache, 16, 8)]
        return got + list(sa.gather_int4(cache, slots + 16 * first))

    for a, b in zip(everything(large, far, pages - c.pages), everything(cache, table, 0)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))


def test_two_streams_with_a_workspace_each():
    c, q_lens, q, cu = _parts_case(8)
    want = _prefill_want(c, q, q_lens)
    args, q_dev = c.gpu(), q.to(DEV)
    q1 = c.q(len(q_lens))
    want1 = _decode_want(c, q1)
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [torch.zeros(sa.int4_workspace_bytes(), dtype=torch.uint8, device=DEV) for _ in range(2)]
    q1_dev = q1.to(DEV)
    torch.cuda.synchronize()
    got = []
    for _ in range(6):
        for stream, ws in zip(streams, spaces):
            got.append((sa.prefill_paged_int4(q_dev, cu, *args, 6, c.max_kv, workspace=ws, stream=stream),
                        sa.decode_int4(q1_dev, *args, c.max_kv, workspace=ws, stream=stream)))
    torch.cuda.synchronize()
    for p, d in got:
        assert_rows(p, want)
        assert_rows(d, want1)


@pytest.mark.parametrize("requests,hkv", [(33, 1), (100, 2), (200, 1), (700, 2)])
def test_prompts_of_many_requests(requests, hkv):
    rng = np.random.default_rng(requests)
    q_lens = [int(x) for x in rng.integers(0, 6, requests)]
    lens = [t + int(x) for t, x in zip(q_lens, rng.integers(0, 40, requests))]
    q_lens[requests - 2], lens[requests - 2] = 4, 2604       # keys in parts where CTAs are few
    q_lens[0], lens[0] = 0, 0
    c = Packed(lens, 4 * hkv, hkv, seed=requests)
    q = c.q(sum(q_lens))
    cu = ints(np.concatenate([[0], np.cumsum(q_lens)]))
    got = sa.prefill_paged_int4(q.to(DEV), cu, *c.gpu(), 40, c.max_kv)
    assert_rows(got, _prefill_want(c, q, q_lens))
