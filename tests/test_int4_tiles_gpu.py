"""Attention over a paged cache held in 4 bits where its kernels' rings go round: prompts
of many key tiles with both query tiles in use, long parts; batches with requests that
have no new tokens, what loose bounds and odd sequences ask of the plan, and the largest
values.

Compared with float64 on the GPU over what the cache stands for (`gather_int4`, whose
rows tests/test_int4_gpu.py compares with the format's, exactly)."""

import numpy as np
import pytest
import torch

import gqa_attention_learned_gb300 as sa
from gqa_attention_learned_gb300 import workloads
from int4_inputs import DEV
from oracle import int4
from test_int4_range_cpu import rows_at_the_top

pytestmark = pytest.mark.gpu

COUNTERS = 16384                 # bytes that a workspace begins with
SLOT = 256 * 64 * 4              # bytes of one CTA's sums after them (more than 32 rows per KV head)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


class Batch:
    """Requests of kv_lens keys, of which the last q_lens are new tokens, on shuffled
    pages; keys grow by e^gain from a request's first to its last.  Free slots hold
    bytes of 255 (scales that are NaN)."""

    def __init__(self, q_lens, kv_lens, hq, hkv, seed=0, gain=0.0, sinks=True, v_gain=1.0):
        self.q_lens, self.kv_lens, self.hq, self.hkv = q_lens, kv_lens, hq, hkv
        gen = torch.Generator(DEV).manual_seed(seed)
        need = [-(-n // 16) for n in kv_lens]
        pages = sum(need) + 3
        ids = torch.randperm(pages, generator=gen, device=DEV).int()
        self.table = torch.full((len(kv_lens), max(need + [1])), -1, dtype=torch.int32, device=DEV)
        self.cache = torch.full((pages, hkv, sa.INT4_BLOCK_BYTES), 255, dtype=torch.uint8, device=DEV)
        self.slots, at = [], 0
        rope = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).to(DEV)       # no rotation
        for b, n in enumerate(kv_lens):
            self.table[b, :need[b]] = mine = ids[at:at + need[b]]
            at += need[b]
            j = torch.arange(n, device=DEV)
            slots = (mine[j // 16] * 16 + j % 16).int()
            kv = torch.randn(n, 2, hkv, 64, generator=gen, device=DEV)
            kv[:, 0] *= torch.exp(gain * j / max(n - 1, 1))[:, None, None]
            kv[:, 1] = v_gain * (kv[:, 1] + 0.25)
            qkv = torch.cat([torch.zeros(n, 64, device=DEV), kv.flatten(1)], 1).bfloat16()
            sa.qkv_prologue_int4(qkv, None, torch.zeros_like(slots), slots, rope, self.cache, 1, hkv)
            self.slots.append(slots)
        self.lens = ints(kv_lens)
        self.cu = ints(np.concatenate([[0], np.cumsum(q_lens)]))
        self.q = torch.randn(sum(q_lens), hq, 64, generator=gen, device=DEV).bfloat16()
        self.sinks = 2 * torch.randn(hq, generator=gen, device=DEV) if sinks else torch.full((hq,), -torch.inf, device=DEV)
        self.scale = 0.125
        self.args = (self.cache, self.table, self.lens, self.sinks, self.scale)

    def attend(self, max_q=None, max_kv=None, **kw):
        return sa.prefill_paged_int4(self.q, self.cu, *self.args, max_q or max(self.q_lens),
                                     max_kv or max(self.kv_lens), **kw)

    def check(self, got, masks=None, few=False):
        """Every row against float64.  Where the bars come from: the weights are rounded to
        bf16 (2^-8 of their value at most) and the output once more; 5% on top for the second
        order.  A score is an fp32 sum of 64 exact products, each addition cut at 2^-23 of what
        there is by then: off by at most d = 2^-17 scale sum |q k|.  The kernel of few rows
        (`few`) adds up q (16 + n), takes (16 + z) sum q off it and multiplies by the step s:
        2^-17 for either, of 31 s sum |q|; s is at most 0.15 of the row's largest number
        before quantisation, which its largest value reaches within s: s <= max |k| / 5.6.  Scores
        off by d move the output by sum p |v| d + sum p |v| sum p d, and the lse by sum p d.
        2^-13 for what fp32 adds over some thousand keys (16 at a time, each time cut at 2^-23:
        2^-14 for 8192) and the exponential (2^-22, its argument below 64 rounded at 2^-24)."""
        out, lse = (x.double().reshape(-1, *x.shape[-k:]) for x, k in zip(got, (2, 1)))
        assert torch.isfinite(out).all()
        at = 0
        for b, (t, n) in enumerate(zip(self.q_lens, self.kv_lens)):
            if t == 0:
                continue
            k, v = (x.double().repeat_interleave(self.hq // self.hkv, 1) for x in sa.gather_int4(self.cache, self.slots[b]))
            q = self.q[at:at + t].double()
            seen = torch.arange(n, device=DEV) <= n - t + torch.arange(t, device=DEV)[:, None]
            if masks is not None:
                bits = masks[b][:, None] >> torch.arange(t, device=DEV) & 1
                seen[:, n - t:] = bits.bool()
            s = self.scale * torch.einsum("ihd,jhd->hij", q, k)
            s.masked_fill_(~seen, -torch.inf)
            sink = self.sinks.double()[:, None]
            top = torch.logaddexp(torch.logsumexp(s, 2), sink)
            p = torch.exp(s - top[:, :, None])
            ref, weight = (torch.einsum("hij,jhd->ihd", p, x) for x in (v, v.abs()))
            if few:
                d = 2.0**-16 * self.scale * 31 * torch.einsum("ih,jh->hij", q.abs().sum(2), k.abs().amax(2) / 5.6)
            else:
                d = 2.0**-17 * self.scale * torch.einsum("ihd,jhd->hij", q.abs(), k.abs())
            p *= d
            moved, d = torch.einsum("hij,jhd->ihd", p, v.abs()), p.sum(2).T
            bar = 1.05 * 2.0**-8 * (weight + ref.abs()) + 2.0**-13 * weight + moved + d[:, :, None] * weight
            err = (out[at:at + t] - ref).abs()
            assert (err <= bar).all(), f"request {b}: {(err / bar).max():.2f} of the bar"
            off = (lse[at:at + t] - top.T).abs()
            assert (off <= d + 2.0**-13).all(), f"request {b}: lse off by {off.max():.1e}"
            at += t


def workspace():
    """Zeros where a workspace has to hold them, a pattern in the rest."""
    w = torch.full((sa.int4_workspace_bytes(),), 0x5A, dtype=torch.uint8, device=DEV)
    w[:COUNTERS] = 0
    return w


def parts(w):
    """CTAs that left sums in a workspace; its counters are zero again."""
    assert not w[:COUNTERS].any()
    rest = w[COUNTERS:]
    rest = rest[:rest.numel() // SLOT * SLOT].view(-1, SLOT)
    return int((rest != 0x5A).any(1).sum())


def sms():
    return torch.cuda.get_device_properties(DEV).multi_processor_count


# A CTA takes 2 * (128 // group) tokens; calls with more than two CTAs per SM are not cut
# into parts.  16 tokens to a query tile: prefixes of 16 mod 32 put every fourth CTA's
# tiles on both sides of a key tile's end, so that the second has one more.
@pytest.mark.parametrize("q_lens,prefix,heads", [([1300], [1488], (64, 8)), ([1290, 45], [1500, 2000], (64, 8)),
                                                 ([700], [1700], (128, 1)), ([5000], [0], (8, 8)),
                                                 ([2001], [1600], (48, 8))])
@pytest.mark.parametrize("gain", [0.0, 2.0])
def test_prompts_of_many_key_tiles(q_lens, prefix, heads, gain):
    tokens = 2 * (128 // (heads[0] // heads[1]))
    blocks = sum(-(-t // tokens) for t in q_lens)
    if heads != (8, 8):
        assert blocks * heads[1] > 2 * sms()             # not in parts
    b = Batch(q_lens, [t + p for t, p in zip(q_lens, prefix)], *heads, seed=1, gain=gain)
    w = workspace()
    got = b.attend(workspace=w)
    assert heads == (8, 8) or parts(w) == 0
    b.check(got)
    again = b.attend(workspace=w, max_q=2**40, max_kv=2**40)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


@pytest.mark.parametrize("gain", [0.0, 2.0, -2.0])
@pytest.mark.parametrize("sinks", [True, False])
def test_long_parts(gain, sinks):
    # both query tiles of every CTA full; parts of more key tiles than the rings hold
    q_lens, kv_lens = [64, 64, 64, 50], [8000, 7777, 8100, 6000]
    b = Batch(q_lens, kv_lens, 64, 8, seed=2, gain=gain, sinks=sinks)
    w = workspace()
    got = b.attend(workspace=w)
    n = parts(w)
    blocks = 8 * sum(-(-t // 32) for t in q_lens)
    assert n > blocks                                    # cut
    assert sum(8 * -(-t // 32) * -(-k // 128) for t, k in zip(q_lens, kv_lens)) / n > 6      # tiles of a part
    b.check(got)
    again = b.attend(workspace=w)
    assert all(torch.equal(x, y) for x, y in zip(got, again))


def test_short_parts_leave_their_mark_and_do_not_depend_on_bounds():
    b = Batch([6, 6, 1, 6, 3], [5009, 1506, 2101, 6, 773], 16, 2, seed=3)
    first = None
    for max_q, max_kv in ((6, 5009), (60, 9000), (2**40, 2**40)):
        w = workspace()
        got = b.attend(workspace=w, max_q=max_q, max_kv=max_kv)
        assert parts(w) > 10
        b.check(got)
        first = first or got
        assert all(torch.equal(x, y) for x, y in zip(got, first))


@pytest.mark.parametrize("q_len,tree", [(8, False), (8, True), (3, True), (1, False), (64, True)])
def test_rows_of_long_caches(q_len, tree):
    # verification, and one token, on what the format's own tests do not reach in length
    kv_lens = [9000 + q_len, 300 + q_len, q_len, 5000]
    b = Batch([q_len] * 4, kv_lens, 64, 8, seed=4, gain=1.0)
    masks = workloads.random_tree_masks(np.random.default_rng(0), 4, q_len).to(DEV) if tree else None
    q = b.q.view(4, q_len, 64, 64)
    for bound in (max(kv_lens), 2**40):
        b.check(sa.verify_int4(q, *b.args, bound, tree_mask=masks), masks, few=8 * q_len <= 32)
    if q_len == 1:
        b.check(sa.decode_int4(b.q, *b.args, max(kv_lens)), few=True)


def test_the_lse_is_that_of_a_bf16_cache():
    # on both sides of it (fp32 sums of the same exact products, some 2^-17 apart)
    kv_lens = [100, 333, 16, 1]
    b = Batch([1] * 4, kv_lens, 64, 8, seed=5)
    pools = [torch.zeros(b.cache.shape[0], 8, 16, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    for slots in b.slots:
        for pool, rows in zip(pools, sa.gather_int4(b.cache, slots)):
            pool[slots.long() // 16, :, slots.long() % 16] = rows
    want = sa.decode(b.q, *pools, *b.args[1:], 333)
    got = sa.decode_int4(b.q, *b.args, 333)
    assert ((got[1] - want[1]).abs() <= 2.0**-12).all()


# ------------------------------------------------------------- the plan's arguments
def test_requests_without_new_tokens_are_no_work():
    # 20 short requests want no parts, however long the cache of one that is idle
    q_lens, kv_lens = [6] * 20 + [0] + [6] * 4, [1000] * 20 + [100000] + [700] * 4
    b = Batch(q_lens, kv_lens, 16, 2, seed=6)
    keep = [i for i in range(25) if i != 20]
    w = workspace()
    got = b.attend(workspace=w)
    assert parts(w) == 0
    b.check(got)
    alone = sa.prefill_paged_int4(b.q, ints(6 * np.arange(25)), b.cache, b.table[keep].contiguous(),
                                  b.lens[keep].contiguous(), b.sinks, b.scale, 6, 1000)
    assert all(torch.equal(x, y) for x, y in zip(got, alone))


@pytest.mark.parametrize("heads", [(256, 1), (512, 2), (64, 8)])
def test_bounds_on_new_tokens_need_not_be_tight(heads):
    # groups of more than 128 heads have a kernel of their own, whatever the rows
    b = Batch([3, 0, 2], [400, 20, 18], *heads, seed=7)
    for max_q in (3, 5, 100, 100000, 2**40):
        b.check(b.attend(max_q=max_q, max_kv=2**40), few=True)


def test_many_prompts_of_a_large_group():
    # row blocks are few beside requests times the longest of them, and the page table is wide
    q_lens = [1, 700] + [1] * 300
    b = Batch(q_lens, [t + 20 for t in q_lens], 256, 1, seed=10)
    wide = torch.full((len(q_lens), 200000), -1, dtype=torch.int32, device=DEV)
    wide[:, :b.table.shape[1]] = b.table
    b.table = wide
    b.args = (b.cache, wide, *b.args[2:])
    b.check(b.attend(max_kv=2**40), few=True)


@pytest.mark.parametrize("times", [10, 60])
def test_rows_of_sequences_that_overlap_are_written(times):
    # sequences that fall back again and again hold more rows than there are, more than
    # the launch has CTAs for; the one behind them is right or NaN, and no row is left
    # as it was
    b = Batch([40], [200], 16, 2, seed=8)
    starts = [0, 40, 0] * times + [0, 40, 80]
    n = len(starts) - 1
    table, lens = b.table.repeat(n, 1), ints([200] * n)
    q = torch.cat([b.q, b.q, b.q[:5]])
    out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    w = workspace()
    sa.prefill_paged_int4(q, ints(starts), b.cache, table, lens, b.sinks, b.scale, 40, 200, out=out, lse=lse, workspace=w)
    assert (out[80:] == 7).all() and (lse[80:] == 7).all()
    want = b.attend()
    b.check(want)
    for rows in (slice(0, 40), slice(40, 80)):
        for got, ref in zip((out, lse), want):
            assert ((got[rows] == ref) | torch.isnan(got[rows])).all()
    assert parts(w) == 0


def test_verification_of_many_rows_after_the_kernel_that_writes_its_queries():
    # the launch mode is the caller's to ask for; above 32 rows per KV head there is one only
    b = Batch([8] * 4, [2000, 8, 500, 1300], 64, 8, seed=9)
    q = b.q.view(4, 8, 64, 64)
    want = sa.verify_int4(q, *b.args, 2000, programmatic=False)
    b.check(want)
    rope = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).to(DEV)
    qkv = torch.cat([b.q, torch.zeros(32, 16, 64, device=DEV).bfloat16()], 1).flatten(1)
    w = workspace()
    for _ in range(20):
        made = torch.full_like(b.q, float("nan"))
        sa.qkv_prologue_int4(qkv, None, ints([0] * 32), ints([-1] * 32), rope, b.cache, 64, 8, q_out=made)
        got = sa.verify_int4(made.view_as(q), *b.args, 2000, programmatic=True, workspace=w)
        assert all(torch.equal(x, y) for x, y in zip(got, want))


# ------------------------------------------------------------------ large values
def test_rows_at_the_top_of_the_range():
    # what the format says, and no value that is not finite
    with np.errstate(over="ignore"):
        x = torch.from_numpy(rows_at_the_top(600)).bfloat16()
        y = x.float().numpy()
        fine = np.isfinite(y).all(-1) & np.isfinite(np.maximum(y.max(-1), 0) - np.minimum(y.min(-1), 0))
    rope = torch.cat([torch.ones(1, 32), torch.zeros(1, 32)], 1).to(DEV)
    cache = sa.int4_cache(40, 1, DEV)
    qkv = torch.cat([torch.zeros_like(x), torch.zeros_like(x), x], 1).to(DEV)
    slots = ints(range(600))
    sa.qkv_prologue_int4(qkv, None, torch.zeros_like(slots), slots, rope, cache, 1, 1)
    v = sa.gather_int4(cache, slots)[1][:, 0].float().cpu().numpy()
    assert fine.sum() > 500 and np.isfinite(v[fine]).all() and np.isnan(v[~fine]).all()
    np.testing.assert_array_equal(v[fine], int4.round_trip(y[fine]).astype(np.float32))


@pytest.mark.parametrize("tokens", [1, 3, 40])           # one row, few rows, tensor cores
def test_large_values_are_summed_without_overflow(tokens):
    # values 2^105 times as large give outputs 2^105 times as large, bit for bit: weights
    # below 2^10, 300 keys and values below 2^3 make sums below 2^(105 + 10 + 9 + 3)
    got = []
    for v_gain in (1.0, 2.0**105):
        b = Batch([tokens] * 2, [300, 250], 16, 2, seed=11, v_gain=v_gain)
        calls = [b.attend(), sa.verify_int4(b.q.view(2, tokens, 16, 64), *b.args, 300)]
        if tokens == 1:
            calls.append(sa.decode_int4(b.q, *b.args, 300))
        got.append([x for call in calls for x in call])
    for small, large in zip(*got):
        if small.dtype == torch.bfloat16:
            assert torch.isfinite(large).all() and torch.equal(small.double() * 2.0**105, large.double())
        else:
            assert torch.equal(small, large)
