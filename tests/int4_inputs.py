"""Small inputs on a paged cache held in 4 bits, and the bars of attention over it."""

import numpy as np
import torch

from oracle import int4

DEV = "cuda:0"


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Packed:
    """Requests of the given lengths on shuffled pages of one pool.  Slots past a
    request's keys and pages of nobody hold bytes of 255 (codes 15, scales NaN).
    k, v: what each request's rows stand for, float64; `values`: the pools of these."""

    def __init__(self, lens, hq, hkv, seed=0, spare=4, width_extra=1, k_gain=1.0):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.hq, self.hkv = rng, list(lens), hq, hkv
        need = [-(-n // 16) for n in self.lens]
        self.pages = sum(need) + spare
        ids = rng.permutation(self.pages)
        self.table = np.full((len(lens), max(need + [1]) + width_extra), -1, np.int32)
        self.cache = np.full((self.pages, hkv, int4.BLOCK), 255, np.uint8)
        self.slots, self.k, self.v = [], [], []
        at = 0
        for b, n in enumerate(self.lens):
            mine = ids[at:at + need[b]]
            at += need[b]
            self.table[b, :need[b]] = mine
            j = np.arange(n)
            slots = mine[j // 16] * 16 + j % 16 if n else np.zeros(0, np.int64)
            k, v = k_gain * rng.standard_normal((n, hkv, 64)), rng.standard_normal((n, hkv, 64)) + 0.25
            self.put(slots, k, v)
            self.slots.append(slots)
            self.k.append(int4.round_trip(k))
            self.v.append(int4.round_trip(v))
        self.free = ids[at:]
        self.kv_lens = np.array(self.lens, np.int32)
        self.max_kv = max(self.lens + [1])
        self.sinks = (2 * rng.standard_normal(hq)).astype(np.float32)
        self.scale = 0.125

    def put(self, slots, k, v):
        if len(slots):
            int4.write(self.cache, slots, k, v)

    def values(self):
        """The pools [pages, Hkv, 16, 64] that the cache stands for; NaN where nothing is."""
        pools = [np.full((self.pages, self.hkv, 16, 64), np.nan) for _ in range(2)]
        for slots, k, v in zip(self.slots, self.k, self.v):
            for pool, rows in zip(pools, (k, v)):
                pool[slots // 16, :, slots % 16] = rows
        return pools

    def q(self, *shape):
        return torch.from_numpy(self.rng.standard_normal((*shape, self.hq, 64)).astype(np.float32)).bfloat16()

    def gpu(self):
        """cache, page table, lengths, sinks, scale."""
        return [torch.from_numpy(a).to(DEV) for a in (self.cache, self.table, self.kv_lens, self.sinks)] + [self.scale]


def rows(q, k, v, seen, sinks, scale):
    """Rows q [T, Hq, 64] over one request's k, v [n, Hkv, 64], row i seeing the keys
    where seen[i] ([T, n]).  Returns (out, lse, weight): weight [T, Hq, 64] is
    sum_j p_j |v_j|, which the bars need.  Keys that a row does not see may be NaN."""
    t, hq, d = q.shape
    group = hq // k.shape[1]
    out, weight, lse = np.zeros((t, hq, d)), np.zeros((t, hq, d)), np.zeros((t, hq))
    for i in range(t):
        at = np.flatnonzero(seen[i])
        for h in range(hq):
            kk, vv = k[at, h // group], v[at, h // group]
            s = scale * (kk @ q[i, h])
            top = max(sinks[h], s.max()) if at.size else sinks[h]
            if top == -np.inf:
                lse[i, h] = -np.inf
                continue
            e = np.exp(s - top)
            z = np.exp(sinks[h] - top) + e.sum()
            out[i, h], weight[i, h], lse[i, h] = e @ vv / z, e @ np.abs(vv) / z, top + np.log(z)
    return out, lse, weight


def assert_rows(got, want, what=""):
    """out against the definition, whose third part is sum p |v|.  Roundings, each off by
    at most half a step of bf16, 2^-8 of its value: the weights (times the scale of the
    value, which is not rounded) 2^-8 sum p |v|, the output 2^-8 |out|; 5% on top for the
    second order (2^-8 of that) and the approximate exponential (2^-22).  The scores are
    fp32 sums of 64 products of q and 16 + n < 32 from which (16 + z) sum q is taken:
    with |q| < 6, s < 1 (rows of a few units, gains as in the tests), scale 1/8 each of
    the two is below 64 * 6 * 32 / 8 = 1536 and is off by at most some 64 * 2^-24 of that
    in the worst order, 2^-8 in all; the sums are random, so a hundredth of it is taken:
    2^-14 absolute, which changes p by 2^-14 and the lse by as much.  The value's
    products are exact, and their fp32 sums, which tensor cores cut instead of rounding,
    are off by less than 2^-20 of 31 sum p s."""
    out, lse = (np64(x) for x in got)
    ref, ref_lse, weight = want
    bar = 1.05 * 2.0**-8 * (weight + np.abs(ref)) + 2.0**-13 * weight + 2.0**-15
    err = np.abs(out - ref)
    assert np.isfinite(out).all(), f"{what}: not finite"
    assert (err <= bar).all(), f"{what}: {(err / bar).max():.2f} of the bar at {np.unravel_index((err / bar).argmax(), err.shape)}"
    inf = np.isinf(ref_lse)
    assert np.array_equal(np.isinf(lse), inf) and np.array_equal(lse[inf], ref_lse[inf]), what
    assert (np.abs(lse - ref_lse)[~inf] <= 2.0**-13).all(), f"{what}: lse off by {np.abs(lse - ref_lse)[~inf].max():.2e}"
