"""Small paged inputs for the tests of windowed attention, mass and eviction."""

import numpy as np
import torch

DEV = "cuda:0"


def bf16(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(torch.bfloat16)


def np64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


class Paged:
    """Requests of the given lengths on shuffled pages of one pool.  Slots past
    a request's keys and pages of nobody hold NaN."""

    def __init__(self, lens, hq, hkv, seed=0, spare=4, width_extra=1):
        rng = np.random.default_rng(seed)
        self.rng, self.lens, self.hq, self.hkv = rng, list(lens), hq, hkv
        need = [-(-n // 16) for n in self.lens]
        self.pages = sum(need) + spare
        ids = rng.permutation(self.pages)
        self.table = torch.full((len(lens), max(need + [1]) + width_extra), -1, dtype=torch.int32)
        self.k_cache = torch.full((self.pages, hkv, 16, 64), float("nan"), dtype=torch.bfloat16)
        self.v_cache = self.k_cache.clone()
        self.k, self.v = [], []
        at = 0
        for b, n in enumerate(self.lens):
            mine = torch.from_numpy(ids[at:at + need[b]].astype(np.int32))
            at += need[b]
            self.table[b, :need[b]] = mine
            k, v = bf16(rng, n, hkv, 64), bf16(rng, n, hkv, 64)
            self.k.append(k)
            self.v.append(v)
            for j in range(n):
                self.k_cache[mine[j // 16].long(), :, j % 16] = k[j]
                self.v_cache[mine[j // 16].long(), :, j % 16] = v[j]
        self.free = torch.from_numpy(ids[at:].astype(np.int32))
        self.kv_lens = torch.tensor(self.lens, dtype=torch.int32)
        self.max_kv = max(self.lens + [1])
        self.sinks = torch.from_numpy((2 * rng.standard_normal(hq)).astype(np.float32))
        self.scale = 0.125

    def hide(self, b, seen):
        """NaN over the keys of request b outside `seen` (boolean [n]), and a
        page id far outside the pool for its pages without a seen key."""
        n = self.lens[b]
        for j in np.flatnonzero(~np.asarray(seen)):
            page = int(self.table[b, j // 16])
            if 0 <= page < self.pages:
                self.k_cache[page, :, j % 16] = float("nan")
                self.v_cache[page, :, j % 16] = float("nan")
        for pg in range(-(-n // 16)):
            if not np.any(seen[16 * pg:16 * pg + 16]):
                self.table[b, pg] = 10 ** 9

    def gpu(self, *names):
        return [getattr(self, n).to(DEV) for n in names]

    def paged(self):
        return self.gpu("k_cache", "v_cache", "table", "kv_lens")
