"""Float64 reference for the paged cache held in 4 bits (test infrastructure only;
shares no code with the CUDA path): quantisation of rows, their layout in a page,
and what they stand for.  Attention over such a cache is the attention of
`oracle` over the values.
"""

import numpy as np

PAGE, DIM, BLOCK = 16, 64, 1088


def quantise(x):
    """Codes [..., 64], scales and zero points [...] of rows x [..., 64], in float32
    steps as the format says; a row whose range is not finite has scale NaN."""
    x = np.asarray(x, np.float32)
    with np.errstate(all="ignore"):
        lo = np.minimum(x.min(-1), np.float32(0))
        hi = np.maximum(x.max(-1), np.float32(0))
        span = hi - lo
        fine = np.isfinite(span)
        s = np.where(fine, span, np.float32(0)) / np.float32(15)
        bits = (s.view(np.uint32).astype(np.uint64) + 0xFFFFF) >> 20 << 20
        s = np.maximum(bits, 1 << 23).astype(np.uint32).view(np.float32)
        z = np.rint(np.where(fine, -lo, np.float32(0)) / s)
        n = np.clip(np.rint(np.where(fine[..., None], x, np.float32(0)) / s[..., None]) + z[..., None], 0, 15)
    n = np.where(fine[..., None], n, 0).astype(np.int64)
    return n, np.where(fine, s, np.float32(np.nan)), z.astype(np.int64)


def stands_for(n, s, z):
    return np.asarray(s, np.float64)[..., None] * (np.asarray(n) - np.asarray(z)[..., None])


def round_trip(x):
    """The values that rows x stand for in the cache."""
    return stands_for(*quantise(x))


def write(cache, slots, k, v):
    """Rows k, v [T, Hkv, 64] into slots [T] (page * 16 + place) of cache, uint8
    [pages, Hkv, 1088]."""
    slots = np.asarray(slots)
    page, j = slots // PAGE, slots % PAGE
    heads = np.arange(cache.shape[1])

    def put(at, words):
        for i in range(4):
            cache[page[:, None], heads, (at + i)[:, None]] = (words >> (8 * i)) & 255

    meta = 0
    for half, x in ((0, k), (1, v)):
        n, s, z = quantise(x)
        top = np.where(np.isnan(s), 0x7FC0, s.view(np.uint32) >> 16).astype(np.int64)
        meta = meta | (top | z) << (16 * half)
        for w in range(8):
            word = sum(n[..., 8 * w + e] << (4 * e) for e in range(8))
            if half == 0:
                word = (word << 3 | word >> 29) & 0xFFFFFFFF
                put(64 * (j % 8) + 16 * (w % 4) + 8 * (j // 8) + 4 * (w // 4), word)
            else:
                put(512 + 64 * w + 16 * (j % 8 // 2) + 8 * (j // 8) + 4 * (j % 2), word)
    put(1024 + 8 * (j % 8) + 4 * (j // 8), meta)


def read(cache, page, slot):
    """k, v [Hkv, 64] that a slot stands for, float64."""
    out = np.zeros((2, cache.shape[1], DIM))
    for h in range(cache.shape[1]):
        block = [int(b) for b in cache[page, h]]

        def word(at):
            return sum(block[at + i] << (8 * i) for i in range(4))

        meta = word(1024 + 8 * (slot % 8) + 4 * (slot // 8))
        for half in range(2):
            m = meta >> (16 * half) & 0xFFFF
            s = np.array((m & 0xFFF0) << 16, np.uint32).view(np.float32)
            n = np.zeros(DIM)
            for w in range(8):
                if half == 0:
                    x = word(64 * (slot % 8) + 16 * (w % 4) + 8 * (slot // 8) + 4 * (w // 4))
                    x = (x >> 3) | (x & 7) << 29
                else:
                    x = word(512 + 64 * w + 16 * (slot % 8 // 2) + 8 * (slot // 8) + 4 * (slot % 2))
                n[8 * w:8 * w + 8] = [x >> (4 * e) & 15 for e in range(8)]
            out[half, h] = float(s) * (n - (m & 15))
    return out[0], out[1]
