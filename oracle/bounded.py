"""Float64 reference for the operators that bound a long context (test
infrastructure only; shares no code with the CUDA path): attention with a
sliding window and first tokens that stay visible, attention mass, eviction.
"""

import numpy as np


def visible(pos, n, window, first_tokens):
    """Boolean [n]: the keys that a row at position pos sees."""
    j = np.arange(n)
    return (j <= pos) & ((j < first_tokens) | (j > pos - window))


def window_rows(q, k, v, positions, sinks, scale, window, first_tokens=0):
    """Rows q [T, Hq, D] at `positions` against one request's keys k, v
    [n, Hkv, D]; each row as the definition says, over its visible keys only.
    Returns (out [T, Hq, D], lse [T, Hq])."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    t, hq, d = q.shape
    hkv = k.shape[1]
    out, lse = np.zeros((t, hq, d)), np.zeros((t, hq))
    for r in range(t):
        at = np.flatnonzero(visible(positions[r], k.shape[0], window, first_tokens))
        for h in range(hq):
            g = h // (hq // hkv)
            s = scale * (k[at, g] @ q[r, h])
            top = max(sinks[h], s.max()) if at.size else sinks[h]
            if top == -np.inf:
                lse[r, h] = -np.inf
                continue
            e = np.exp(s - top)
            z = np.exp(sinks[h] - top) + e.sum()
            out[r, h] = e @ v[at, g] / z
            lse[r, h] = top + np.log(z)
    return out, lse


def mass_rows(q, k, positions, lse, scale):
    """[Hkv, n]: the weight that rows q [T, Hq, D] give to one request's keys
    k [n, Hkv, D]."""
    q, k, lse = (np.asarray(a, np.float64) for a in (q, k, lse))
    t, hq, _ = q.shape
    n, hkv, _ = k.shape
    mass = np.zeros((hkv, n))
    for r in range(t):
        m = min(positions[r] + 1, n)
        for h in range(hq):
            if lse[r, h] == -np.inf:
                continue
            g = h // (hq // hkv)
            mass[g, :m] += np.exp(scale * (k[:m, g] @ q[r, h]) - lse[r, h])
    return mass


def keep(mass, n, budget, first_tokens, recent):
    """Indices, ascending, that one KV head keeps of n keys with mass [>= n]."""
    if n <= budget:
        return list(range(n))
    rest = range(first_tokens, n - recent)

    def order(i):                    # heaviest first, NaN last, ties by index
        nan = np.isnan(mass[i])
        return (nan, 0.0 if nan else -float(mass[i]), i)

    chosen = sorted(rest, key=order)[:budget - first_tokens - recent]
    return sorted([*range(first_tokens), *chosen, *range(n - recent, n)])
