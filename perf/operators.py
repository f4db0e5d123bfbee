"""Measured cases of the operators that bound a long context: attention with a
sliding window and a few first tokens that stay visible, the attention weight
that each cached key has drawn, and eviction from the paged cache by it.

`prepare` makes what a serving loop holds before the call (queries, paged
caches, page tables, lengths, scratch), `run` makes one call.  With `own`
false the call is the operator's plain form in 32 bits; with `own` true it is
the library's entry point.  `exact` gives the same outputs in 64 bits.
"""

import math
import random

import numpy as np
import torch

own = False

PAGE, DIM = 16, 64
SCRATCH_BYTES = 64 << 20       # the zero-filled workspace that a program keeps for its split plans


# ------------------------------------------------------------------- cases
def _case(op, name=None, **kw):
    c = {} if name is None else {"name": name}
    c.update(op=op, hq=64, hkv=8, lens_seed=1)
    c.update(kw)
    return c


def listed():
    return [
        # one user, a short answer under way: the smallest call of a sliding layer, latency only
        _case("decode_window", "decode_window_one", batch=1, min_kv=2000, max_kv=2000, window=128, first=4),
        # a full decode batch in a sliding layer of 128 keys
        _case("decode_window", "decode_window_batch", batch=64, min_kv=1, max_kv=4096, window=128, first=0),
        # endless streams on a long cache: a wide window and first tokens that stay
        _case("decode_window", "decode_window_long", batch=8, min_kv=32768, max_kv=131072, window=16384, first=16),
        # prompts of a ragged batch in a sliding layer of 128 keys
        _case("prefill_window", "prefill_window_ragged", batch=4, min_q=2048, max_q=8192, window=128, first=0),
        # fewer heads, an odd window and first tokens, odd lengths
        _case("prefill_window", "prefill_window_odd", batch=3, min_q=1001, max_q=4099, window=1023, first=5, hq=16, hkv=2),
        # chunked prefill: 2048 new tokens on prefixes of up to 14336 cached ones
        _case("prefill_paged_window", "prefill_paged_window_chunk", batch=4, min_q=2048, max_q=2048,
              min_prefix=0, max_prefix=14336, window=4096, first=4),
        # every decode step of an evicting layer adds its weights
        _case("decode_mass", "decode_mass_batch", batch=64, min_kv=1, max_kv=4096),
        # the same on long caches
        _case("decode_mass", "decode_mass_long", batch=8, min_kv=32768, max_kv=131072),
        # a whole prompt's weights, for eviction right after prefill
        _case("prefill_mass", "prefill_mass_prompt", batch=4, min_q=1024, max_q=4096, min_prefix=0, max_prefix=0),
        # only the last 32 tokens of long prompts vote
        _case("prefill_mass", "prefill_mass_tail", batch=8, min_q=32, max_q=32, min_prefix=8160, max_prefix=32736),
        # a decode batch is cut to 1024 keys each
        _case("evict", "evict_batch", batch=64, min_kv=1, max_kv=4096, budget=1024, first=4, recent=256),
        # long caches are cut to 8192 keys each
        _case("evict", "evict_long", batch=8, min_kv=32768, max_kv=131072, budget=8192, first=16, recent=1024),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["decode_window", "prefill_window", "prefill_paged_window", "decode_mass", "prefill_mass", "evict"])
    hq, hkv = rng.choice([(64, 8), (64, 8), (16, 2), (4, 1), (8, 8), (40, 8), (32, 2)])
    c = _case(op, hq=hq, hkv=hkv, lens_seed=rng.randrange(1 << 30))
    if op in ("decode_window", "decode_mass", "evict"):
        c["batch"] = log(1, 64)
        c["max_kv"] = log(8, min(131072, (1 << 19) // c["batch"]))
        c["min_kv"] = rng.choice([0 if op != "evict" else 1, c["max_kv"] // 3, c["max_kv"]])
    else:
        c["batch"] = log(1, 8)
        if op == "prefill_mass" and rng.random() < 0.5:
            c["max_q"] = log(1, 64)
            c["max_prefix"] = log(16, (1 << 18) // c["batch"])
        else:
            c["max_q"] = log(1, 8192 // c["batch"])
            c["max_prefix"] = 0 if op == "prefill_window" else rng.choice([0, log(1, 8192 // c["batch"])])
        c["min_q"] = rng.choice([1, max(1, c["max_q"] // 2), c["max_q"]])
        c["min_prefix"] = rng.choice([0, c["max_prefix"]])
        if op == "prefill_window":
            del c["min_prefix"], c["max_prefix"]
    if op.endswith("window"):
        c["window"] = log(1, 16384 if op == "decode_window" else 4096)
        c["first"] = rng.choice([0, 1, 4, 16, 17, 64])
    if op == "evict":
        c["budget"] = log(2, max(2, c["max_kv"] * 3 // 4))
        c["first"] = min(rng.choice([0, 4, 16]), c["budget"] // 4)
        c["recent"] = rng.randint(0, c["budget"] // 2)
    return c


def _between(rng, lo, hi, n):
    """n lengths over lo..hi, the largest always among them."""
    return [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]


def _lengths(case):
    """(query tokens, keys) of each request: the case's alone, whatever the data's seed."""
    rng = random.Random(case["lens_seed"])
    n = case["batch"]
    if "max_kv" in case:
        return [1] * n, _between(rng, case["min_kv"], case["max_kv"], n)
    q = _between(rng, case["min_q"], case["max_q"], n)
    pre = _between(rng, case.get("min_prefix", 0), case.get("max_prefix", 0), n)
    return q, [a + b for a, b in zip(q, pre)]


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    rng = random.Random(seed)
    op, batch, hq, hkv = case["op"], case["batch"], case["hq"], case["hkv"]
    q_lens, kv_lens = _lengths(case)

    def normal(*shape, dtype=torch.bfloat16):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    tokens = sum(q_lens)
    s = {"op": op, "scale": 1 / 8, "window": case.get("window"), "first": case.get("first", 0),
         "max_q": max(q_lens), "max_kv": max(kv_lens), "kv_lens": ints(kv_lens),
         "cu_q": ints([0] + torch.tensor(q_lens).cumsum(0).tolist()),
         "sinks": normal(hq, dtype=torch.float32) * 2,
         "scratch": torch.zeros(SCRATCH_BYTES, dtype=torch.uint8, device=dev)}
    if op != "evict":
        s["q"] = normal(tokens, hq, DIM)
    if op == "prefill_window":
        s["k"], s["v"] = normal(tokens, hkv, DIM), normal(tokens, hkv, DIM)
        return s

    # pages in shuffled order, as an allocator hands them out after a while
    need = [-(-n // PAGE) for n in kv_lens]
    kept = [-(-case["budget"] // PAGE)] * batch if op == "evict" else [0] * batch
    ids = list(range(sum(need) + sum(kept) + 8))
    rng.shuffle(ids)
    s["k_cache"] = normal(len(ids), hkv, PAGE, DIM)
    if not op.endswith("mass"):
        s["v_cache"] = normal(len(ids), hkv, PAGE, DIM)

    def table(counts):
        width = max(1, max(counts))
        rows = []
        for c in counts:
            rows.append([ids.pop() for _ in range(c)] + [0] * (width - c))
        return ints(rows)

    s["page_table"] = table(need)
    if op in ("decode_mass", "prefill_mass"):
        s["lse"] = _row_lse(s)
    if op in ("decode_mass", "prefill_mass", "evict"):
        # what earlier steps have left: most keys near nothing, a few heavy
        s["mass"] = torch.exp(normal(batch, hkv, max(s["max_kv"], 1), dtype=torch.float32) * 2 - 7)
    if op == "evict":
        s["budget"], s["recent"] = case["budget"], case["recent"]
        s["dst_table"] = table(kept)
        s["dst_mass"] = torch.zeros(batch, hkv, case["budget"], device=dev)
    return s


def _padded(s):
    """Query rows as [request, place]: the row of q, whether it is one, and its position among the keys."""
    cu = s["cu_q"].long()
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(s["max_q"], device=cu.device)
    live = i < q_len[:, None]
    row = torch.where(live, cu[:-1, None] + i, 0)
    return row, live, s["kv_lens"].long()[:, None] - q_len[:, None] + i


def _keys(s, which, head, pos):
    """Rows `pos` [request, ...] of one KV head's keys or values, in 32 bits; positions are in range."""
    r = torch.arange(pos.shape[0], device=pos.device).view(-1, *[1] * (pos.dim() - 1))
    if s["op"] == "prefill_window":
        return s[which][s["cu_q"].long()[:-1][r] + pos, head].float()
    return s[which + "_cache"][s["page_table"].long()[r, pos // PAGE], head, pos % PAGE].float()


def _row_lse(s):
    """The log of each row's full softmax denominator, sink included, as the attention call returns it."""
    row, live, place = _padded(s)
    hkv = s["k_cache"].shape[1]
    group = s["sinks"].numel() // hkv
    lse = torch.empty(s["q"].shape[:2], device=row.device)
    j = torch.arange(max(s["max_kv"], 1), device=row.device)
    pos = torch.minimum(j, (s["kv_lens"].long()[:, None] - 1).clamp(min=0))
    for h in range(hkv):
        heads = slice(h * group, (h + 1) * group)
        sc = torch.einsum("rigd,rjd->rgij", s["q"][row, heads].float(), _keys(s, "k", h, pos)) * s["scale"]
        sc = sc.masked_fill(j > place[:, None, :, None], -math.inf)
        full = torch.logaddexp(sc.logsumexp(-1), s["sinks"][heads][None, :, None])
        lse[row[live], heads] = full.transpose(1, 2)[live]
    return lse


# ------------------------------------------------------------- plain forms
def _softmax_with_sink(sc, sink):
    """Weights and log denominator of scores [..., keys] (-inf where masked) joined by one sink logit."""
    top = torch.maximum(sc.amax(-1), sink)
    e = torch.exp(sc - top[..., None])
    total = e.sum(-1) + torch.exp(sink - top)
    return e / total[..., None], top + torch.log(total)


def _plain_decode_window(s):
    q, n, first = s["q"], s["kv_lens"].long(), s["first"]
    batch, hq, _ = q.shape
    hkv = s["k_cache"].shape[1]
    wide = min(s["window"], max(s["max_kv"], 1))
    head = torch.arange(first, device=q.device).expand(batch, -1)
    tail = n[:, None] - wide + torch.arange(wide, device=q.device)
    pos = torch.cat([head, tail], 1)
    seen = torch.cat([head < n[:, None] - wide, tail >= 0], 1)
    pos = torch.where(seen, pos, 0)
    page = s["page_table"].long().gather(1, pos // PAGE)
    k = s["k_cache"][page, :, pos % PAGE].float()
    v = s["v_cache"][page, :, pos % PAGE].float()
    sc = torch.einsum("bhgd,bjhd->bhgj", q.float().view(batch, hkv, -1, DIM), k) * s["scale"]
    sc = sc.masked_fill(~seen[:, None, None], -math.inf)
    p, lse = _softmax_with_sink(sc, s["sinks"].view(hkv, -1).expand(batch, -1, -1))
    out = torch.einsum("bhgj,bjhd->bhgd", p, v)
    return {"out": out.reshape(batch, hq, DIM).to(q.dtype), "lse": lse.reshape(batch, hq)}


def _plain_prefill_window(s):
    """Blocks of rows against the band of keys that their windows reach, one KV head after another."""
    q, window, first = s["q"], s["window"], s["first"]
    row, live, place = _padded(s)
    n_req, longest = row.shape
    hq = q.shape[1]
    hkv = (s["k"] if "k" in s else s["k_cache"]).shape[1]
    group = hq // hkv
    wide = min(window, s["max_kv"])
    block = min(longest, max(128, min(wide, 1024)))
    blocks = -(-longest // block)
    pad = blocks * block - longest
    at = place[:, :1] + torch.arange(blocks * block, device=q.device)
    at = at.view(n_req, blocks, block)
    q_row = torch.nn.functional.pad(row, (0, pad)).view(n_req, blocks, block)
    last = (s["kv_lens"].long() - 1)[:, None, None]
    band = at[..., :1] - (wide - 1) + torch.arange(block + wide - 1, device=q.device)
    head = torch.arange(first, device=q.device).expand(n_req, blocks, -1)
    j, i = band[:, :, None], at[..., None]
    seen = torch.cat([(head[:, :, None] <= i - wide), (j >= 0) & (j <= i) & (j > i - wide)], -1)
    pos = torch.minimum(torch.cat([head, band], -1).clamp(min=0), last)
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)
    for h in range(hkv):
        heads = slice(h * group, (h + 1) * group)
        sc = torch.einsum("rbigd,rbjd->rbigj", q[q_row, heads].float(), _keys(s, "k", h, pos)) * s["scale"]
        sc = sc.masked_fill(~seen[:, :, :, None], -math.inf)
        p, full = _softmax_with_sink(sc, s["sinks"][heads].expand(sc.shape[:-1]))
        o = torch.einsum("rbigj,rbjd->rbigd", p, _keys(s, "v", h, pos)).to(q.dtype)
        out[row[live], heads] = o.flatten(1, 2)[:, :longest][live]
        lse[row[live], heads] = full.flatten(1, 2)[:, :longest][live]
    return {"out": out, "lse": lse}


def _plain_decode_mass(s):
    q, n, mass = s["q"], s["kv_lens"].long(), s["mass"]
    batch, hq, _ = q.shape
    hkv = s["k_cache"].shape[1]
    j = torch.arange(mass.shape[2], device=q.device).expand(batch, -1)
    seen = j < n[:, None]
    pos = torch.where(seen, j, 0)
    k = s["k_cache"][s["page_table"].long().gather(1, pos // PAGE), :, pos % PAGE].float()
    sc = torch.einsum("bhgd,bjhd->bhgj", q.float().view(batch, hkv, -1, DIM), k) * s["scale"]
    p = torch.exp(sc - s["lse"].view(batch, hkv, -1, 1))
    mass += p.masked_fill(~seen[:, None, None], 0).sum(2)
    return mass


def _plain_prefill_mass(s):
    row, live, place = _padded(s)
    mass = s["mass"]
    hkv = mass.shape[1]
    group = s["q"].shape[1] // hkv
    j = torch.arange(mass.shape[2], device=mass.device)
    hidden = (j > place[..., None]) | ~live[..., None]
    pos = torch.minimum(j, s["kv_lens"].long()[:, None] - 1)
    for h in range(hkv):
        heads = slice(h * group, (h + 1) * group)
        sc = torch.einsum("rigd,rjd->rgij", s["q"][row, heads].float(), _keys(s, "k", h, pos)) * s["scale"]
        p = torch.exp(sc - s["lse"][row, heads].transpose(1, 2)[..., None])
        mass[:, h] += p.masked_fill(hidden[:, None], 0).sum((1, 2))
    return mass


def _plain_evict(s):
    n, mass, budget = s["kv_lens"].long(), s["mass"], s["budget"]
    hkv = mass.shape[1]
    j = torch.arange(mass.shape[2], device=mass.device)
    left = n[:, None, None]
    held = (j < s["first"]) | (j >= left - s["recent"])
    rank = mass.masked_fill(held, math.inf).masked_fill(j >= left, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.nn.functional.pad(order.sort(-1).values, (0, budget - order.shape[-1]))
    slot = torch.arange(budget, device=mass.device)
    fits = slot < left.clamp(max=budget)
    kept = torch.where(fits, order, -1)
    src = torch.where(fits, order, 0)
    b = torch.arange(n.numel(), device=mass.device)[:, None, None]
    h = torch.arange(hkv, device=mass.device)[:, None]
    a = (s["page_table"].long()[b, src // PAGE], h, src % PAGE)
    d = (s["dst_table"].long()[b, slot // PAGE].expand(-1, hkv, -1), h, slot % PAGE)
    for c in (s["k_cache"], s["v_cache"]):
        c[d] = torch.where(fits[..., None], c[a], c[d])
    s["dst_mass"].copy_(torch.where(fits, mass.gather(2, src), s["dst_mass"]))
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "mass": s["dst_mass"],
            "kv_lens": n.clamp(max=budget).int(), "kept": kept.int()}


PLAIN = {"decode_window": _plain_decode_window, "prefill_window": _plain_prefill_window,
         "prefill_paged_window": _plain_prefill_window, "decode_mass": _plain_decode_mass,
         "prefill_mass": _plain_prefill_mass, "evict": _plain_evict}


# ------------------------------------------------------- the library's calls
def _own(s):
    import gqa_attention_learned_gb300 as sa

    op = s["op"]
    paged = [s.get(n) for n in ("k_cache", "v_cache", "page_table", "kv_lens")]
    if op == "decode_window":
        out, lse = sa.decode_window(s["q"], *paged, s["sinks"], s["scale"], s["max_kv"], s["window"], s["first"],
                                    workspace=s["scratch"])
        return {"out": out, "lse": lse}
    if op == "prefill_window":
        out, lse = sa.prefill_window(s["q"], s["k"], s["v"], s["cu_q"], s["sinks"], s["scale"], s["max_q"],
                                     s["window"], s["first"])
        return {"out": out, "lse": lse}
    if op == "prefill_paged_window":
        out, lse = sa.prefill_paged_window(s["q"], s["cu_q"], *paged, s["sinks"], s["scale"], s["max_q"],
                                           s["max_kv"], s["window"], s["first"])
        return {"out": out, "lse": lse}
    if op == "decode_mass":
        return sa.decode_mass(s["q"], s["k_cache"], s["page_table"], s["kv_lens"], s["lse"], s["scale"],
                              s["max_kv"], s["mass"])
    if op == "prefill_mass":
        return sa.prefill_mass(s["q"], s["cu_q"], s["k_cache"], s["page_table"], s["kv_lens"], s["lse"],
                               s["scale"], s["max_q"], s["max_kv"], s["mass"])
    kv_lens, kept = sa.evict(*paged, s["mass"], s["budget"], s["max_kv"], first_tokens=s["first"],
                             recent=s["recent"], dst_page_table=s["dst_table"], dst_mass=s["dst_mass"])
    return {"k_cache": s["k_cache"], "v_cache": s["v_cache"], "mass": s["dst_mass"], "kv_lens": kv_lens, "kept": kept}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# --------------------------------------------------------------------- work
def work(case):
    """What one call cannot do without: every input that counts read once, every output written once."""
    op, hq, hkv = case["op"], case["hq"], case["hkv"]
    q_lens, kv_lens = _lengths(case)
    row = 2 * DIM                                     # bytes of one head's bf16 row
    tokens, keys = sum(q_lens), sum(kv_lens)
    if op == "evict":
        moved = sum(min(n, case["budget"]) for n in kv_lens) * hkv
        return {"bytes": 4 * keys * hkv + moved * (2 * 2 * row + 4 + 4) + 8 * len(kv_lens), "flops": 0}
    if op in ("decode_mass", "prefill_mass"):
        pairs = sum(sum(range(n - t + 1, n + 1)) for t, n in zip(q_lens, kv_lens) if n)
        return {"bytes": tokens * hq * (row + 4) + keys * hkv * (row + 8), "flops": 2 * DIM * hq * pairs}
    window, first = case["window"], case["first"]

    def seen(p):                                      # keys visible from position p
        return min(p + 1, window) + max(0, min(first, p + 1 - window))

    pairs = sum(sum(seen(p) for p in range(n - t, n)) for t, n in zip(q_lens, kv_lens) if n)
    needed = sum(min(n, t - 1 + window + first) for t, n in zip(q_lens, kv_lens))
    return {"bytes": tokens * hq * (2 * row + 4) + needed * hkv * 2 * row, "flops": 4 * DIM * hq * pairs}


# -------------------------------------------------------------------- 64 bits
def _request(s, b):
    """One request's query rows, keys and values, in 64 bits and contiguous."""
    lo, hi = int(s["cu_q"][b]), int(s["cu_q"][b + 1])
    n = int(s["kv_lens"][b])
    if "k" in s:
        return lo, hi, s["k"][lo:hi].double(), s["v"][lo:hi].double()
    pages = s["page_table"][b, :-(-n // PAGE)].long()

    def rows(cache):
        return cache[pages].transpose(1, 2).reshape(-1, cache.shape[1], DIM)[:n].double()

    return lo, hi, rows(s["k_cache"]), rows(s["v_cache"]) if "v_cache" in s else None


def _exact_window(s):
    q = s["q"].double()
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    sinks = s["sinks"].double()
    for b in range(s["kv_lens"].numel()):
        lo, hi, k, v = _request(s, b)
        n, hkv = k.shape[0], k.shape[1]
        group = q.shape[1] // hkv
        for a in range(lo, hi, 512):
            z = min(a + 512, hi)
            p = torch.arange(a - lo, z - lo, device=q.device) + n - (hi - lo)
            start = max(0, int(p[0]) - s["window"] + 1)
            cols = list(range(min(s["first"], start)))
            idx = torch.cat([torch.tensor(cols, dtype=torch.long, device=q.device),
                             torch.arange(start, int(p[-1]) + 1, device=q.device)])
            see = (idx <= p[:, None]) & ((idx < s["first"]) | (idx > p[:, None] - s["window"]))
            for g in range(hkv):
                hs = slice(g * group, (g + 1) * group)
                sc = (q[a:z, hs] @ k[idx, g].T) * s["scale"]
                sc[~see[:, None].expand_as(sc)] = -math.inf
                full = torch.logsumexp(torch.cat([sc, sinks[hs].expand(z - a, -1)[..., None]], -1), -1)
                out[a:z, hs] = torch.exp(sc - full[..., None]) @ v[idx, g]
                lse[a:z, hs] = full
    return {"out": out, "lse": lse}


def _exact_mass(s):
    mass = s["mass"].double()
    q, lse = s["q"].double(), s["lse"].double()
    for b in range(mass.shape[0]):
        lo, hi, k, _ = _request(s, b)
        n, hkv = k.shape[0], k.shape[1]
        group = q.shape[1] // hkv
        for g in range(hkv if n else 0):
            hs = slice(g * group, (g + 1) * group)
            for a in range(lo, hi, 256):
                z = min(a + 256, hi)
                top = n - (hi - z)                        # keys that the last of these rows sees
                w = torch.exp(q[a:z, hs] @ k[:top, g].T * s["scale"] - lse[a:z, hs, None])
                late = torch.arange(top, device=q.device) > torch.arange(n - (hi - a), top + 1, device=q.device)[:z - a, None]
                w[late[:, None].expand_as(w)] = 0
                mass[b, g, :top] += w.sum((0, 1))
    return mass


def _exact_evict(s):
    k_cache, v_cache, dst = s["k_cache"].double(), s["v_cache"].double(), s["dst_mass"].double()
    batch, hkv, budget = dst.shape
    kept = torch.full((batch, hkv, budget), -1, dtype=torch.int32)
    mass, table, to = s["mass"].cpu(), s["page_table"].cpu().long(), s["dst_table"].cpu().long()
    left = []
    for b in range(batch):
        n = int(s["kv_lens"][b])
        count = min(n, budget)
        left.append(count)
        for g in range(hkv):
            keep = np.arange(n)
            if n > budget:
                middle = keep[s["first"]:n - s["recent"]]
                heavy = middle[np.lexsort((middle, -mass[b, g, middle].numpy()))]
                heavy = heavy[:budget - s["first"] - s["recent"]]
                keep = np.sort(np.concatenate([keep[:s["first"]], heavy, keep[n - s["recent"]:]]))
            at, slot = torch.from_numpy(keep).long(), torch.arange(count)
            kept[b, g, :count] = at.int()
            for c, old in ((k_cache, s["k_cache"]), (v_cache, s["v_cache"])):
                c[to[b, slot // PAGE].cuda(), g, (slot % PAGE).cuda()] = \
                    old[table[b, at // PAGE].cuda(), g, (at % PAGE).cuda()].double()
            dst[b, g, :count] = mass[b, g, at].double().cuda()
    return {"k_cache": k_cache, "v_cache": v_cache, "mass": dst,
            "kv_lens": torch.tensor(left, dtype=torch.int32), "kept": kept}


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "evict":
        return _exact_evict(s)
    if op.endswith("mass"):
        return _exact_mass(s)
    return _exact_window(s)
