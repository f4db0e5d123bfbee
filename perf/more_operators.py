"""Measured cases of the operators on a paged cache held in 4 bits: keys and
values appended with bias and rotary encoding on the way, decode, verification
and chunked prefill over that cache, and its rows read back as values.

`prepare` makes what a serving loop holds before the call (queries, the packed
cache, page tables, lengths, scratch), `run` makes one call.  With `own` false
the call is the operator's plain form in 32 bits, on the same packed cache;
with `own` true it is the library's entry point.  `exact` gives the same
outputs in 64 bits.

The cache: uint8 [pages, Hkv, 1088], 16 slots to a page.  A row of 64 values is
64 codes n of 4 bits and 16 bits (s, z), and stands for s * (n - z); s has 4
significant bits, so every such value is a bf16 number.  In 32-bit words, for
slot j of the page:
    K     word 16 (j % 8) + 4 t + 2 (j / 8) + u, t < 4, u < 2: dims 32 u + 8 t + e
          at bits 4 e, e < 8, the word rotated left by 3
    V     word 128 + 16 g + 4 (j % 8 / 2) + 2 (j / 8) + j % 2, g < 8: dims 8 g + e
    (s, z) word 256 + 2 (j % 8) + j / 8: K's in the low half, V's in the high one,
          s as a bf16 number whose last 4 bits are z's
"""

import math
import random

import numpy as np
import torch

own = False

PAGE, DIM, WORDS = 16, 64, 272
ROW_BYTES = 4 * WORDS // PAGE  # 68: one key's K and V of one head
SCRATCH_BYTES = 64 << 20       # the zero-filled workspace that a program keeps for its split plans


# ------------------------------------------------------------------- cases
def _case(op, name=None, **kw):
    c = {} if name is None else {"name": name}
    c.update(op=op, hq=64, hkv=8, lens_seed=1)
    c.update(kw)
    return c


def listed():
    return [
        # one user, an answer under way: latency only
        _case("decode", "decode_one", batch=1, min_kv=2000, max_kv=2000),
        # a full decode batch
        _case("decode", "decode_batch", batch=64, min_kv=1, max_kv=4096),
        # long conversations, what the small cache is for
        _case("decode", "decode_long", batch=8, min_kv=32768, max_kv=131072),
        # speculative decoding, one draft token: two rows per request
        _case("verify", "verify_mtp", batch=64, q_len=2, tree=False, min_kv=2, max_kv=4096),
        # a draft tree of eight tokens on long caches
        _case("verify", "verify_tree", batch=16, q_len=8, tree=True, min_kv=4096, max_kv=32768),
        # a short turn on two long conversations, odd lengths
        _case("prefill", "prefill_turn", batch=2, min_q=77, max_q=201, min_prefix=20001, max_prefix=30011),
        # chunked prefill: 2048 new tokens on prefixes of up to 14336 cached ones
        _case("prefill", "prefill_chunk", batch=4, min_q=2048, max_q=2048, min_prefix=0, max_prefix=14336),
        # whole prompts of a model with fewer heads, odd lengths
        _case("prefill", "prefill_odd", batch=3, min_q=1001, max_q=4099, min_prefix=0, max_prefix=0, hq=16, hkv=2),
        # every decode step appends one token per request
        _case("append", "append_step", batch=64, min_q=1, max_q=1, min_prefix=0, max_prefix=4095),
        # whole prompts of a ragged batch are appended
        _case("append", "append_prompts", batch=4, min_q=2048, max_q=8192, min_prefix=0, max_prefix=0),
        # a few rows are looked at
        _case("gather", "gather_few", batch=1, min_q=100, max_q=100, min_prefix=0, max_prefix=4000),
        # prefixes move to a cache that is not packed
        _case("gather", "gather_prefixes", batch=8, min_q=2000, max_q=8000, min_prefix=0, max_prefix=0),
    ]


def draw(rng):
    def log(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))

    op = rng.choice(["decode", "decode", "verify", "prefill", "prefill", "append", "gather"])
    hq, hkv = rng.choice([(64, 8), (64, 8), (16, 2), (4, 1), (8, 8), (40, 8), (32, 2)])
    c = _case(op, hq=hq, hkv=hkv, lens_seed=rng.randrange(1 << 30))
    if op in ("decode", "verify"):
        c["batch"] = log(1, 64)
        least = 0
        if op == "verify":
            least = c["q_len"] = rng.choice([1, 2, 3, 4, 5, 8, 16, 33, 64])
            c["tree"] = rng.random() < 0.5
        c["max_kv"] = max(least, log(8, min(131072, (1 << (19 if op == "decode" else 17)) // c["batch"])))
        c["min_kv"] = rng.choice([least, max(least, c["max_kv"] // 3), c["max_kv"]])
        return c
    c["batch"] = log(1, 8)
    c["max_q"] = log(1, (8192 if op == "prefill" else 20000) // c["batch"])
    c["min_q"] = rng.choice([1, max(1, c["max_q"] // 2), c["max_q"]])
    c["max_prefix"] = rng.choice([0, log(1, 16384 // c["batch"])])
    c["min_prefix"] = rng.choice([0, c["max_prefix"]])
    return c


def _between(rng, lo, hi, n):
    """n lengths over lo..hi, the largest always among them."""
    return [hi] + [rng.randint(lo, hi) for _ in range(n - 1)]


def _lengths(case):
    """(new tokens, keys) of each request: the case's alone, whatever the data's seed."""
    rng = random.Random(case["lens_seed"])
    n = case["batch"]
    if "max_kv" in case:
        return [case.get("q_len", 1)] * n, _between(rng, case["min_kv"], case["max_kv"], n)
    q = _between(rng, case["min_q"], case["max_q"], n)
    pre = _between(rng, case["min_prefix"], case["max_prefix"], n)
    return q, [a + b for a, b in zip(q, pre)]


# ------------------------------------------------------------ the packed cache
def _places(dev):
    """Word numbers of K [16, 8], V [16, 8] (in the order of the dims) and (s, z) [16] of each slot."""
    j = torch.arange(PAGE, device=dev)[:, None]
    w = torch.arange(8, device=dev)
    k = 16 * (j % 8) + 4 * (w % 4) + 2 * (j // 8) + w // 4
    v = 128 + 16 * w + 4 * (j % 8 // 2) + 2 * (j // 8) + j % 2
    return k, v, (256 + 2 * (j % 8) + j // 8)[:, 0]


def _quantise(x):
    """Codes [..., 64] and (s, z) [...] of rows x [..., 64], step by step in 32 bits."""
    lo, hi = x.amin(-1).clamp(max=0), x.amax(-1).clamp(min=0)
    s = (hi - lo) / torch.full_like(hi, 15)
    bits = (s.contiguous().view(torch.int32) + 0xFFFFF) & ~0xFFFFF      # up to 4 significant bits
    bits = bits.clamp(min=1 << 23)
    s = bits.view(torch.float32)
    z = torch.round(-lo / s)
    n = (torch.round(x / s[..., None]) + z[..., None]).clamp(0, 15)
    return n.to(torch.int32), (bits >> 16) + z.to(torch.int32)


def _in_words(codes):
    """Codes [..., 64] as words [..., 8], eight dims to a word."""
    shift = 4 * torch.arange(8, device=codes.device, dtype=torch.int32)
    return (codes.unflatten(-1, (8, 8)) << shift).sum(-1, dtype=torch.int32)


def _out_of_words(words):
    shift = 4 * torch.arange(8, device=words.device, dtype=torch.int32)
    return ((words[..., None] >> shift) & 15).flatten(-2).float()


def _rotated(w, left):
    """32-bit words rotated left."""
    return (w << left) | ((w >> (32 - left)) & ((1 << left) - 1))


def _rows_to_words(k, v):
    """What rows k, v [..., 64] are in the cache: words of K, of V, and the pair's (s, z)."""
    (kn, km), (vn, vm) = _quantise(k), _quantise(v)
    return _rotated(_in_words(kn), 3), _in_words(vn), km | (vm << 16)


def _stand_for(codes, meta):
    """The values of codes [..., 64] with (s, z) in the low halves of meta [...]."""
    s = ((meta << 16) & ~0xFFFFF).view(torch.float32)
    return s[..., None] * (codes - (meta & 15)[..., None].float())


def _words_to_rows(kw, vw, meta):
    """Values k, v [..., 64] of words [..., 8], [..., 8] and (s, z) [...], in 32 bits."""
    return (_stand_for(_out_of_words(_rotated(kw, 29)), meta),
            _stand_for(_out_of_words(vw), (meta >> 16) & 0xFFFF))


def _page_rows(words):
    """Values k, v [..., 16, 64] of whole blocks [..., 272]."""
    pk, pv, pm = _places(words.device)
    return _words_to_rows(words[..., pk], words[..., pv], words[..., pm])


# ------------------------------------------------------------------ inputs
def _rope(positions, dev):
    """cos and sin [positions, 32 + 32] of YaRN-scaled rotary angles (base 150000, factor 32 over 4096), as a
    program keeps them for all of its layers."""
    theta = 150000.0 ** (-torch.arange(0, DIM, 2, device=dev, dtype=torch.float64) / DIM)
    ramp = ((4096 * theta / (2 * math.pi) - 1) / 31).clamp(0, 1)
    freq = ramp * theta + (1 - ramp) * theta / 32
    angle = torch.arange(positions, device=dev, dtype=torch.float64)[:, None] * freq
    return ((0.1 * math.log(32) + 1) * torch.cat([angle.cos(), angle.sin()], 1)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    rng = random.Random(seed)
    op, batch, hq, hkv = case["op"], case["batch"], case["hq"], case["hkv"]
    q_lens, kv_lens = _lengths(case)

    def normal(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=gen, device=dev, dtype=dtype)

    def ints(v):
        return torch.tensor(v, dtype=torch.int32, device=dev)

    # pages in shuffled order, as an allocator hands them out after a while
    need = [-(-n // PAGE) for n in kv_lens]
    ids = list(range(sum(need) + 8))
    rng.shuffle(ids)
    cache = torch.empty(len(ids), hkv, 4 * WORDS, dtype=torch.uint8, device=dev)
    words = cache.view(torch.int32)
    pk, pv, pm = _places(dev)
    gain = torch.exp(normal(hkv, 1, DIM) / 2)          # some channels of K are larger than others
    for a in range(0, len(ids), 4096):
        n = min(4096, len(ids) - a)
        kw, vw, meta = _rows_to_words(normal(n, hkv, PAGE, DIM) * gain, normal(n, hkv, PAGE, DIM))
        part = words[a:a + n]
        part[:, :, pk], part[:, :, pv], part[:, :, pm] = kw, vw, meta
    width = max(1, max(need))
    table, at = [], 0
    for c in need:
        table.append(ids[at:at + c] + [0] * (width - c))
        at += c
    s = {"op": op, "cache": cache, "page_table": ints(table), "kv_lens": ints(kv_lens), "hq": hq, "hkv": hkv,
         "max_kv": max(kv_lens), "max_q": max(q_lens)}
    if op in ("append", "gather"):
        place = [p for t, n in zip(q_lens, kv_lens) for p in range(n - t, n)]
        slot = [row[p // PAGE] * PAGE + p % PAGE for row, t, n in zip(table, q_lens, kv_lens) for p in range(n - t, n)]
        s["slots"] = ints(slot)
        if op == "append":
            s["positions"], s["rope"] = ints(place), _rope(max(kv_lens), dev)
            s["qkv"] = normal(len(slot), (hq + 2 * hkv) * DIM).bfloat16()
            s["bias"] = (normal((hq + 2 * hkv) * DIM) / 2).bfloat16()
        return s
    s["scale"], s["sinks"] = 1 / 8, normal(hq) * 2
    s["scratch"] = torch.zeros(SCRATCH_BYTES, dtype=torch.uint8, device=dev)
    s["cu_q"] = ints([0] + torch.tensor(q_lens).cumsum(0).tolist())
    s["q"] = normal(sum(q_lens), hq, DIM).bfloat16()
    s["tree"] = None
    if op == "verify":
        s["q"] = s["q"].view(batch, case["q_len"], hq, DIM)
        if case["tree"]:
            # each draft token hangs off an earlier one or off the prefix, and sees itself and its ancestors
            rows = []
            for _ in range(batch):
                bits = []
                for u in range(case["q_len"]):
                    above = rng.randint(-1, u - 1)
                    bits.append((bits[above] if above >= 0 else 0) | 1 << u)
                rows.append([b - (1 << 64) if b >> 63 else b for b in bits])
            s["tree"] = torch.tensor(rows, dtype=torch.int64, device=dev)
    return s


# ------------------------------------------------------------- plain forms
def _hidden(s):
    """[request, row, key]: the keys that a row does not see; and the flat number of each row, and whether it is one."""
    n = s["kv_lens"].long()
    cu = s["cu_q"].long()
    q_len = cu[1:] - cu[:-1]
    i = torch.arange(s["max_q"], device=n.device)
    live = i < q_len[:, None]
    row = torch.where(live, cu[:-1, None] + i, 0)
    j = torch.arange(max(s["max_kv"], 1), device=n.device)
    old = (n - q_len)[:, None, None]
    seen = j <= old + i[:, None]
    if s["tree"] is not None:
        bit = (s["tree"][..., None] >> (j - old).clamp(0, 63)) & 1
        seen = (j < old) | (bit == 1)
    return ~seen | (j >= n[:, None, None]), row, live


def _plain_attention(s):
    """Scores of all rows and keys of one KV head after another, a softmax with the sink as one more logit."""
    hidden, row, live = _hidden(s)
    q = s["q"].view(-1, s["hq"], DIM)
    words = s["cache"].view(torch.int32)
    keys = hidden.shape[2]
    group = s["hq"] // s["hkv"]
    out, lse = torch.empty_like(q), torch.empty(q.shape[:2], device=q.device)
    table = s["page_table"].long()
    gone = (torch.arange(keys, device=q.device) >= s["kv_lens"][:, None])[..., None]
    for h in range(s["hkv"]):
        k, v = _page_rows(words[table, h])
        k, v = k.flatten(1, 2)[:, :keys], v.flatten(1, 2)[:, :keys].masked_fill(gone, 0)
        heads = slice(h * group, (h + 1) * group)
        sc = torch.einsum("rigd,rjd->rgij", q[row, heads].float(), k) * s["scale"]
        sc = sc.masked_fill_(hidden[:, None], -math.inf)
        sink = s["sinks"][heads][:, None].expand(sc.shape[:-1])
        top = torch.maximum(sc.amax(-1), sink)
        e = sc.sub_(top[..., None]).exp_()
        total = e.sum(-1) + torch.exp(sink - top)
        o = torch.einsum("rgij,rjd->rigd", e, v) / total.transpose(1, 2)[..., None]
        out[row[live], heads] = o[live].to(q.dtype)
        lse[row[live], heads] = (top + total.log()).transpose(1, 2)[live]
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}


def _plain_gather(s):
    slot = s["slots"].long()
    words = s["cache"].view(torch.int32)[slot // PAGE]
    pk, pv, pm = (p[slot % PAGE] for p in _places(slot.device))
    h = torch.arange(s["hkv"], device=slot.device)
    t = torch.arange(slot.numel(), device=slot.device)[:, None]
    k, v = _words_to_rows(words[t[..., None], h[:, None], pk[:, None]], words[t[..., None], h[:, None], pv[:, None]],
                          words[t, h, pm[:, None]])
    return {"k": k.bfloat16(), "v": v.bfloat16()}


def _plain_append(s):
    hq, hkv = s["hq"], s["hkv"]
    x = (s["qkv"].float() + s["bias"].float()).unflatten(-1, (-1, DIM))
    cos, sin = s["rope"][s["positions"].long()][:, None].split(DIM // 2, -1)
    a, b = x[:, :hq + hkv].split(DIM // 2, -1)
    qk = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    slot = s["slots"].long()
    words = s["cache"].view(torch.int32)
    kw, vw, meta = _rows_to_words(qk[:, hq:], x[:, hq + hkv:])
    pk, pv, pm = (p[slot % PAGE] for p in _places(slot.device))
    page, h = (slot // PAGE)[:, None], torch.arange(hkv, device=slot.device)
    words[page[..., None], h[:, None], pk[:, None]] = kw
    words[page[..., None], h[:, None], pv[:, None]] = vw
    words[page, h, pm[:, None]] = meta
    return {"q": qk[:, :hq].bfloat16(), **_plain_gather(s)}


PLAIN = {"decode": _plain_attention, "verify": _plain_attention, "prefill": _plain_attention,
         "append": _plain_append, "gather": _plain_gather}


# ------------------------------------------------------- the library's calls
def _own(s):
    import gqa_attention_learned_gb300 as sa

    op = s["op"]
    if op in ("append", "gather"):
        got = {}
        if op == "append":
            got["q"] = sa.qkv_prologue_int4(s["qkv"], s["bias"], s["positions"], s["slots"], s["rope"], s["cache"],
                                            s["hq"], s["hkv"])
        # what was appended, as the values that it stands for
        got["k"], got["v"] = sa.gather_int4(s["cache"], s["slots"])
        return got
    paged = [s[n] for n in ("cache", "page_table", "kv_lens", "sinks", "scale")]
    if op == "decode":
        out, lse = sa.decode_int4(s["q"], *paged, s["max_kv"], workspace=s["scratch"])
    elif op == "verify":
        out, lse = sa.verify_int4(s["q"], *paged, s["max_kv"], tree_mask=s["tree"], workspace=s["scratch"])
    else:
        out, lse = sa.prefill_paged_int4(s["q"], s["cu_q"], *paged, s["max_q"], s["max_kv"], workspace=s["scratch"])
    return {"out": out, "lse": lse}


def run(state):
    if own:
        return _own(state)
    return PLAIN[state["op"]](state)


# --------------------------------------------------------------------- work
def work(case):
    """What one call cannot do without: every input that counts read once, every output written once.  An appended
    row is written packed and read back."""
    op, hq, hkv = case["op"], case["hq"], case["hkv"]
    q_lens, kv_lens = _lengths(case)
    row = 2 * DIM                                     # bytes of one head's bf16 row
    tokens, keys = sum(q_lens), sum(kv_lens)
    read = tokens * hkv * (ROW_BYTES + 2 * row)
    if op == "gather":
        return {"bytes": read, "flops": 0}
    if op == "append":
        return {"bytes": tokens * ((2 * hq + 2 * hkv) * row + hkv * ROW_BYTES + 4 * DIM) + read, "flops": 0}
    pairs = sum(sum(range(n - t + 1, n + 1)) for t, n in zip(q_lens, kv_lens) if n)
    return {"bytes": tokens * hq * (2 * row + 4) + keys * hkv * ROW_BYTES, "flops": 4 * DIM * hq * pairs}


# -------------------------------------------------------------------- 64 bits
def _nibbles(b):
    """Bytes [...] as codes [..., 2], the low one first."""
    return torch.stack([b & 15, b >> 4], -1)


def _slot_values(block, j):
    """k, v [..., 64] in 64 bits that slot j of blocks [..., 1088] of bytes holds."""
    block = block.long()
    at = 64 * (j % 8) + 8 * (j // 8)
    k = torch.empty(*block.shape[:-1], DIM, dtype=torch.int64, device=block.device)
    v = torch.empty_like(k)
    for t in range(4):
        for u in range(2):
            b = block[..., at + 16 * t + 4 * u:at + 16 * t + 4 * u + 4]
            w = b[..., 0] + (b[..., 1] << 8) + (b[..., 2] << 16) + (b[..., 3] << 24)
            w = (w >> 3) + ((w & 7) << 29)
            k[..., 32 * u + 8 * t:32 * u + 8 * t + 8] = torch.stack([(w >> 4 * e) & 15 for e in range(8)], -1)
    for g in range(8):
        a = 512 + 64 * g + 16 * (j % 8 // 2) + 8 * (j // 8) + 4 * (j % 2)
        v[..., 8 * g:8 * g + 8] = _nibbles(block[..., a:a + 4]).flatten(-2)
    m = block[..., 1024 + 8 * (j % 8) + 4 * (j // 8):][..., :4]

    def values(n, low, high):
        e, f = ((high & 127) << 1) + (low >> 7), (low >> 4) & 7
        s = torch.ldexp(1 + f.double() / 8, e - 127)
        return s[..., None] * (n - (low & 15)[..., None]).double()

    return values(k, m[..., 0], m[..., 1]), values(v, m[..., 2], m[..., 3])


def _request(s, b):
    """One request's keys and values [Hkv, n, 64], in 64 bits."""
    n = int(s["kv_lens"][b])
    pages = s["cache"][s["page_table"][b, :-(-n // PAGE)].long()]
    out = [torch.empty(s["hkv"], pages.shape[0], PAGE, DIM, dtype=torch.float64, device=pages.device) for _ in range(2)]
    for j in range(PAGE):
        for full, part in zip(out, _slot_values(pages, j)):
            full[:, :, j] = part.transpose(0, 1)
    return [full.flatten(1, 2)[:, :n] for full in out]


def _exact_attention(s):
    q = s["q"].double().view(-1, s["hq"], DIM)
    out, lse = torch.zeros_like(q), torch.zeros(q.shape[:2], dtype=torch.float64, device=q.device)
    sinks, group = s["sinks"].double(), s["hq"] // s["hkv"]
    for b in range(s["kv_lens"].numel()):
        lo, hi = int(s["cu_q"][b]), int(s["cu_q"][b + 1])
        k, v = _request(s, b)
        n = k.shape[1]
        for a in range(lo, hi, 512):
            z = min(a + 512, hi)
            at = torch.arange(a - lo, z - lo, device=q.device)
            old, top = n - (hi - lo), n - (hi - z)     # keys before the new tokens; keys that the last row may see
            if s["tree"] is not None:
                top = n
            see = torch.arange(top, device=q.device) <= old + at[:, None]
            if s["tree"] is not None:
                masks = s["tree"][b].tolist()
                for i in at.tolist():
                    see[i - (a - lo), old:] = torch.tensor([(masks[i] >> u) & 1 == 1 for u in range(hi - lo)], device=q.device)
            for g in range(s["hkv"]):
                hs = slice(g * group, (g + 1) * group)
                sc = (q[a:z, hs] @ k[g, :top].T) * s["scale"]
                sc[~see[:, None].expand_as(sc)] = -math.inf
                full = torch.logsumexp(torch.cat([sc, sinks[hs].expand(z - a, -1)[..., None]], -1), -1)
                out[a:z, hs] = torch.exp(sc - full[..., None]) @ v[g, :top]
                lse[a:z, hs] = full
    return {"out": out.view(s["q"].shape), "lse": lse.view(s["q"].shape[:-1])}


def _exact_rows(s):
    slot = s["slots"].cpu().numpy()
    k = torch.empty(slot.size, s["hkv"], DIM, dtype=torch.float64, device=s["cache"].device)
    v = torch.empty_like(k)
    for j in range(PAGE):
        at = np.flatnonzero(slot % PAGE == j)
        here = torch.from_numpy(at).to(k.device)
        k[here], v[here] = _slot_values(s["cache"][torch.from_numpy(slot[at] // PAGE).long().to(k.device)], j)
    return {"k": k, "v": v}


def _nearest(x):
    """Rows x [..., 64] in 64 bits, each value replaced by the one that its code stands for."""
    least = torch.minimum(x.min(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
    most = torch.maximum(x.max(-1).values, torch.zeros((), dtype=x.dtype, device=x.device))
    step = (most - least) / 15
    unit = torch.exp2(torch.floor(torch.log2(step.clamp(min=2.0 ** -126))) - 3)
    step = torch.ceil(step.clamp(min=2.0 ** -126) / unit) * unit
    zero = torch.round(-least / step)
    code = torch.clamp(torch.round(x / step[..., None]) + zero[..., None], 0, 15)
    return (code - zero[..., None]) * step[..., None]


def _exact_append(s):
    hq, hkv, half = s["hq"], s["hkv"], DIM // 2
    x = (s["qkv"].double() + s["bias"].double()).reshape(-1, hq + 2 * hkv, DIM)
    turn = s["rope"].double()[s["positions"].long()]
    turn = torch.complex(turn[:, None, :half], turn[:, None, half:])
    z = torch.complex(x[..., :half], x[..., half:])[:, :hq + hkv] * turn
    qk = torch.cat([z.real, z.imag], -1)
    return {"q": qk[:, :hq], "k": _nearest(qk[:, hq:]), "v": _nearest(x[:, hq + hkv:])}


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "append":
        return _exact_append(s)
    return _exact_rows(s) if s["op"] == "gather" else _exact_attention(s)
