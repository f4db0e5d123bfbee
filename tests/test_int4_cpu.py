"""The paged cache held in 4 bits without a GPU: the format's properties, the
reference against hand-made rows, and every host-side refusal."""

import ctypes
import os

import numpy as np
import pytest
import torch

import gqa_attention_learned_gb300 as sa
from oracle import int4
from test_bounded_cpu import FAKE, ODD, _call


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sa.LIB_PATH):
        from gqa_attention_learned_gb300 import build
        build.build()
    return sa.load()


# ------------------------------------------------------------------ the format
def test_a_row_by_hand():
    # range 15: steps of one, zero point where the low end is
    x = np.zeros(64, np.float32)
    x[0], x[1], x[2], x[3] = -5, 10, 2.5, 3.5
    n, s, z = int4.quantise(x)
    assert float(s) == 1 and int(z) == 5
    assert n[:5].tolist() == [0, 15, 7, 9, 5]                # ties to even
    assert int4.round_trip(x)[:5].tolist() == [-5, 10, 2, 4, 0]
    # a step of 1.0625 (17 / 16) goes up to 9 / 8: four significant bits
    x[1] = 15 * 1.0625 - 5
    assert float(int4.quantise(x)[1]) == 1.125
    # one-sided rows keep zero, rows of zeros are zeros
    assert int4.quantise(np.full(64, 3.0, np.float32))[2] == 0
    assert int4.quantise(np.full(64, -3.0, np.float32))[2] == 15
    assert not int4.round_trip(np.zeros(64)).any()
    for bad in (np.nan, np.inf, -np.inf):
        x[9] = bad
        assert np.isnan(int4.round_trip(x)).all()


@pytest.mark.parametrize("scale", [2.0**-130, 1e-6, 1.0, 300.0, 1e37])
def test_every_value_is_bf16_and_within_a_step(scale):
    rng = np.random.default_rng(0)
    x = (rng.standard_normal((500, 64)) * scale + rng.standard_normal((500, 1)) * scale).astype(np.float32)
    n, s, z = int4.quantise(x)
    y = int4.stands_for(n, s, z)
    assert np.array_equal(torch.from_numpy(y).bfloat16().double().numpy(), y)
    inside = (n > 0) & (n < 15)
    err = np.abs(y - x)
    assert (err[inside] <= np.broadcast_to(s[:, None], n.shape)[inside] * (0.5 + 2.0**-20)).all()
    assert (err <= s[:, None] * (1 + 2.0**-20)).all()
    span = np.maximum(x.max(-1), 0).astype(np.float64) - np.minimum(x.min(-1), 0)
    assert (s >= span / 15 * (1 - 2.0**-22)).all()
    assert (s <= np.maximum(span / 15 * 1.125 * (1 + 2.0**-22), 2.0**-126)).all()


def test_what_is_written_is_read():
    rng = np.random.default_rng(1)
    cache = rng.integers(0, 256, (5, 3, int4.BLOCK)).astype(np.uint8)
    before = cache.copy()
    slots = rng.permutation(80)[:37]
    k, v = rng.standard_normal((37, 3, 64)), rng.standard_normal((37, 3, 64))
    k[3, 1, 5] = np.nan
    int4.write(cache, slots, k, v)
    for t, slot in enumerate(slots):
        rk, rv = int4.read(cache, slot // 16, slot % 16)
        np.testing.assert_array_equal(rk, int4.round_trip(k[t]))
        np.testing.assert_array_equal(rv, int4.round_trip(v[t]))
    # tokens own whole bytes: the others' are as they were
    for slot in set(range(80)) - set(slots):
        for a, b in zip(int4.read(cache, slot // 16, slot % 16), int4.read(before, slot // 16, slot % 16)):
            np.testing.assert_array_equal(a, b)
    assert (cache == before).sum() >= 43 * 3 * 68


def test_the_rope_table_is_the_rotary_angles():
    freq, ms = sa.yarn_table()
    table = sa.rope_table(freq, ms, 131072, device="cpu")
    assert table.shape == (131072, 64) and table.dtype == torch.float32
    for p in (0, 1, 4097, 131071):
        a = p * np.asarray(freq, np.float64)
        np.testing.assert_allclose(table[p].numpy(), ms * np.concatenate([np.cos(a), np.sin(a)]), rtol=2.0**-22, atol=2.0**-26)


# -------------------------------------------------------------------- workspace
def test_the_workspace_depends_on_the_gpu_alone(lib):
    assert sa.int4_workspace_bytes(152) % 256 == 0
    assert sa.int4_workspace_bytes(1) < sa.int4_workspace_bytes(152)
    with pytest.raises(sa.SinkAttnError):
        sa.int4_workspace_bytes(-1)


# -------------------------------------------------------------------- refusals
def test_prologue_refusals(lib):
    order = "qkv bias pos slots rope ropes style q cache tokens hq hkv d page pages stream"
    good = dict(qkv=FAKE, bias=None, pos=FAKE, slots=FAKE, rope=FAKE, ropes=1, style=0, q=FAKE, cache=FAKE,
                tokens=1, hq=8, hkv=1, d=64, page=16, pages=1, stream=None)

    def call(**kw):
        return _call(lib.sinkattn_qkv_prologue_int4, order, good, **kw)

    assert call(tokens=0) == sa.OK
    for kw in (dict(qkv=None), dict(pos=None), dict(slots=None), dict(rope=None), dict(q=None), dict(cache=None),
               dict(qkv=ODD), dict(bias=ODD), dict(cache=ODD), dict(ropes=0), dict(style=2), dict(tokens=-1),
               dict(hkv=0), dict(pages=0)):
        assert call(**kw) == sa.INVALID_ARGUMENT, kw
    assert call(d=128) == sa.UNSUPPORTED
    assert call(page=32) == sa.UNSUPPORTED
    assert call(tokens=2**28, hq=64, hkv=8) == sa.UNSUPPORTED
    assert call(hq=2**26) == sa.UNSUPPORTED


def test_gather_refusals(lib):
    order = "cache slots rows k v hkv d page pages stream"
    good = dict(cache=FAKE, slots=FAKE, rows=1, k=FAKE, v=FAKE, hkv=1, d=64, page=16, pages=1, stream=None)

    def call(**kw):
        return _call(lib.sinkattn_gather_int4, order, good, **kw)

    assert call(rows=0) == sa.OK
    for kw in (dict(cache=None), dict(slots=None), dict(k=None), dict(v=ODD), dict(rows=-1), dict(hkv=0),
               dict(pages=0)):
        assert call(**kw) == sa.INVALID_ARGUMENT, kw
    assert call(d=32) == sa.UNSUPPORTED
    assert call(rows=2**31 - 1, hkv=2**31 - 1) == sa.UNSUPPORTED


ATTENTION = dict(q=FAKE, cache=FAKE, table=FAKE, maxp=1, lens=FAKE, sinks=FAKE, scale=0.125, out=FAKE, lse=None,
                 hq=8, hkv=1, d=64, page=16, pages=1, maxkv=16, ws=FAKE, wsb=1 << 30, stream=None)
BAD = (dict(q=None), dict(cache=None), dict(table=None), dict(lens=None), dict(sinks=None), dict(out=None),
       dict(q=ODD), dict(cache=ODD), dict(out=ODD), dict(lse=ctypes.c_void_p(0x10002)), dict(hq=6, hkv=4),
       dict(hkv=0), dict(scale=float("nan")), dict(pages=0), dict(maxp=0), dict(maxkv=-1))


def test_decode_and_verify_refusals(lib):
    order = "q cache table maxp lens sinks scale out lse batch hq hkv d page pages maxkv ws wsb flags stream"
    good = dict(ATTENTION, batch=1, flags=0)

    def decode(**kw):
        return _call(lib.sinkattn_decode_int4, order, good, **kw)

    order_v = order.replace("lens", "lens mask").replace("batch", "batch qlen")

    def verify(**kw):
        return _call(lib.sinkattn_verify_int4, order_v, dict(good, mask=None, qlen=2), **kw)

    for call in (decode, verify):
        assert call(batch=0) == sa.OK
        for kw in BAD + (dict(batch=-1), dict(flags=3)):
            assert call(**kw) == sa.INVALID_ARGUMENT, kw
        assert call(d=128) == sa.UNSUPPORTED
        assert call(page=8) == sa.UNSUPPORTED
        assert call(batch=2**25, hq=64, hkv=8) == sa.UNSUPPORTED
    for kw in (dict(qlen=0), dict(qlen=65), dict(mask=ctypes.c_void_p(0x10004))):
        assert verify(**kw) == sa.INVALID_ARGUMENT, kw


def test_prefill_refusals(lib):
    order = "q cu n total maxq cache table maxp lens pages maxkv sinks scale out lse hq hkv d page ws wsb stream"
    good = dict(ATTENTION, cu=FAKE, n=1, total=4, maxq=4)

    def call(**kw):
        return _call(lib.sinkattn_prefill_paged_int4, order, good, **kw)

    assert call(n=0) == sa.OK and call(total=0) == sa.OK
    for kw in BAD + (dict(cu=None), dict(n=-1), dict(total=-1), dict(maxq=-1)):
        assert call(**kw) == sa.INVALID_ARGUMENT, kw
    assert call(d=128) == sa.UNSUPPORTED


def test_the_binding_refuses_before_the_library(lib):
    bf = torch.bfloat16
    q, cache = torch.zeros(2, 4, 64, dtype=bf), torch.zeros(3, 1, 1088, dtype=torch.uint8)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    sinks = torch.zeros(4)
    with pytest.raises(ValueError):                       # CPU tensors
        sa.decode_int4(q, cache, table, lens, sinks, 0.125, 16)
    with pytest.raises(TypeError):
        sa.decode_int4(q.float(), cache, table, lens, sinks, 0.125, 16)
    with pytest.raises(TypeError):
        sa.gather_int4(cache.int(), lens)
    with pytest.raises(ValueError):
        sa.qkv_prologue_int4(torch.zeros(2, 6 * 64, dtype=bf), None, lens, lens, torch.zeros(4, 64), cache, 4, 1)
    with pytest.raises(ValueError):
        sa.prefill_paged_int4(q, torch.zeros(0, dtype=torch.int32), cache, table, lens, sinks, 0.125, 1, 16)
