"""Windowed attention, attention mass and eviction without a GPU: the oracle's
hand-worked pins, the split plan, and every host-side refusal."""

import ctypes
import os

import numpy as np
import pytest
import torch

import gqa_attention_learned_gb300 as sa
import oracle
from oracle import bounded


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(sa.LIB_PATH):
        from gqa_attention_learned_gb300 import build
        build.build()
    return sa.load()


# ------------------------------------------------------------------ oracle
def test_visible_keys_by_hand():
    see = lambda pos, w, f: np.flatnonzero(bounded.visible(pos, 10, w, f)).tolist()  # noqa: E731
    assert see(0, 1, 0) == [0]
    assert see(5, 1, 0) == [5]
    assert see(5, 3, 0) == [3, 4, 5]
    assert see(5, 3, 2) == [0, 1, 3, 4, 5]
    assert see(5, 3, 9) == [0, 1, 2, 3, 4, 5]
    assert see(9, 100, 0) == list(range(10))
    assert see(-1, 3, 2) == []


def test_a_wide_window_is_full_attention():
    rng = np.random.default_rng(0)
    q, k, v = rng.standard_normal((7, 4, 64)), rng.standard_normal((7, 2, 64)), rng.standard_normal((7, 2, 64))
    sinks = rng.standard_normal(4)
    ro, rl = oracle.prefill(q, k, v, [0, 7], sinks, 0.125)
    for w, f in ((7, 0), (100, 3), (1, 7)):
        out, lse = bounded.window_rows(q, k, v, range(7), sinks, 0.125, w, f)
        np.testing.assert_allclose(out, ro, atol=1e-12)
        np.testing.assert_allclose(lse, rl, atol=1e-12)


def test_a_window_of_one_sees_itself():
    # one visible key: out = v * sigmoid(s - sink)
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((3, 1, 64)), rng.standard_normal((3, 1, 64)), rng.standard_normal((3, 1, 64))
    out, _ = bounded.window_rows(q, k, v, range(3), np.array([0.3]), 0.125, 1)
    s = 0.125 * np.einsum("td,td->t", q[:, 0], k[:, 0])
    np.testing.assert_allclose(out[:, 0], v[:, 0] / (1 + np.exp(0.3 - s))[:, None], atol=1e-12)


def test_mass_sums_to_the_weights_that_are_not_the_sinks():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((6, 4, 64)), rng.standard_normal((9, 2, 64))
    sinks = rng.standard_normal(4)
    pos = list(range(3, 9))
    _, lse = bounded.window_rows(q, k, k, pos, sinks, 0.125, 9)
    mass = bounded.mass_rows(q, k, pos, lse, 0.125)
    want = (1 - np.exp(sinks - lse)).sum(0).reshape(2, 2).sum(1)
    np.testing.assert_allclose(mass.sum(1), want, atol=1e-12)
    assert np.all(mass[:, -1] < mass.sum(1))


def test_keep_by_hand():
    m = np.array([5, 1, 9, 1, 7, 1, 0, 0], float)
    assert bounded.keep(m, 8, 8, 0, 0) == list(range(8))
    assert bounded.keep(m, 8, 3, 0, 0) == [0, 2, 4]
    assert bounded.keep(m, 8, 4, 0, 0) == [0, 1, 2, 4]           # the tie goes to the lower index
    assert bounded.keep(m, 8, 4, 1, 2) == [0, 2, 6, 7]
    assert bounded.keep(m, 8, 3, 1, 2) == [0, 6, 7]
    m[2] = np.nan
    assert bounded.keep(m, 8, 3, 0, 0) == [0, 1, 4]
    assert bounded.keep(m, 3, 5, 0, 0) == [0, 1, 2]


# -------------------------------------------------------------------- plan
def test_the_window_plan_covers_the_visible_pages_only(lib):
    # 128 keys and 4 first tokens of a long request: 10 pages at most, so few chunks
    s, ws = sa.decode_window_plan(1, 64, 8, 131072, 128, 4, num_splits=64, num_sms=152)
    assert s <= 10 and ws > 0
    assert sa.decode_window_plan(64, 64, 8, 131072, 128, 4, num_sms=152)[0] == 1
    # a window without bound plans for every page
    whole = sa.decode_window_plan(8, 64, 8, 131072, 131072, 0, num_sms=152)
    assert whole[0] > 8
    assert sa.decode_window_plan(8, 64, 8, 131072, 2**31 - 1, 2**31 - 1, num_sms=152) == whole
    assert sa.decode_window_plan(1, 8, 1, 0, 5, num_sms=152) == (1, 0)
    for bad in (dict(window=0), dict(window=-1), dict(first_tokens=-1), dict(head_dim=128)):
        kw = dict(window=1, first_tokens=0)
        kw.update(bad)
        with pytest.raises(sa.SinkAttnError):
            sa.decode_window_plan(1, 8, 1, 100, num_sms=1, **kw)


# ---------------------------------------------------------------- refusals
FAKE, ODD = ctypes.c_void_p(0x10000), ctypes.c_void_p(0x10008)


def _call(fn, order, defaults, **kw):
    args = dict(defaults)
    assert set(kw) <= set(args), kw
    args.update(kw)
    return fn(*[args[n] for n in order.split()])


def test_decode_window_refusals(lib):
    order = ("q k v table maxp lens sinks scale window first out lse batch hq hkv d page pages "
             "maxkv splits ws wsb flags stream")
    good = dict(q=FAKE, k=FAKE, v=FAKE, table=FAKE, maxp=1, lens=FAKE, sinks=FAKE, scale=0.125,
                window=4, first=0, out=FAKE, lse=None, batch=1, hq=8, hkv=1, d=64, page=16, pages=1,
                maxkv=16, splits=0, ws=None, wsb=0, flags=0, stream=None)

    def call(**kw):
        return _call(lib.sinkattn_decode_window, order, good, **kw)

    assert call(batch=0) == sa.OK
    for kw in (dict(window=0), dict(first=-1), dict(hq=6, hkv=4), dict(pages=0), dict(flags=3),
               dict(scale=float("inf")), dict(q=None), dict(q=ODD), dict(out=None), dict(maxkv=-1)):
        assert call(**kw) == sa.INVALID_ARGUMENT, kw
    assert call(d=128) == sa.UNSUPPORTED
    assert call(page=32) == sa.UNSUPPORTED


def test_prefill_window_refusals(lib):
    order = "q k v cu n total maxs sinks scale window first out lse hq hkv d stream"
    good = dict(q=FAKE, k=FAKE, v=FAKE, cu=FAKE, n=1, total=4, maxs=4, sinks=FAKE, scale=0.125,
                window=4, first=0, out=FAKE, lse=None, hq=8, hkv=1, d=64, stream=None)

    def call(**kw):
        return _call(lib.sinkattn_prefill_window, order, good, **kw)

    assert call(n=0) == sa.OK and call(total=0) == sa.OK
    for kw in (dict(window=0), dict(first=-1), dict(hq=6, hkv=4), dict(scale=float("nan")),
               dict(q=None), dict(k=ODD), dict(cu=None), dict(sinks=None), dict(total=-1)):
        assert call(**kw) == sa.INVALID_ARGUMENT, kw
    assert call(d=32) == sa.UNSUPPORTED
    assert call(hq=129, hkv=1) == sa.UNSUPPORTED

    order = ("q cu n total maxq k v table maxp lens pages maxkv sinks scale window first out lse hq "
             "hkv d page stream")
    good = dict(q=FAKE, cu=FAKE, n=1, total=4, maxq=4, k=FAKE, v=FAKE, table=FAKE, maxp=1, lens=FAKE,
                pages=1, maxkv=16, sinks=FAKE, scale=0.125, window=4, first=0, out=FAKE, lse=None,
                hq=8, hkv=1, d=64, page=16, stream=None)

    def paged(**kw):
        return _call(lib.sinkattn_prefill_paged_window, order, good, **kw)

    assert paged(n=0) == sa.OK
    for kw in (dict(window=0), dict(first=-1), dict(table=None), dict(lens=None), dict(pages=0),
               dict(maxp=0), dict(v=ODD), dict(maxkv=-1)):
        assert paged(**kw) == sa.INVALID_ARGUMENT, kw
    assert paged(page=8) == sa.UNSUPPORTED


def test_mass_refusals(lib):
    order = "q k table maxp lens lse scale mass stride batch hq hkv d page pages maxkv stream"
    good = dict(q=FAKE, k=FAKE, table=FAKE, maxp=1, lens=FAKE, lse=FAKE, scale=0.125, mass=FAKE,
                stride=16, batch=1, hq=8, hkv=1, d=64, page=16, pages=1, maxkv=16, stream=None)

    def call(**kw):
        return _call(lib.sinkattn_decode_mass, order, good, **kw)

    assert call(batch=0) == sa.OK
    assert call(mass=None, stride=0, maxkv=0) == sa.OK
    for kw in (dict(stride=15), dict(lse=None), dict(mass=None), dict(hq=6, hkv=4), dict(q=ODD),
               dict(mass=ctypes.c_void_p(0x10002)), dict(scale=float("nan")), dict(batch=-1)):
        assert call(**kw) == sa.INVALID_ARGUMENT, kw
    assert call(d=128) == sa.UNSUPPORTED

    order = ("q cu n total maxq k table maxp lens pages maxkv lse scale mass stride hq hkv d page "
             "stream")
    good = dict(q=FAKE, cu=FAKE, n=1, total=4, maxq=4, k=FAKE, table=FAKE, maxp=1, lens=FAKE, pages=1,
                maxkv=16, lse=FAKE, scale=0.125, mass=FAKE, stride=16, hq=8, hkv=1, d=64, page=16,
                stream=None)

    def prefill(**kw):
        return _call(lib.sinkattn_prefill_mass, order, good, **kw)

    assert prefill(n=0) == sa.OK and prefill(total=0) == sa.OK
    for kw in (dict(cu=None), dict(stride=3), dict(maxq=-1), dict(k=ODD)):
        assert prefill(**kw) == sa.INVALID_ARGUMENT, kw
    assert prefill(hq=256, hkv=1) == sa.UNSUPPORTED


def test_evict_refusals(lib):
    order = ("k v table maxp lens mass stride budget first recent dtable dmaxp dmass dstride new kept "
             "batch hkv d page pages maxkv stream")
    p = lambda a: ctypes.c_void_p(a)  # noqa: E731
    good = dict(k=p(0x10000), v=p(0x20000), table=p(0x30000), maxp=4, lens=p(0x40000), mass=p(0x50000),
                stride=64, budget=8, first=2, recent=2, dtable=None, dmaxp=0, dmass=None, dstride=0,
                new=p(0x60000), kept=p(0x70000), batch=2, hkv=2, d=64, page=16, pages=8, maxkv=64,
                stream=None)

    def call(**kw):
        return _call(lib.sinkattn_evict, order, good, **kw)

    assert call(batch=0) == sa.OK
    for kw in (dict(budget=0), dict(first=-1), dict(recent=-1), dict(first=5, recent=4),
               dict(first=2**31 - 1, recent=2**31 - 1), dict(stride=63), dict(new=p(0x40004)),
               dict(new=None), dict(kept=None), dict(mass=None), dict(dtable=p(0x80000), dmaxp=0),
               dict(dmass=p(0x90000), dstride=7), dict(dmass=p(0x50000), dstride=32),
               dict(dmass=p(0x50010), dstride=64), dict(pages=0), dict(k=p(0x10004))):
        assert call(**kw) == sa.INVALID_ARGUMENT, kw
    assert call(d=128) == sa.UNSUPPORTED


def test_the_binding_refuses_before_the_library(lib):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    kc = torch.zeros(3, 1, 16, 64, dtype=torch.bfloat16)
    table, lens = torch.zeros(2, 1, dtype=torch.int32), torch.ones(2, dtype=torch.int32)
    sinks = torch.zeros(4)
    with pytest.raises(ValueError):                       # CPU tensors
        sa.decode_window(q, kc, kc, table, lens, sinks, 0.125, 16, 4)
    with pytest.raises(TypeError):
        sa.decode_mass(q.float(), kc, table, lens, torch.zeros(2, 4), 0.125, 16, torch.zeros(2, 1, 16))
    with pytest.raises(ValueError):
        sa.evict(kc, kc, table, lens, torch.zeros(2, 1, 16), 0, 16)
    assert sa._size(2**40, "window", 1) == 2**31 - 1
    with pytest.raises(ValueError):
        sa._size(0, "window", 1)
