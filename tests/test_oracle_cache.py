"""Pins of the serving oracle against things other than itself, and the refusals of the rotary and
cache entry points that are made on the host (CPU only)."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
from oracle import cache as oc


def test_e4m3_matches_the_torch_cast_on_every_midpoint():
    vals = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()   # 0 .. 448, 126 codes
    mids = (vals[1:] + vals[:-1]) / 2
    y = np.concatenate([vals, mids, mids * (1 + 1e-9), mids * (1 - 1e-9)])
    y = np.concatenate([y, -y])
    want = torch.tensor(y, dtype=torch.float32)
    keep = want.double().numpy() == y                       # those that float32 holds exactly
    got = oc.e4m3(y)
    assert np.array_equal(got[keep], want.to(torch.float8_e4m3fn).double().numpy()[keep])
    assert np.isnan(oc.e4m3(np.nan)) and oc.e4m3(2.0 ** -10) == 0.0 and oc.e4m3(1.5 * 2.0 ** -9) == 2.0 ** -8


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (1.75, -8), (1.7500001, -7), (1.0, -8), (0.0, -117),
                                    (2.0 ** -133, -117), (3.3895313892515355e38, 120)])
def test_scale_exponent(amax, e):
    assert oc.scale_exponent(amax) == e


def test_rope_against_complex_numbers_and_its_invariances():
    rng = np.random.default_rng(0)
    x = rng.standard_normal((2, 3, 5, 12))
    pos, w = rng.integers(0, 1000, (2, 5)), 10000.0 ** (-np.arange(4) / 4)
    for inter in (False, True):
        y = oc.rope(x, pos, w, inter, 1.3)
        i1, i2 = (np.arange(0, 8, 2), np.arange(1, 8, 2)) if inter else (np.arange(4), np.arange(4, 8))
        z = (x[..., i1] + 1j * x[..., i2]) * np.exp(1j * pos[:, None, :, None] * w) * 1.3
        np.testing.assert_allclose(y[..., i1] + 1j * y[..., i2], z, atol=1e-12)
        assert np.array_equal(y[..., 8:], x[..., 8:])
        np.testing.assert_allclose(oc.rope(y, pos, w, inter, 1 / 1.3, True), x, atol=1e-12)
        # scores depend on the distance of positions alone
        a = oc.rope(x, pos, w, inter)[:, :, 1:2] @ oc.rope(x, pos, w, inter)[:, :, 3:4].swapaxes(2, 3)
        b = oc.rope(x, pos + 77, w, inter)[:, :, 1:2] @ oc.rope(x, pos + 77, w, inter)[:, :, 3:4].swapaxes(2, 3)
        np.testing.assert_allclose(a, b, atol=1e-9)


def test_cache_attention_of_a_whole_prompt_is_causal_attention_over_its_values():
    rng = np.random.default_rng(1)
    c = oc.Cache(pages=8, heads=2, page=16, Dh=64, slots=3, max_pages=6)
    k, v, q = (rng.standard_normal((1, 2, 40, 64)) for _ in range(3))
    assert c.reserve([1], [40])
    c.append([1], [40], k, v)
    kd, vd = c.values("k", 1)[None], c.values("v", 1)[None]
    assert np.abs(kd - k).max() <= np.abs(k).max() * 2.0 ** -4      # half a step of e4m3
    o, lse, _ = c.attend(1, q[0], 40)
    want_o, want_lse = oracle.attn_fwd_heads(q, kd, vd, True)
    np.testing.assert_allclose(o, np.asarray(want_o)[0], atol=1e-12)
    np.testing.assert_allclose(lse, np.asarray(want_lse)[0], atol=1e-12)


def test_appending_token_by_token_restates_older_codes_only_when_the_scale_grows():
    c = oc.Cache(4, 1, 16, 64, 1, 2)
    xs = [0.5, 100.0, 3.0, 1e4]
    for i, x in enumerate(xs):
        assert c.reserve([0], [1])
        new = np.full((1, 1, 1, 64), x)
        c.append([0], [1], new, new)
        got = c.values("k", 0)[0, :, 0]
        want = np.array(xs[:i + 1])
        assert np.all(np.abs(got - want) <= np.maximum(want * 2.0 ** -4, 2.0 ** (c.exp["k"][c.table[0, 0], 0] - 10)) * 1.001)


def test_pages_are_shared_copied_trimmed_and_compacted():
    c = oc.Cache(10, 1, 16, 64, 4, 5)
    rng = np.random.default_rng(2)
    x = rng.standard_normal((1, 1, 20, 64))
    c.reserve([0], [20])
    c.append([0], [20], x, x)
    before = c.values("k", 0).copy()
    c.fork([0, 0], [1, 2])
    assert list(c.refs[:2]) == [3, 3]
    assert c.reserve([0, 1, 2], [1, 1, 1])                  # two copies, the last holder keeps the page
    assert list(c.refs[:4]) == [3, 1, 1, 1] and c.table[2, 1] == 1
    y = rng.standard_normal((3, 1, 1, 64))
    c.append([0, 1, 2], [1, 1, 1], y, y)
    for s in range(3):
        assert np.array_equal(c.values("k", s)[:, :16], before[:, :16])
    keep = c.values("k", 2).copy()
    c.trim([0, 1], [0, 16])
    assert list(c.refs[:4]) == [2, 1, 0, 0]
    assert not c.reserve([3], [16 * 9]) and c.lens[3] == 0
    c.reserve([3], [16 * 2])
    c.trim([1], [0])
    c.trim([2], [21])
    c.compact()
    assert np.array_equal(c.values("k", 2), keep) and sorted(np.flatnonzero(c.refs)) == [0, 1, 2, 3]


# ------------------------------------------------------------------------------------ host-side refusals
@pytest.fixture(scope="module")
def ra(lib_path):
    from long_context_exact_fwd_b200 import ring_attn
    return ring_attn


P = ctypes.c_void_p
LL = ctypes.c_longlong


def test_rope_argument_errors(ra):
    f = ra.raw.ring_attn_rope

    def call(**kw):
        st = (LL * 6)(*kw.get("strides", (4 * 384, 384, 128, 4 * 384, 384, 128)))
        kst = (LL * 6)(4 * 384, 384, 128, 4 * 384, 384, 128)
        k = kw.get("k", 0)
        return f(P(kw.get("q", 1 << 20)), P(kw.get("out", 1 << 24)), kw.get("Hq", 4), st, P(k) if k else None,
                 P(kw.get("k_out", 1 << 28)) if k else None, kw.get("Hk", 4 if k else 0), kst if k else None,
                 kw.get("B", 2), kw.get("S", 3), kw.get("Dh", 128), P(kw.get("steps", 256)), kw.get("rot", 128), 0,
                 kw.get("amp", 1.0), P(kw.get("pos", 0)) if kw.get("pos") else None, kw.get("pos_b", 0), 1, 0, 0,
                 kw.get("dtype", 0), None)

    assert call(q=0) == ra.RA_ERR_ARG and call(steps=0) == ra.RA_ERR_ARG and call(B=0) == ra.RA_ERR_ARG
    assert call(Hq=0) == ra.RA_ERR_ARG and call(dtype=5) == ra.RA_ERR_ARG
    assert call(amp=float("nan")) == ra.RA_ERR_ARG and call(amp=float("inf")) == ra.RA_ERR_ARG
    for rot in (0, -2, 3, 130):
        assert call(rot=rot) == ra.RA_ERR_SHAPE
    assert call(Dh=127) == ra.RA_ERR_SHAPE and call(Dh=2048, rot=64) == ra.RA_ERR_SHAPE
    assert call(strides=(4 * 384, 384, 128, 4 * 384, 384, 64)) == ra.RA_ERR_SHAPE       # output rows fold together
    assert call(strides=(4 * 384, 384, 128, 384, 384, 128)) == ra.RA_ERR_SHAPE          # batches on heads
    assert call(strides=(-8, 384, 128, 4 * 384, 384, 128)) == ra.RA_ERR_SHAPE
    assert call(out=(1 << 20) + 256) == ra.RA_ERR_ARG                                   # half over the input
    assert call(out=1 << 20, strides=(4 * 384, 384, 128, 4 * 384, 128, 4 * 128)) == ra.RA_ERR_ARG   # in place, permuted
    assert call(q=(1 << 20) + 1) == ra.RA_ERR_ALIGN and call(steps=260) == ra.RA_ERR_ALIGN
    assert call(pos=256, pos_b=-1) == ra.RA_ERR_SHAPE and call(pos=260) == ra.RA_ERR_ALIGN
    assert call(k=1 << 26, k_out=1 << 24) == ra.RA_ERR_ARG                              # both outputs on one
    if not torch.cuda.is_available():
        assert call() in (ra.RA_ERR_CUDA, ra.RA_ERR_DEVICE)
        assert call(out=1 << 20) in (ra.RA_ERR_CUDA, ra.RA_ERR_DEVICE)                  # in place is fine
        assert call(k=1 << 26) in (ra.RA_ERR_CUDA, ra.RA_ERR_DEVICE)


def _cache_struct(ra, **kw):
    d = dict(k=1 << 20, v=1 << 30, k_scale=256, v_scale=512, table=1024, lens=2048, refs=4096, layers=2, pages=100, heads=4,
             page=64, head_dim=128, slots=8, max_pages=16)
    d.update(kw)
    return ctypes.byref(ra._CacheStruct(*d.values()))


BAD_CACHES = [(dict(k=0), "RA_ERR_ARG"), (dict(lens=0), "RA_ERR_ARG"), (dict(layers=0), "RA_ERR_ARG"),
              (dict(pages=0), "RA_ERR_ARG"), (dict(max_pages=-1), "RA_ERR_ARG"), (dict(page=48), "RA_ERR_SHAPE"),
              (dict(page=256), "RA_ERR_SHAPE"), (dict(head_dim=96), "RA_ERR_SHAPE"),
              (dict(max_pages=1 << 25), "RA_ERR_SHAPE"), (dict(heads=40000), "RA_ERR_SHAPE"),
              (dict(k=(1 << 20) + 8), "RA_ERR_ALIGN"), (dict(table=1026), "RA_ERR_ALIGN")]


def _calls(ra, cache, **kw):
    """Every cache call on `cache` with good other arguments, replaced by keyword."""
    g = kw.get
    raw = ra.raw
    st = (LL * 3)(*g("strides", (4 * 5 * 128, 5 * 128, 128)))
    sl, n, B, T = P(g("slots", 256)), P(g("n_new", 512)), g("B", 3), g("T", 5)
    x = P(g("x", 1 << 20))
    ws, size, layer = P(g("ws", 256)), ctypes.c_size_t(g("size", 1 << 40)), g("layer", 1)
    return {
        "reserve": lambda: raw.ring_attn_cache_reserve(cache, sl, n, B, ws, size, None),
        "append": lambda: raw.ring_attn_cache_append(cache, layer, sl, n, B, T, x, st, P(1 << 22), st, None),
        "read": lambda: raw.ring_attn_cache_read(cache, layer, sl, n, B, T, x, P(g("x2", 1 << 22)), None),
        "attend": lambda: raw.ring_attn_cache_attend(cache, layer, sl, n, B, T, g("Hq", 8), x, st, 0.0, 1, P(g("o", 1 << 24)),
                                                     g("dtype", 0), P(g("lse", 1 << 26)), ws, size, None),
        "fork": lambda: raw.ring_attn_cache_fork(cache, sl, n, B, ws, size, None),
        "trim": lambda: raw.ring_attn_cache_trim(cache, sl, n, B, None),
        "compact": lambda: raw.ring_attn_cache_compact(cache, ws, size, None),
    }


@pytest.mark.parametrize("bad,code", BAD_CACHES)
def test_every_cache_call_refuses_a_bad_cache(ra, bad, code):
    for name, call in _calls(ra, _cache_struct(ra, **bad)).items():
        assert call() == getattr(ra, code), name


def test_cache_argument_errors(ra):
    c = _cache_struct(ra)

    def expect(names, code, **kw):
        calls = _calls(ra, c, **kw)
        for name in names.split():
            assert calls[name]() == code, (name, kw)

    batched = "reserve append read attend fork trim"
    expect(batched, ra.RA_ERR_ARG, slots=0)
    expect(batched, ra.RA_ERR_ARG, B=0)
    expect(batched, ra.RA_ERR_SHAPE, B=1025)
    expect(batched, ra.RA_ERR_ALIGN, slots=258)
    expect("reserve append attend read trim", ra.RA_ERR_ALIGN, n_new=514)
    expect("reserve fork", ra.RA_ERR_ARG, n_new=0)
    expect("append read attend", ra.RA_ERR_ARG, layer=2)
    expect("append read attend", ra.RA_ERR_ARG, layer=-1)
    expect("append read attend", ra.RA_ERR_ARG, T=0)
    expect("append read attend", ra.RA_ERR_ARG, x=0)
    expect("append read attend", ra.RA_ERR_ALIGN, x=(1 << 20) + 8)
    expect("append attend", ra.RA_ERR_ALIGN, strides=(2560, 640, 132))
    expect("append attend", ra.RA_ERR_SHAPE, strides=(2560, -640, 128))
    expect("read", ra.RA_ERR_ARG, x2=1 << 20)
    expect("attend", ra.RA_ERR_SHAPE, Hq=6)
    expect("attend", ra.RA_ERR_ARG, Hq=0)
    expect("attend", ra.RA_ERR_ARG, dtype=3)
    expect("attend", ra.RA_ERR_ARG, o=0)
    expect("attend", ra.RA_ERR_ALIGN, lse=(1 << 26) + 2)
    expect("attend", ra.RA_ERR_ARG, o=(1 << 20) + 256)                                  # the output over the queries
    for kw in (dict(ws=0), dict(ws=272), dict(size=64)):
        expect("reserve attend fork compact", ra.RA_ERR_WORKSPACE, **kw)
    if not torch.cuda.is_available():
        for name, call in _calls(ra, c).items():
            assert call() in (ra.RA_ERR_CUDA, ra.RA_ERR_DEVICE), name


def test_cache_workspace_sizes(ra):
    assert ra.cache_attend_workspace_bytes(0, 8, 8, 128) == 0 and ra.cache_attend_workspace_bytes(1, 8, 3, 128) == 0
    assert ra.cache_attend_workspace_bytes(1, 8, 8, 96) == 0
    assert ra.cache_attend_workspace_bytes(1, 32, 8, 128) >= 2 * 148 * 8 * 130 * 4
    assert ra.cache_pages_workspace_bytes(4, 0) == 0
    assert ra.cache_pages_workspace_bytes(4, 100) >= 4 * (100 + 8) and ra.cache_pages_workspace_bytes(0, 100) >= 1200


def test_rope_plans(ra):
    w, a = ra.rope_inv_freq(8)
    np.testing.assert_allclose(w.numpy(), [1.0, 0.1, 0.01, 0.001], rtol=1e-12)
    assert a == 1.0
    w4, _ = ra.rope_inv_freq(8, scaling="linear", factor=4.0)
    np.testing.assert_allclose(w4.numpy(), w.numpy() / 4, rtol=1e-15)
    wb, _ = ra.rope_inv_freq(8, scaling="base", factor=4.0)
    assert wb[0] == 1.0
    np.testing.assert_allclose(float(wb[-1]), 0.001 / 4, rtol=1e-12)
    wr, ar = ra.rope_inv_freq(64, scaling="ramp", factor=8.0, original_length=4096)
    full, _ = ra.rope_inv_freq(64)
    assert wr[0] == full[0] and abs(float(wr[-1]) * 8 / float(full[-1]) - 1) < 1e-12
    assert torch.all(wr <= full) and torch.all(wr >= full / 8) and abs(ar - (0.1 * math.log(8) + 1)) < 1e-15
    plan = ra.rope_plan(torch.tensor([2 * math.pi * 0.25, -2 * math.pi * 0.125, 2 * math.pi * 3.0]), device="cpu")
    steps = [s % (1 << 64) for s in plan.steps.tolist()]
    assert plan.rot == 6 and not plan.interleaved
    for got, want in zip(steps, (1 << 62, (1 << 64) - (1 << 61), 0)):
        # float32 input: the turn is known to 2^-24 of itself
        assert min(abs(got - want), (1 << 64) - abs(got - want)) < 3.5 * 2.0 ** 40 * 2
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=-1.0), dict(rot=8, factor=0.0), dict(rot=8, scaling="other"),
                dict(rot=8, scaling="ramp", factor=2.0), dict(rot=2, scaling="base", factor=2.0)):
        with pytest.raises(ValueError):
            ra.rope_inv_freq(**bad)
    for bad in (dict(layout="odd"), dict(amplitude=float("inf"))):
        with pytest.raises(ValueError):
            ra.rope_plan(w, device="cpu", **bad)
    with pytest.raises(ValueError):
        ra.rope_plan(torch.tensor([float("nan")]), device="cpu")


def test_the_bindings_refuse_cpu_tensors(ra):
    x = torch.zeros((1, 2, 3, 64), dtype=torch.bfloat16)
    plan = ra.rope_plan(ra.rope_inv_freq(64)[0], device="cpu")
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        ra.rope(x, plan)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        ra.kv_cache(1, 4, 2, 16, 64, 2, 2, device="cpu")


def test_a_table_whose_pages_cannot_be_counted_is_refused(ra):
    """A batch may ask for every entry of the table and a copy each; the plans add them up in 32 bits."""
    most = 2 ** 31 - 1 - 2 * 1024
    for slots, max_pages in ((17, (2 ** 31 - 1025) // 16), (2 ** 20, 2048), (most // 5 + 1, 5), (2 ** 31 - 1, 1)):
        for name, call in _calls(ra, _cache_struct(ra, slots=slots, max_pages=max_pages, page=16)).items():
            assert call() == ra.RA_ERR_SHAPE, (name, slots, max_pages)
    if not torch.cuda.is_available():
        for slots, max_pages in ((16, 2 ** 20), (most // 5, 5)):
            for name, call in _calls(ra, _cache_struct(ra, slots=slots, max_pages=max_pages, page=16)).items():
                assert call() in (ra.RA_ERR_CUDA, ra.RA_ERR_DEVICE), (name, slots, max_pages)


def test_outputs_over_other_tensors_are_refused(ra):
    f = ra.raw.ring_attn_rope
    B, S, Dh, Hq, Hk = 2, 3, 128, 4, 2

    def call(q, q_out, k, k_out, st, kst=None, st_out=None, kst_out=None):
        kst = kst or st
        return f(P(q), P(q_out), Hq, (LL * 6)(*st, *(st_out or st)), P(k), P(k_out), Hk, (LL * 6)(*kst, *(kst_out or kst)), B, S, Dh,
                 P(256), 128, 0, 1.0, None, 0, 0, 0, 0, 0, None)

    dense, kdense = (Hq * S * Dh, S * Dh, Dh), (Hk * S * Dh, S * Dh, Dh)
    row, fine = 2 * Dh, (ra.RA_OK, ra.RA_ERR_CUDA, ra.RA_ERR_DEVICE)     # bytes of a head's row
    q, k, qo, ko = 1 << 20, 1 << 22, 1 << 24, 1 << 26
    bad = [(q, k, k, ko), (q, qo, k, q), (q, q, k, q), (q, qo, k, qo),                 # one tensor for two
           (q, qo, k, qo + row), (q, qo, k, qo - row), (q, k + row, k, ko), (q, k - row, k, ko), (q, qo, k, q + row),
           (q, qo, k, qo + B * Hq * S * row - row), (q, q, k, q - B * Hk * S * row + row)]
    for args in bad:
        assert call(*args, dense, kdense) == ra.RA_ERR_ARG, args
    fused = (S * (Hq + 2 * Hk) * Dh, Dh, (Hq + 2 * Hk) * Dh)                           # heads of a projection's rows
    assert call(q, q, q + (Hq - 1) * row, q + (Hq - 1) * row, fused) == ra.RA_ERR_ARG
    heads = ((Hq + 2 * Hk) * S * Dh, S * Dh, Dh)                                       # heads one after the other
    assert call(q, q, q + (Hq - 1) * S * row, q + (Hq - 1) * S * row, heads) == ra.RA_ERR_ARG
    if not torch.cuda.is_available():
        for args in ((q, qo, k, ko), (q, q, k, k), (q, qo, q, ko), (q, qo, k, qo + B * Hq * S * row), (q, qo, k, qo - B * Hk * S * row)):
            assert call(*args, dense, kdense) in fine, args
        assert call(q, q, q + Hq * row, q + Hq * row, fused) in fine
        assert call(q, q, q + Hq * S * row, q + Hq * S * row, heads) in fine
        assert call(q, qo, q + Hq * row, ko, fused, None, dense, kdense) in fine

    c = _cache_struct(ra)
    n = 3 * 8 * 5                                                                      # rows of _calls' attend
    for kw in (dict(lse=1 << 24), dict(lse=(1 << 24) + n * 256 - 4), dict(lse=(1 << 24) - 4 * n + 4), dict(lse=1 << 20),
               dict(lse=(1 << 20) + 512)):
        assert _calls(ra, c, **kw)["attend"]() == ra.RA_ERR_ARG, kw
    for x2 in ((1 << 20) + 256, (1 << 20) - 256, (1 << 20) + 3 * 4 * 5 * 256 - 16):
        assert _calls(ra, c, x2=x2)["read"]() == ra.RA_ERR_ARG
    if not torch.cuda.is_available():
        assert _calls(ra, c, lse=(1 << 24) + n * 256)["attend"]() in fine
        assert _calls(ra, c, x2=(1 << 20) + 3 * 4 * 5 * 256)["read"]() in fine


# 100 digits behind the point
PI = "3.1415926535897932384626433832795028841971693993751058209749445923078164062862089986280348253421170679"


def exact_turns(theta, units=1):
    """theta / 2 pi * units of a double theta without whole turns, in (-units / 2, units / 2], to some 70 digits."""
    from decimal import Decimal, localcontext
    with localcontext() as c:
        c.prec = 110
        turns = Decimal(theta) / (2 * Decimal(PI)) * units
        return turns - units * (turns / units).to_integral_value()


def test_rope_steps_are_the_nearest(ra):
    thetas = [1.0, -1.0, 0.5, 2.5, 6.283185307179586, 1e-300, 1e-9, 1e9, -3e12, 1e20]
    for kw in (dict(), dict(base=500000.0), dict(scaling="linear", factor=3.0), dict(scaling="ramp", factor=8.0, original_length=8192)):
        thetas += ra.rope_inv_freq(128, **kw)[0].tolist()
    steps = ra.rope_plan(torch.tensor(thetas, dtype=torch.float64), device="cpu").steps.tolist()
    for theta, s in zip(thetas, steps):
        want = exact_turns(theta, 2 ** 64)
        whole = int(want)
        off = (whole - s + 2 ** 63) % 2 ** 64 - 2 ** 63 + float(want - whole)
        assert abs(off) <= 0.5000001, (theta, off)
