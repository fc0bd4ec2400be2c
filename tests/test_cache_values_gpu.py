"""Cache attention where pages' value scales lie far apart, with the oracle of test_cache_gpu.py.

Tolerance of a row, from the arithmetic (u = 2^-24), over the tokens j that the row sees, p_j its softmax
weights, s_j the value scale of token j's page:
  scores, P's bits, sums, output   as in test_cache_gpu.py;
  P's lower end   P is fp16 at 2^7 times p_j s_j over the row's largest such product (or up to 2^8 more): half a
              step of its smallest numbers is 2^-25, so a term is off by 2^-32 max_j (p_j s_j) times its code, at
              most 448."""
import numpy as np
import pytest
import torch

from test_cache_gpu import Both, _i32, _randn, ra  # noqa: F401

pytestmark = pytest.mark.gpu


def check_rows(c, slots, n_new, q, o, lse, scale, causal=True, seen=None):
    """o, lse of every new token against the oracle's values; seen[b] [len]: tokens that count at all."""
    half = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -24
    o, lse, q = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for b, s in enumerate(slots):
        k, v, n = c.values("k", s), c.values("v", s), int(c.lens[s])
        steps = np.repeat(np.ldexp(1.0, c.exp["v"][c.table[s, :c._count(n)]]), c.page, axis=0)[:n]   # [n, heads]
        g = q.shape[1] // c.heads
        for t in range(n_new[b]):
            m = min(n, n - n_new[b] + t + 1) if causal else n
            ok = np.arange(n) < m
            if seen is not None:
                ok &= seen[b]
            for h in range(q.shape[1]):
                if not ok.any():
                    assert np.all(o[b, h, t] == 0) and lse[b, h, t] == -np.inf
                    continue
                kk, vv, st = k[h // g][ok], v[h // g][ok], steps[ok, h // g]
                x = kk @ q[b, h, t] * scale
                top = x.max()
                p = np.exp(x - top)
                z = p.sum()
                want, want_l, p = p @ vv / z, top + np.log(z), p / z
                ds = (c.Dh + 8) * 2.0 ** -23 * (np.abs(kk) @ np.abs(q[b, h, t])).max() * scale
                sums = (m / 16 + 64) * 2.0 ** -23
                tol = ((2.0 ** -11 + 2 * ds + 2.0 ** -20 + sums) * (p @ np.abs(vv))
                       + m * 2.0 ** -32 * 448 * (p * st).max() + half * np.abs(want))
                err = np.abs(o[b, h, t] - want)
                assert np.all(err <= tol), (b, t, h, float((err / tol).max()), int((err / tol).argmax()))
                assert abs(lse[b, h, t] - want_l) <= ds + 2.0 ** -20 + (m / 8 + 64) * 2.0 ** -24 + 2.0 ** -22 * abs(want_l)


def _attend(two, slots, n_new, q, scale, causal=True, seen=None, out_dtype=torch.float32, status=0):
    o, lse = two.ra.cache_attend(two.gpu, 0, _i32(slots), _i32(n_new), q.cuda(), scale=scale, causal=causal, out_dtype=out_dtype)
    assert two.ra.device_status() == status
    check_rows(two.cpu[0], slots, n_new, q, o, lse, scale, causal, seen)


# rows per key/value head: one to three column blocks of 8, many blocks of one token, and the kernel of many rows
FORMS = [(1, 2), (2, 6), (4, 5), (30, 2), (1, 40), (4, 40)]


@pytest.mark.parametrize("Dh,page", [(128, 16), (64, 32)])
@pytest.mark.parametrize("g,T", FORMS)
@pytest.mark.parametrize("far", [2.0 ** 12, 2.0 ** 30, 2.0 ** 90])
def test_a_later_page_of_large_values_is_not_seen_by_earlier_tokens(ra, Dh, page, g, T, far):  # noqa: F811
    """Values of the last pages are far larger: the queries before them, in the same tile and the same block
    of rows, keep theirs."""
    two = Both(ra, 40, 1, page, Dh, 1, 20)
    n = 7 * page + 9
    two.add([0], [n - T])
    k, v = _randn((1, 1, T, Dh), 1), _randn((1, 1, T, Dh), 2)
    v[:, :, T // 2:] = v[:, :, T // 2:] * far
    assert two.reserve([0], [T])
    two.append([0], [T], kv=(k, v))
    two.check()
    # the page that both kinds share holds the small ones as codes of the large scale: queries before it
    _attend(two, [0], [T], _randn((1, g, T, Dh), 3), Dh ** -0.5)
    new = Both(ra, 40, 1, page, Dh, 1, 20)
    k, v = _randn((1, 1, n, Dh), 4), _randn((1, 1, n, Dh), 5)
    cut = n // page * page
    v[:, :, cut:] = v[:, :, cut:] * far                      # a whole page of its own
    assert new.reserve([0], [n])
    new.append([0], [n], kv=(k, v))
    new.check()
    for m in sorted({T, min(T, n - cut + 3)}):
        _attend(new, [0], [m], _randn((1, g, m, Dh), 6), Dh ** -0.5)


@pytest.mark.parametrize("Dh,page", [(128, 16), (64, 64)])
@pytest.mark.parametrize("g,T", FORMS)
@pytest.mark.parametrize("low,far,gap", [(0, 24, 60), (0, 32, 50), (-50, 60, 100), (-100, 100, 190), (-110, 110, 230),
                                         (-100, 100, 210), (-20, 20, 0)])
def test_weight_on_pages_of_small_values(ra, Dh, page, g, T, low, far, gap):  # noqa: F811
    """Pages of values at 2^low and at 2^far in turn; scores give the large ones 2^-gap of the weight, so that
    either kind, or both, make the result."""
    two = Both(ra, 80, 1, page, Dh, 1, 30)
    n = 9 * page + 5
    k, v = 0.01 * _randn((1, 1, n, Dh), 1).float(), _randn((1, 1, n, Dh), 2).float()
    odd = (torch.arange(n) // page % 2).bool()
    v[:, :, odd] *= 2.0 ** far
    v[:, :, ~odd] *= 2.0 ** low
    k[..., 0] = 1.0
    k[:, :, odd, 0] = -1.0                                   # exact in 8 bits: scores +- gap / 2 in log2 units
    assert two.reserve([0], [n])
    two.append([0], [n], kv=(k.to(torch.bfloat16), v.to(torch.bfloat16)))
    two.check()
    q = 0.1 * _randn((1, g, T, Dh), 3).float()
    q[..., 0] = 1.0
    scale = max(gap, 1) / 2 * float(np.log(2.0))
    _attend(two, [0], [T], q.to(torch.bfloat16), scale)
    _attend(two, [0], [T], q.to(torch.bfloat16), scale, causal=False)


def test_many_parts_of_pages_far_apart(ra):  # noqa: F811
    """A context that every SM has a part of, scales changing all along it."""
    for g, T in ((2, 1), (2, 40)):
        two = Both(ra, 700, 1, 16, 128, 1, 650)
        n = 10000
        k, v = _randn((1, 1, n, 128), 1), _randn((1, 1, n, 128), 2)
        e = torch.randint(-40, 41, ((n + 15) // 16,), generator=torch.Generator().manual_seed(3)).repeat_interleave(16)[:n]
        v = v * torch.exp2(e.float()).view(1, 1, n, 1)
        k[..., 0] = -e.float() / 8                           # the larger the values, the smaller the weight
        assert two.reserve([0], [n])
        two.append([0], [n], kv=(k, v.to(torch.bfloat16)))
        q = 0.1 * _randn((1, g, T, 128), 4)
        q[..., 0] = 8.0
        _attend(two, [0], [T], q.to(torch.bfloat16), float(np.log(2.0)) * 0.9)


@pytest.mark.parametrize("g,T", FORMS)
@pytest.mark.parametrize("size", [3.3e38, 1e37, 1e-36])
def test_values_at_the_ends_of_the_range(ra, g, T, size):  # noqa: F811
    """Averages of values near the type's largest stay finite, of tiny ones keep their bits; in one part and in
    many."""
    for n in (T + 3, 3000):
        two = Both(ra, 200, 1, 16, 64, 1, 190)
        k, v = 0.05 * _randn((1, 1, n, 64), 1), torch.rand((1, 1, n, 64), generator=torch.Generator().manual_seed(2)) * 0.5 + 0.5
        v[..., 1::2] *= -1
        assert two.reserve([0], [n])
        two.append([0], [n], kv=(k.to(torch.bfloat16), (v * size).to(torch.bfloat16)))
        two.check()
        _attend(two, [0], [T], _randn((1, g, T, 64), 3), 0.125)
        _attend(two, [0], [T], _randn((1, g, T, 64), 3), 0.125, out_dtype=torch.bfloat16)


# ------------------------------------------------------------------------------------ pages out of range
@pytest.mark.parametrize("Dh,page", [(128, 16), (64, 32), (128, 128)])
@pytest.mark.parametrize("g,T", FORMS)
def test_tokens_on_a_bad_page_are_left_out(ra, Dh, page, g, T):  # noqa: F811
    """A table entry out of range is reported, and its tokens have no weight, whatever the others' scores."""
    two = Both(ra, 80, 1, page, Dh, 2, 30)
    n = [max(9 * page, T) + 5, 2 * page]
    k, v = _randn((2, 1, n[0], Dh), 1), _randn((2, 1, n[0], Dh), 2)
    k[..., 0] = 2.0
    assert two.reserve([0, 1], n)
    two.append([0, 1], n, kv=(k, v))
    seen = [np.ones(m, dtype=bool) for m in n]
    for j, bad in ((2, 87), (3, -3), (6, 80)):
        two.gpu.table[0, j] = bad
        seen[0][j * page:(j + 1) * page] = False
    for shift in (0.0, -2000.0):                             # scores around 0, and all far below it
        q = _randn((1, g, T, Dh), 3)
        q[..., 0] = shift
        for causal in (True, False):
            _attend(two, [0], [T], q, Dh ** -0.5, causal, seen, status=ra.RA_ERR_PAGES)
    # nothing left to see
    two.gpu.table[1, :] = 99
    m = min(T, n[1])
    q = _randn((1, g, m, Dh), 4)
    _attend(two, [1], [m], q, Dh ** -0.5, True, [np.zeros(n[1], dtype=bool)], status=ra.RA_ERR_PAGES)


def test_reading_a_bad_length_is_reported(ra):  # noqa: F811
    two = Both(ra, 8, 1, 16, 64, 2, 3)
    two.add([0], [20])
    for bad in (-1, 3 * 16 + 1, 2 ** 31 - 1):
        two.gpu.lens[1] = bad
        k, v = ra.cache_read(two.gpu, 0, _i32([1, 0]), 24)
        assert ra.device_status() == ra.RA_ERR_PAGES
        np.testing.assert_array_equal(k[1, :, :20].double().cpu().numpy(), two.cpu[0].values("k", 0))
        assert torch.all(v[1, :, 20:] == 0) and torch.all(k[0] == 0) and torch.all(v[0] == 0)
