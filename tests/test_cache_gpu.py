"""The paged 8-bit key/value cache against the float64 oracle (oracle/cache.py).

Page tables, lengths, counts, codes and scales are compared exactly.  Tolerance of the attention,
from the arithmetic (u = 2^-24):
  scores      products are exact, the sum of Dh of them and the scaling are float32:
              ds = (Dh + 8) 2 u scale sum_i |q_i k_i|, and a relative 2^-21 of exp;
  P           rounded to fp16: half a step, 2^-11 of each term, or 2^-32 of the largest where the
              term is below fp16's normal range (its unit is 2^7, the reference at most 2^8 below);
  sums        float32 in tiles of 16 tokens, then over warps, blocks: (n / 16 + 64) 2 u;
  o           (2^-11 + 2 max ds + 2^-20 + sums) sum_j p_j |v_j| + n 2^-31 max |v|, then half a step of the
              output type: 2^-8 |o| in bf16;
  lse         max ds + 2^-20 + (n / 8 + 64) u + 2^-22 |lse|."""
import numpy as np
import pytest
import torch

import oracle
from oracle import cache as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    from long_context_exact_fwd_b200 import build
    build.ensure_built()
    from long_context_exact_fwd_b200 import ring_attn
    return ring_attn


def _i32(x):
    return torch.tensor(list(x), dtype=torch.int32, device="cuda")


def _randn(shape, seed, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (scale * torch.randn(shape, generator=g)).to(torch.bfloat16)


class Both:
    """The cache on the GPU and the oracle's, given the same calls."""

    def __init__(self, ra, pages, heads, page, Dh, slots, max_pages, layers=1):
        self.ra, self.layers, self.page = ra, layers, page
        self.gpu = ra.kv_cache(layers, pages, heads, page, Dh, slots, max_pages)
        self.cpu = [oc.Cache(pages, heads, page, Dh, slots, max_pages) for _ in range(layers)]
        self.seed = 100

    def reserve(self, slots, n):
        self.ra.cache_reserve(self.gpu, _i32(slots), _i32(n))
        return [c.reserve(slots, n) for c in self.cpu][0]

    def append(self, slots, n, scale=1.0, kv=None):
        T = max(max(n), 1)
        for l in range(self.layers):
            self.seed += 1
            k, v = kv or (_randn((len(slots), self.cpu[0].heads, T, self.cpu[0].Dh), 2 * self.seed + i, scale) for i in (0, 1))
            self.ra.cache_append(self.gpu, l, _i32(slots), _i32(n), k.cuda(), v.cuda())
            self.cpu[l].append(slots, n, k.float().numpy(), v.float().numpy())

    def add(self, slots, n, scale=1.0):
        assert self.reserve(slots, n)
        self.append(slots, n, scale)

    def fork(self, src, dst):
        self.ra.cache_fork(self.gpu, _i32(src), _i32(dst))
        [c.fork(src, dst) for c in self.cpu]

    def trim(self, slots, keep):
        self.ra.cache_trim(self.gpu, _i32(slots), _i32(keep))
        [c.trim(slots, keep) for c in self.cpu]

    def compact(self):
        self.ra.cache_compact(self.gpu)
        [c.compact() for c in self.cpu]

    def check(self, status=0):
        assert self.ra.device_status() == status
        c = self.cpu[0]
        assert np.array_equal(self.gpu.table.cpu().numpy(), c.table)
        assert np.array_equal(self.gpu.lens.cpu().numpy(), c.lens)
        assert np.array_equal(self.gpu.refs.cpu().numpy(), c.refs)
        for l, c in enumerate(self.cpu):
            for name, codes, scale in (("k", self.gpu.k, self.gpu.k_scale), ("v", self.gpu.v, self.gpu.v_scale)):
                codes = codes[l].view(torch.float8_e4m3fn).double().cpu().numpy()
                scale = scale[l].double().cpu().numpy()
                for s in np.flatnonzero(c.lens):
                    for j in range(c._count(c.lens[s])):
                        p, m = c.table[s, j], min(self.page, c.lens[s] - j * self.page)
                        np.testing.assert_array_equal(codes[p][:, :m], c.codes[name][p][:, :m])
                        np.testing.assert_array_equal(scale[p], np.ldexp(1.0, c.exp[name][p]))

    def attend(self, slots, n_new, Hq, T, layer=0, scale=None, causal=True, q_scale=1.0, seed=7, out_dtype=torch.bfloat16):
        c = self.cpu[layer]
        q = _randn((len(slots), Hq, T, c.Dh), seed, q_scale)
        o = torch.full((len(slots), Hq, T, c.Dh), 7.0, dtype=out_dtype, device="cuda")
        lse = torch.full((len(slots), Hq, T), 7.0, device="cuda")
        self.ra.cache_attend(self.gpu, layer, _i32(slots), _i32(n_new), q.cuda(), scale=scale, causal=causal, out=o, lse=lse,
                             out_dtype=out_dtype)
        assert self.ra.device_status() == 0
        check_attend(c, slots, n_new, q, o, lse, scale, causal)
        return q, o, lse


def check_attend(c, slots, n_new, q, o, lse, scale=None, causal=True):
    half = 2.0 ** -8 if o.dtype == torch.bfloat16 else 2.0 ** -24
    o, lse, qd = o.double().cpu().numpy(), lse.double().cpu().numpy(), q.double().cpu().numpy()
    for b, (s, n) in enumerate(zip(slots, n_new)):
        n_here = n if s >= 0 else 0
        assert np.all(o[b, :, n_here:] == 7.0) and np.all(lse[b, :, n_here:] == 7.0)     # rows of padding
        if not n_here:
            continue
        want, want_l, size = c.attend(s, qd[b, :, :n], n, scale, causal)
        k, v = np.abs(c.values("k", s)), np.abs(c.values("v", s))
        m, g = k.shape[1], qd.shape[1] // c.heads
        if m == 0:
            assert np.all(o[b, :, :n] == 0) and np.all(lse[b, :, :n] == -np.inf)
            continue
        sizes = np.stack([np.abs(qd[b, h, :n]) @ k[h // g].T for h in range(qd.shape[1])]) * (scale or c.Dh ** -0.5)
        ds = (c.Dh + 8) * 2.0 ** -23 * sizes.max(-1)                                     # [Hq, n]
        sums = (m / 16 + 64) * 2.0 ** -23
        tol = (2.0 ** -11 + 2 * ds[..., None] + 2.0 ** -20 + sums) * size + m * 2.0 ** -31 * v.max() + half * np.abs(want)
        err = np.abs(o[b, :, :n] - want)
        assert np.all(err <= tol), (b, float((err / tol).max()))
        fin = np.isfinite(want_l)
        assert np.array_equal(np.isneginf(lse[b, :, :n]), ~fin)
        ltol = ds + 2.0 ** -20 + (m / 8 + 64) * 2.0 ** -24 + 2.0 ** -22 * np.abs(want_l)
        assert np.all(np.abs(lse[b, :, :n] - want_l)[fin] <= ltol[fin])


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("Dh", [64, 128])
def test_appending_reading_and_attending_step_by_step(ra, page, Dh):
    """A prompt that ends inside a page, then single tokens whose size grows (scales grow, older codes are
    restated), several tokens at once, ragged; everything compared after each step."""
    two = Both(ra, pages=40, heads=2, page=page, Dh=Dh, slots=5, max_pages=20, layers=2)
    slots = [3, 0, 4]
    for step, (n, size) in enumerate([([37, 1, 130], 1.0), ([1, 1, 1], 0.1), ([1, 1, 1], 30.0), ([5, 0, 17], 3.0),
                                      ([1, 60, 2], 1000.0)]):
        two.add(slots, n, size)
        two.check()
        two.attend(slots, n, Hq=6, T=max(n) + step % 2, layer=step % 2, q_scale=0.05 if size > 2 else 1.0, seed=step)
    length = int(two.cpu[0].lens.max()) + 3
    for start in ([0, 0, 0], [5, -2, 100]):
        k, v = ra.cache_read(two.gpu, 1, _i32(slots), length, start=_i32(start))
        assert ra.device_status() == 0
        for b, s in enumerate(slots):
            for name, x in (("k", k), ("v", v)):
                want = np.zeros((2, length, Dh))
                have = two.cpu[1].values(name, s)
                for t in range(length):
                    if 0 <= start[b] + t < have.shape[1]:
                        want[:, t] = have[:, start[b] + t]
                np.testing.assert_array_equal(x[b].double().cpu().numpy(), want)


# (heads, Hq, T, Dh, page, lengths): lengths around tiles of 32 and stretches of blocks, one to three
# column blocks of rows and more, many sequences, one long one
ATTEND = [(1, 1, 1, 128, 16, [1]), (2, 4, 1, 128, 64, [0 + 31, 32, 33, 255, 256, 257]), (1, 8, 1, 64, 16, [1000, 2, 17]),
          (2, 2, 3, 128, 32, [3, 5, 100]), (2, 16, 1, 64, 128, [129, 700]), (1, 6, 5, 128, 64, [400, 5]),
          (4, 4, 13, 64, 16, [64, 13, 333]), (2, 10, 7, 128, 64, [150, 49]), (1, 3, 100, 128, 64, [260]),
          (8, 8, 1, 128, 64, list(range(1, 40, 3))), (1, 4, 1, 128, 128, [20000]), (1, 2, 70, 64, 32, [70, 71, 500])]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,Hq,T,Dh,page,lengths", ATTEND)
def test_attention_matches_oracle(ra, heads, Hq, T, Dh, page, lengths, causal):
    need = [-(-n // page) for n in lengths]
    two = Both(ra, sum(need) + 2, heads, page, Dh, len(lengths), max(need) + 1)
    slots = list(np.random.default_rng(1).permutation(len(lengths)))
    two.add(slots, lengths)
    n_new = [min(T, n) for n in lengths]
    two.attend(slots, n_new, Hq, T, causal=causal, q_scale=2.0)
    two.attend(slots, n_new, Hq, T, causal=causal, scale=0.3, seed=8, out_dtype=torch.float32)


def test_sharp_flat_and_tiny_scores(ra):
    """One key far above the others; all keys alike; keys and values at the ends of bf16's range, pages
    of zeros between pages of large values."""
    two = Both(ra, 100, 1, 16, 128, 4, 70)
    lengths = [1000, 300, 100, 64]
    assert two.reserve([0, 1, 2, 3], lengths)
    k, v = _randn((4, 1, 1000, 128), 1), _randn((4, 1, 1000, 128), 2)
    k[0, 0, 500] = 8.0
    k[1] = k[1, :, :1]
    k[2] *= 1e-30
    v[2, :, 16:48] = 0
    v[3, :, 16:32] *= 1e4
    v[3, :, 32:48] *= 1e-4
    two.append([0, 1, 2, 3], lengths, kv=(k, v))
    two.check()
    two.attend([0, 1, 2, 3], [1, 1, 1, 1], 4, 1)
    two.attend([0, 1, 2, 3], [2, 2, 2, 2], 4, 2, scale=4.0)
    two.attend([3, 2], [1, 1], 2, 1, q_scale=1e-20)
    big = Both(ra, 4, 1, 16, 64, 1, 4)
    assert big.reserve([0], [20])
    x = _randn((1, 1, 20, 64), 3)
    x[0, 0, 3] = 3.3e38
    x[0, 0, 18] = torch.finfo(torch.bfloat16).max
    big.append([0], [20], kv=(x, x))
    big.check()


def test_values_that_are_not_finite(ra):
    """Stored as NaN; they reach the queries that see them and no others, whatever lies behind a
    sequence's end."""
    two = Both(ra, 12, 1, 32, 64, 2, 5)
    two.gpu.k.fill_(0x7f)
    two.gpu.v.fill_(0x7f)                                   # what the pages held before
    assert two.reserve([0, 1], [70, 70])
    k, v = _randn((2, 1, 70, 64), 1), _randn((2, 1, 70, 64), 2)
    v[0, 0, 67, 5], v[0, 0, 66, 9], k[1, 0, 68, 3] = float("nan"), float("-inf"), float("inf")
    two.append([0, 1], [70, 70], kv=(k, v))
    two.check()
    q = _randn((2, 2, 6, 64), 3)
    for n in (6, 3):
        o, lse = ra.cache_attend(two.gpu, 0, _i32([0, 1]), _i32([n, n]), q[:, :, :n].contiguous().cuda())
        assert ra.device_status() == 0
        for t in range(n):
            pos = 70 - n + t
            bad = torch.isnan(o[0, :, t]).cpu()
            want = torch.zeros_like(bad)
            want[:, 5], want[:, 9] = pos >= 67, pos >= 66
            assert torch.equal(bad, want), (n, t)
            assert torch.isfinite(lse[0, :, t]).all()
            assert torch.isnan(o[1, :, t]).all() == (pos >= 68) and torch.isnan(lse[1, :, t]).all() == (pos >= 68)
            if pos < 68:
                assert torch.isfinite(o[1, :, t]).all()


def test_empty_sequences_and_padding(ra):
    two = Both(ra, 8, 2, 16, 64, 4, 4)
    two.add([2], [20])
    # slot 1 holds nothing but is asked; -1 is padding; n_new 0 writes nothing
    q, o, lse = two.attend([1, -1, 2, 2], [1, 1, 0, 1], Hq=2, T=2, causal=False)
    assert torch.all(o[0, :, 0] == 0) and torch.all(torch.isneginf(lse[0, :, 0]))


def test_one_token_calls_agree_with_one_call_for_all(ra):
    """Causal attention of 9 tokens at once = each alone at its own length (bit for bit is not asked: the
    work is cut elsewhere)."""
    two = Both(ra, 20, 2, 16, 128, 2, 10)
    two.add([0], [100])
    q = _randn((1, 8, 9, 128), 5).cuda()
    o, lse = ra.cache_attend(two.gpu, 0, _i32([0]), None, q)
    for t in range(9):
        two.gpu.lens.fill_(92 + t)
        a, l = ra.cache_attend(two.gpu, 0, _i32([0]), None, q[:, :, t:t + 1])
        assert (a.float() - o[:, :, t:t + 1].float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
        assert (l - lse[:, :, t:t + 1]).abs().max() <= 1e-5
    assert ra.device_status() == 0


def test_results_do_not_change_from_run_to_run(ra):
    two = Both(ra, 700, 2, 16, 128, 3, 400)
    two.add([0, 1, 2], [5000, 333, 1777])
    q = _randn((3, 8, 2, 128), 5).cuda()
    first = [x.clone() for x in ra.cache_attend(two.gpu, 0, _i32([0, 1, 2]), None, q)]
    for _ in range(10):
        for a, b in zip(first, ra.cache_attend(two.gpu, 0, _i32([0, 1, 2]), None, q)):
            assert torch.equal(a, b)


def test_pages_through_forks_trims_and_compactions(ra):
    """A random walk of page operations with appends, every state compared."""
    rng = np.random.default_rng(3)
    two = Both(ra, pages=60, heads=2, page=16, Dh=64, slots=8, max_pages=12, layers=2)
    two.add([0, 1], [50, 16])
    for step in range(40):
        live = [s for s in range(8) if two.cpu[0].lens[s]]
        empty = [s for s in range(8) if not two.cpu[0].lens[s]]
        what = rng.choice(["add", "fork", "trim", "compact", "free"])
        if what == "add":
            slots = [int(s) for s in rng.permutation(8)[: rng.integers(1, 6)]]
            n = [int(min(rng.integers(0, 20), 12 * 16 - two.cpu[0].lens[s])) for s in slots]
            if two.reserve(slots, n):
                two.append(slots, n)
            else:
                assert ra.device_status() == ra.RA_ERR_PAGES
        elif what == "fork" and live and empty:
            dst = [int(s) for s in rng.permutation(empty)[: rng.integers(1, len(empty) + 1)]]
            two.fork([int(rng.choice(live)) for _ in dst], dst)
        elif what == "trim" and live:
            slots = [int(s) for s in rng.permutation(live)[: rng.integers(1, len(live) + 1)]]
            two.trim(slots, [int(rng.integers(0, two.cpu[0].lens[s] + 3)) for s in slots])
        elif what == "free" and len(live) > 3:
            two.trim([live[0], -1], [0, 5])
        elif what == "compact":
            two.compact()
        two.check()
    live = [s for s in range(8) if two.cpu[0].lens[s]]
    two.attend(live, [1] * len(live), 4, 1, layer=1)


def test_a_fork_does_not_see_what_the_other_appends(ra):
    two = Both(ra, 30, 2, 32, 128, 4, 6, layers=3)
    two.add([1], [75])
    two.fork([1, 1, -1], [0, 3, -1])
    two.check()
    two.add([0, 1, 3], [1, 1, 1])                            # three holders of one page: two copies
    two.check()
    two.add([3, 0], [40, 2], scale=50.0)
    two.check()
    two.attend([0, 1, 3], [1, 1, 1], 4, 1, layer=2, q_scale=0.05)
    two.trim([1], [0])
    two.compact()
    two.check()
    two.attend([0, 3], [3, 3], 2, 3, layer=1, q_scale=0.05)


def test_pool_of_many_pages(ra):
    """More pages than one sweep of the planning block looks at, holes everywhere."""
    two = Both(ra, pages=40000, heads=1, page=16, Dh=64, slots=3, max_pages=30000)
    n_pages = [9000, 12000]
    for s, n in enumerate(n_pages):
        ra.cache_reserve(two.gpu, _i32([s]), _i32([16 * n]))
        two.cpu[0].reserve([s], [16 * n])
    two.trim([0], [16 * 100])
    ra.cache_compact(two.gpu)
    two.cpu[0].compact()
    assert ra.device_status() == 0
    for got, want in ((two.gpu.table, two.cpu[0].table), (two.gpu.refs, two.cpu[0].refs), (two.gpu.lens, two.cpu[0].lens)):
        assert np.array_equal(got.cpu().numpy(), want)


def test_bad_entries_are_left_out_and_reported(ra):
    two = Both(ra, 6, 1, 16, 64, 3, 4)
    two.add([0], [10])
    two.fork([0], [1])
    two.check()

    def reported(call):
        call()
        assert ra.device_status() == ra.RA_ERR_PAGES
        two.check()

    x = _randn((1, 1, 1, 64), 1).cuda()
    x2 = x.expand(2, 1, 1, 64).contiguous()
    reported(lambda: ra.cache_reserve(two.gpu, _i32([3]), _i32([1])))
    reported(lambda: ra.cache_reserve(two.gpu, _i32([-2]), _i32([1])))
    reported(lambda: ra.cache_reserve(two.gpu, _i32([2]), _i32([16 * 4 + 1])))       # beyond max_pages
    reported(lambda: ra.cache_reserve(two.gpu, _i32([0]), _i32([-1])))
    reported(lambda: ra.cache_reserve(two.gpu, _i32([2, 0]), _i32([64, 32])))        # too few pages: all or nothing
    reported(lambda: ra.cache_append(two.gpu, 0, _i32([0]), None, x, x))             # the page has two holders
    reported(lambda: ra.cache_append(two.gpu, 0, _i32([2]), None, x, x))             # nothing was reserved
    reported(lambda: ra.cache_append(two.gpu, 0, _i32([7]), None, x, x))
    reported(lambda: ra.cache_append(two.gpu, 0, _i32([0]), _i32([2]), x, x))        # n_new beyond T
    reported(lambda: ra.cache_fork(two.gpu, _i32([0]), _i32([1])))                   # not empty
    reported(lambda: ra.cache_fork(two.gpu, _i32([0]), _i32([0])))
    reported(lambda: ra.cache_fork(two.gpu, _i32([0]), _i32([5])))
    reported(lambda: ra.cache_trim(two.gpu, _i32([9]), _i32([0])))
    reported(lambda: ra.cache_trim(two.gpu, _i32([0]), _i32([-1])))
    reported(lambda: ra.cache_attend(two.gpu, 0, _i32([4]), None, x))
    reported(lambda: ra.cache_read(two.gpu, 0, _i32([4]), 5))
    # the same slot twice: the first entry counts
    ra.cache_reserve(two.gpu, _i32([2, 2]), _i32([3, 4]))
    two.cpu[0].reserve([2], [3])
    assert ra.device_status() == ra.RA_ERR_PAGES
    ra.cache_append(two.gpu, 0, _i32([2, 2]), None, x2, x2)
    assert ra.device_status() == ra.RA_ERR_PAGES
    ra.cache_trim(two.gpu, _i32([2, 2]), _i32([0, 1]))
    two.cpu[0].trim([2], [0])
    assert ra.device_status() == ra.RA_ERR_PAGES
    two.check()
    ra.cache_fork(two.gpu, _i32([0, 1]), _i32([2, 2]))
    two.cpu[0].fork([0], [2])
    assert ra.device_status() == ra.RA_ERR_PAGES
    two.check()
    # a page number out of range in the table
    two.gpu.table[2, 0] = 77
    ra.cache_attend(two.gpu, 0, _i32([2]), None, x)
    assert ra.device_status() == ra.RA_ERR_PAGES
    ra.cache_append(two.gpu, 0, _i32([2]), None, x, x)
    assert ra.device_status() == ra.RA_ERR_PAGES
    ra.cache_read(two.gpu, 0, _i32([2]), 5)
    assert ra.device_status() == ra.RA_ERR_PAGES


def test_a_serving_loop_in_a_graph(ra):
    """Rotate, reserve, append, attend captured once and replayed token by token, with a row of padding,
    against the oracle; and two graphs of the same calls used in turn."""
    B, H, Hk, Dh, page = 3, 4, 2, 128, 16
    two = Both(ra, 40, Hk, page, Dh, 4, 12)
    two.add([0, 2], [30, 7])
    w, _ = ra.rope_inv_freq(Dh)
    plan = ra.rope_plan(w)
    slots, n = _i32([2, -1, 0]), _i32([1, 1, 1])
    rows = torch.zeros((B, 1, H + 2 * Hk, Dh), dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros((B, 1), dtype=torch.int64, device="cuda")
    o = torch.full((B, H, 1, Dh), 7.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, H, 1), 7.0, device="cuda")
    q, k, v = (rows[:, :, a:b].permute(0, 2, 1, 3) for a, b in ((0, H), (H, H + Hk), (H + Hk, H + 2 * Hk)))

    def step():
        qr, kr = ra.rope(q, plan, k=k, pos=pos)
        ra.cache_reserve(two.gpu, slots, n)
        ra.cache_append(two.gpu, 0, slots, n, kr, v)
        ra.cache_attend(two.gpu, 0, slots, n, qr, out=o, lse=lse)

    saved = [t.clone() for t in (two.gpu.table, two.gpu.lens, two.gpu.refs)]
    step()                                                   # warm up, then undone
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
    for t, s in zip((two.gpu.table, two.gpu.lens, two.gpu.refs), saved):
        t.copy_(s)
    c = two.cpu[0]
    for i in range(20):
        rows.copy_(_randn(rows.shape, 50 + i))
        at = [c.lens[2], 0, c.lens[0]]
        pos.copy_(torch.tensor(at).view(B, 1))
        graphs[i % 2].replay()
        assert ra.device_status() == 0
        kr = ra.rope(k, plan, pos=pos).float().cpu().numpy()
        qr = ra.rope(q, plan, pos=pos)
        assert c.reserve([2, -1, 0], [1, 1, 1])
        c.append([2, -1, 0], [1, 1, 1], kr, v.float().cpu().numpy())
        two.check()
        check_attend(c, [2, -1, 0], [1, 1, 1], qr, o, lse)


def test_parts_of_a_context_merge(ra):
    """Float32 outputs over two caches are parts for merge(): the whole context in one cache."""
    whole, a, z = (Both(ra, 20, 2, 16, 64, 1, 10) for _ in range(3))
    k, v = _randn((1, 2, 112, 64), 1), _randn((1, 2, 112, 64), 2)
    for two, lo, hi in ((whole, 0, 112), (a, 0, 64), (z, 64, 112)):
        assert two.reserve([0], [hi - lo])
        two.append([0], [hi - lo], kv=(k[:, :, lo:hi].contiguous(), v[:, :, lo:hi].contiguous()))
    q = _randn((1, 4, 1, 64), 3)
    parts = [ra.cache_attend(t.gpu, 0, _i32([0]), None, q.cuda(), causal=False, out_dtype=torch.float32) for t in (a, z)]
    o, lse = ra.merge(torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts]))
    assert ra.device_status() == 0
    check_attend(whole.cpu[0], [0], [1], q, o, lse)
    # and of a prompt, its attention on the cached values is the dense forward on what cache_read gives
    kd, vd = ra.cache_read(whole.gpu, 0, _i32([0]), 112)
    q = _randn((1, 2, 112, 64), 4).cuda()
    dense, dense_lse = ra.fwd(q, kd, vd, 1, True)
    o, lse = ra.cache_attend(whole.gpu, 0, _i32([0]), None, q)
    ref, _ = oracle.attn_fwd_heads(q.cpu(), kd.cpu(), vd.cpu(), True)
    for x in (o, dense):
        assert np.abs(x.double().cpu().numpy() - np.asarray(ref)).max() <= 2e-2
    assert (lse - dense_lse).abs().max() <= 1e-3


def test_another_stream_and_strided_inputs(ra):
    two = Both(ra, 20, 2, 32, 128, 2, 8)
    two.add([0, 1], [100, 40])
    rows = _randn((2, 3, 8, 128), 1).cuda()                  # [B, T, heads, Dh]
    q = rows.permute(0, 2, 1, 3)
    want = ra.cache_attend(two.gpu, 0, _i32([0, 1]), None, q.contiguous())
    side = torch.cuda.Stream()
    slots = _i32([0, 1])
    side.wait_stream(torch.cuda.current_stream())
    got = [ra.cache_attend(two.gpu, 0, slots, None, q, stream=side) for _ in range(3)]
    torch.cuda.current_stream().wait_stream(side)
    for o, lse in got:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])


def test_refusals(ra):
    two = Both(ra, 4, 2, 16, 64, 2, 4)
    c, s = two.gpu, _i32([0])
    x = _randn((1, 2, 1, 64), 1).cuda()
    with pytest.raises(ValueError):
        ra.kv_cache(1, 4, 2, 24, 64, 2, 4)
    with pytest.raises(ValueError):
        ra.kv_cache(1, 4, 2, 16, 96, 2, 4)
    with pytest.raises(ValueError):
        ra.KVCache(c.k, c.v, c.k_scale, c.v_scale, c.table, c.lens, c.refs.long())
    with pytest.raises(ValueError):
        ra.KVCache(c.k, c.v[:, :3], c.k_scale, c.v_scale, c.table, c.lens, c.refs)
    for bad in (s.long(), s.cpu(), _i32([0, 1])):
        with pytest.raises(ValueError):
            ra.cache_append(c, 0, bad, None, x, x)
        with pytest.raises(ValueError):
            ra.cache_attend(c, 0, bad, None, x)
    with pytest.raises(ValueError):
        ra.cache_append(c, 0, s, None, x.float(), x)
    with pytest.raises(ValueError):
        ra.cache_append(c, 0, s, None, x[:, :1], x[:, :1])
    with pytest.raises(ValueError):
        ra.cache_attend(c, 0, s, None, _randn((1, 3, 1, 64), 2).cuda())
    with pytest.raises(ValueError):
        ra.cache_attend(c, 0, s, None, x, out_dtype=torch.float16)
    with pytest.raises(ra.RingAttnError):
        ra.cache_append(c, 1, s, None, x, x)
    with pytest.raises(ra.RingAttnError):
        ra.cache_attend(c, 0, s, None, x, workspace=torch.empty(64, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ra.RingAttnError):
        ra.cache_attend(c, 0, s, None, _randn((1, 2, 1, 68), 3).cuda()[..., 4:])     # rows off 16 bytes
    assert ra.device_status() == 0


@pytest.mark.parametrize("Hq,Dh", [(24, 128), (31, 64), (256, 128), (300, 64)])
def test_a_value_that_no_row_of_a_block_sees(ra, Hq, Dh):
    """So many query heads on one key/value head that a block of rows holds one token only: a NaN behind that
    token, in the same tile, does not reach it."""
    two = Both(ra, 8, 1, 32, Dh, 1, 4)
    n = 100
    assert two.reserve([0], [n])
    k, v = _randn((1, 1, n, Dh), 1), _randn((1, 1, n, Dh), 2)
    v[0, 0, n - 1, 7] = float("nan")
    two.append([0], [n], kv=(k, v))
    q = _randn((1, Hq, 2, Dh), 3).cuda()
    o, lse = ra.cache_attend(two.gpu, 0, _i32([0]), None, q)
    bad = torch.isnan(o[0]).cpu()
    want = torch.zeros((Hq, 2, Dh), dtype=torch.bool)
    want[:, 1, 7] = True
    assert torch.equal(bad, want) and torch.isfinite(lse).all() and ra.device_status() == 0


@pytest.mark.parametrize("T,captured", [(1, False), (1, True), (40, False), (40, True)])
def test_launches_set_up_early_wait_for_both_streams(ra, T, captured):
    """Inputs that another stream writes late, behind an event, between calls whose launches are set up behind
    one another."""
    H, Dh, n = 2, 128, 300
    k, v, q = _randn((1, H, n, Dh), 1).cuda(), _randn((1, H, n, Dh), 2).cuda(), _randn((1, 4, T, Dh), 3).cuda()
    k2, v2 = _randn((1, H, T, Dh), 4).cuda(), _randn((1, H, T, Dh), 5).cuda()
    slots, first, more = _i32([0]), _i32([n]), _i32([T])
    busy = torch.randn((4096, 4096), device="cuda")
    side, at = torch.cuda.Stream(), {}

    def run(cache, kk, vv, qq, late):
        ra.cache_reserve(cache, slots, first)
        ra.cache_append(cache, 0, slots, None, k, v)
        ra.cache_reserve(cache, slots, more)
        if late:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(4):
                    at["busy"] = busy @ busy
                kk.copy_(k2)
                vv.copy_(v2)
            torch.cuda.current_stream().wait_stream(side)
        ra.cache_append(cache, 0, slots, None, kk, vv)
        if late:
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(side):
                for _ in range(4):
                    at["busy"] = busy @ busy
                qq.copy_(q)
            torch.cuda.current_stream().wait_stream(side)
        return ra.cache_attend(cache, 0, slots, None, qq)

    new = lambda: ra.kv_cache(1, 16, H, 32, Dh, 1, 16)  # noqa: E731
    want = run(new(), k2, v2, q, False)
    cache, late = new(), [torch.zeros_like(x) for x in (k2, v2, q)]
    if captured:
        busy @ busy
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = run(cache, *late, True)
        g.replay()
    else:
        got = run(cache, *late, True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and ra.device_status() == 0


def test_many_calls_back_to_back(ra):
    """A hundred rounds of all calls without a pause give what the same rounds with pauses give."""
    B, H, Dh, page = 6, 2, 64, 16
    xs = [_randn((B, H, 7, Dh), 10 + i).cuda() for i in range(5)]
    qs = [_randn((B, 4, 7, Dh), 20 + i).cuda() for i in range(5)]
    slots, a, b = _i32([0, 1, 2, 3, 4, 5]), _i32([0, 1, 2]), _i32([3, 4, 5])
    counts = [_i32([(3 * i + j) % 7 + 1 for j in range(B)]) for i in range(5)]
    keep = _i32([20, 33, 47])

    def rounds(pause):
        cache, outs = ra.kv_cache(1, 400, H, page, Dh, B, 64), []
        for i in range(100):
            n = counts[i % 5]
            ra.cache_reserve(cache, slots, n)
            ra.cache_append(cache, 0, slots, n, xs[i % 5], xs[(i + 1) % 5])
            o = torch.zeros_like(qs[0])
            lse = torch.zeros(qs[0].shape[:3], device="cuda")
            outs.append(ra.cache_attend(cache, 0, slots, n, qs[i % 5], out=o, lse=lse)[0])
            if i % 10 == 9:
                ra.cache_trim(cache, a, keep)
                ra.cache_free(cache, b)
                ra.cache_fork(cache, a, b)
                ra.cache_compact(cache)
            if pause:
                torch.cuda.synchronize()
        return torch.stack(outs), cache

    (o1, c1), (o2, c2) = rounds(True), rounds(False)
    assert ra.device_status() == 0
    assert torch.equal(o1, o2)
    for name in ("table", "lens", "refs"):
        assert torch.equal(getattr(c1, name), getattr(c2, name))
    assert torch.equal(ra.cache_read(c1, 0, slots, 100)[0], ra.cache_read(c2, 0, slots, 100)[0])
