"""Calls on the cache that its documentation allows: rows of padding in fresh outputs, errors of several kinds, a
reserve that failed inside a captured step, and batches of hundreds of sequences."""
import numpy as np
import pytest
import torch

from test_cache_gpu import Both, _i32, _randn, check_attend, ra  # noqa: F401

pytestmark = pytest.mark.gpu


def _poison(*shapes_dtypes):
    """Freed memory of these sizes holds NaN."""
    for _ in range(4):
        xs = [torch.full(s, float("nan"), dtype=d, device="cuda") for s, d in shapes_dtypes for _ in range(2)]
        del xs


# ------------------------------------------------------------------------------------ rows of padding
@pytest.mark.parametrize("g,T", [(1, 2), (3, 5), (4, 40)])
def test_fresh_outputs_hold_nothing_in_rows_of_padding(ra, g, T):  # noqa: F811
    two = Both(ra, 40, 2, 16, 64, 4, 10)
    two.add([0, 2], [100, 50])
    slots, n = [2, -1, 0, 3, 0], [1, T, T, 0, 0]
    q = _randn((5, 2 * g, T, 64), 3)
    for dt in (torch.bfloat16, torch.float32):
        _poison((q.shape, dt), (q.shape[:3], torch.float32))
        o, lse = ra.cache_attend(two.gpu, 0, _i32(slots), _i32(n), q.cuda(), out_dtype=dt)
        assert ra.device_status() == 0
        for b, m in enumerate([1, 0, T, 0, 0]):
            assert torch.all(o[b, :, m:] == 0) and torch.all(torch.isneginf(lse[b, :, m:])), b
            o[b, :, m:], lse[b, :, m:] = 7.0, 7.0
        check_attend(two.cpu[0], slots, n, q, o, lse)
        # a given output keeps its rows, the fresh one beside it is filled
        given = torch.full(q.shape, 7.0, dtype=dt, device="cuda")
        _poison((q.shape[:3], torch.float32))
        _, lse = ra.cache_attend(two.gpu, 0, _i32(slots), _i32(n), q.cuda(), out_dtype=dt, out=given)
        assert torch.all(given[1] == 7.0) and torch.all(given[0, :, 1:] == 7.0) and torch.all(torch.isneginf(lse[1]))
    # entries out of range, too
    _poison((q.shape, torch.bfloat16), (q.shape[:3], torch.float32))
    o, lse = ra.cache_attend(two.gpu, 0, _i32([9, 0, 0, 0, 0]), _i32([1, T + 1, T, 0, -1]), q.cuda())
    assert ra.device_status() == ra.RA_ERR_PAGES
    for b in (0, 1, 3, 4):
        assert torch.all(o[b] == 0) and torch.all(torch.isneginf(lse[b]))
    # and the same through a graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    s, m = _i32(slots), _i32(n)
    qc = q.cuda()
    with torch.cuda.graph(graph):
        o, lse = ra.cache_attend(two.gpu, 0, s, m, qc)
    o.fill_(float("nan")), lse.fill_(float("nan"))
    graph.replay()
    assert torch.all(o[1] == 0) and torch.all(torch.isneginf(lse[1])) and ra.device_status() == 0


def test_fresh_reads_hold_zero_in_rows_of_padding(ra):  # noqa: F811
    two = Both(ra, 40, 2, 16, 64, 4, 10)
    two.add([0, 2], [100, 50])
    shape = (4, 2, 60, 64)
    _poison((shape, torch.bfloat16), (shape, torch.bfloat16))
    k, v = ra.cache_read(two.gpu, 0, _i32([-1, 2, 3, -1]), 60)
    assert ra.device_status() == 0
    for x in (k, v):
        assert torch.all(x[0] == 0) and torch.all(x[2:] == 0) and torch.all(x[1, :, 50:] == 0)
    np.testing.assert_array_equal(k[1, :, :50].double().cpu().numpy(), two.cpu[0].values("k", 2))
    given = torch.full(shape, 7.0, dtype=torch.bfloat16, device="cuda")
    _poison((shape, torch.bfloat16))
    _, v = ra.cache_read(two.gpu, 0, _i32([-1, 2, 9, -1]), 60, k=given)
    assert ra.device_status() == ra.RA_ERR_PAGES
    assert torch.all(given[0] == 7.0) and torch.all(given[2:] == 7.0) and torch.all(v[0] == 0) and torch.all(v[2:] == 0)


# ------------------------------------------------------------------------------------ two kinds of error
@pytest.mark.parametrize("cache_first", [True, False])
def test_an_entry_out_of_range_does_not_hide_a_timeout(ra, cache_first):  # noqa: F811
    two = Both(ra, 8, 1, 16, 64, 2, 3)

    def bad_slot():
        ra.cache_trim(two.gpu, _i32([9]))

    for call in ([bad_slot, lambda: ra.wait_selftest(0.02)] if cache_first else [lambda: ra.wait_selftest(0.02), bad_slot]):
        call()
    assert ra.device_status() == ra.RA_ERR_TIMEOUT
    assert ra.device_status() == ra.RA_ERR_PAGES
    assert ra.device_status() == 0


def test_a_ring_does_not_raise_for_a_cache_entry(ra):  # noqa: F811
    from long_context_exact_fwd_b200 import ring_dist as rd
    two = Both(ra, 8, 1, 16, 64, 2, 3)
    q, k, v = (_randn((1, 2, 128, 64), i).cuda() for i in (1, 2, 3))
    ra.cache_trim(two.gpu, _i32([9]))
    o, lse = rd.ring_fwd(q, k, v, True)
    assert torch.isfinite(lse).all()
    assert ra.device_status() == ra.RA_ERR_PAGES             # still there for the cache's caller
    ra.wait_selftest(0.02)
    ra.cache_trim(two.gpu, _i32([9]))
    with pytest.raises(ra.RingAttnError) as e:
        rd.ring_fwd(q, k, v, True)
    assert e.value.code == ra.RA_ERR_TIMEOUT
    assert ra.device_status() == ra.RA_ERR_PAGES and ra.device_status() == 0


# ------------------------------------------------------------------------------------ a reserve that failed
def test_a_step_without_room_keeps_what_is_cached(ra):  # noqa: F811
    """Reserve, append, attend captured once: where reserve finds no room, append writes nothing over the
    tokens that are there."""
    two = Both(ra, pages=4, heads=1, page=16, Dh=64, slots=3, max_pages=2)
    two.add([0, 1], [15, 30])
    slots, n = _i32([0, 1, -1, 2]), _i32([1, 1, 1, 0])
    granted = _i32([9, 9, 9, 9])
    x = torch.zeros((4, 1, 1, 64), dtype=torch.bfloat16, device="cuda")
    q = _randn((4, 2, 1, 64), 3).cuda()

    def step():
        ra.cache_reserve(two.gpu, slots, n, granted=granted)
        ra.cache_append(two.gpu, 0, slots, granted, x, x)
        return ra.cache_attend(two.gpu, 0, slots, granted, q)

    books = [t.clone() for t in (two.gpu.table, two.gpu.lens, two.gpu.refs, two.gpu.k, two.gpu.v, two.gpu.k_scale, two.gpu.v_scale)]
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = step()
    for t, b in zip((two.gpu.table, two.gpu.lens, two.gpu.refs, two.gpu.k, two.gpu.v, two.gpu.k_scale, two.gpu.v_scale), books):
        t.copy_(b)
    for i in range(6):
        # slot 1 is full after two tokens (its entry alone is refused); slot 0 goes on to its second page
        x.copy_(_randn(x.shape, 20 + i))
        graph.replay()
        room = two.cpu[0].lens[1] < 32
        got = [1, 1 if room else 0, 0, 0]
        assert ra.device_status() == (0 if room else ra.RA_ERR_PAGES)
        assert granted.tolist() == got
        two.cpu[0].reserve([0, 1], got[:2])
        two.cpu[0].append([0, 1], got[:2], x[:2].float().cpu().numpy(), x[:2].float().cpu().numpy())
        two.check()
        # check_attend leaves rows that were not granted at 7
        for b in (2, 3) if room else (1, 2, 3):
            assert torch.all(o[b] == 0) and torch.all(torch.isneginf(lse[b]))
            o[b], lse[b] = 7.0, 7.0
        check_attend(two.cpu[0], [0, 1, -1, -1], got, q, o, lse)
    # no page left for the batch: nobody is granted anything
    x.copy_(_randn(x.shape, 40))
    ra.cache_trim(two.gpu, _i32([1]), _i32([16]))
    two.cpu[0].trim([1], [16])
    two.add([2], [16])
    ra.cache_reserve(two.gpu, _i32([0, 1]), _i32([1, 1]), granted=granted[:2])
    assert ra.device_status() == ra.RA_ERR_PAGES and granted.tolist()[:2] == [0, 0]
    ra.cache_append(two.gpu, 0, _i32([0, 1]), granted[:2], x[:2], x[:2])
    two.check()


def test_granted_is_checked(ra):  # noqa: F811
    two = Both(ra, 8, 1, 16, 64, 2, 3)
    for bad in (torch.zeros(2, dtype=torch.int64, device="cuda"), torch.zeros(2, dtype=torch.int32), _i32([0])):
        with pytest.raises(ValueError):
            ra.cache_reserve(two.gpu, _i32([0, 1]), _i32([1, 1]), granted=bad)
    n = _i32([1, 1])
    with pytest.raises(ra.RingAttnError):
        ra.cache_reserve(two.gpu, n, _i32([1, 1]), granted=n)                  # over the slots
    ra.cache_reserve(two.gpu, _i32([0, 1]), n, granted=n)                      # over the counts themselves
    assert n.tolist() == [1, 1] and ra.device_status() == 0


# ------------------------------------------------------------------------------------ contexts cut across ranks
def test_cached_parts_in_a_graph(ra):  # noqa: F811
    from long_context_exact_fwd_b200 import ring_dist as rd
    two = Both(ra, 20, 2, 16, 64, 3, 8)
    two.add([0, 2], [100, 37])
    q = _randn((3, 4, 1, 64), 3).cuda()
    slots, n = _i32([2, -1, 0]), _i32([1, 1, 1])
    want = rd.ring_cache_attend(two.gpu, 0, slots, n, q, True)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = rd.ring_cache_attend(two.gpu, 0, slots, n, q, True)
    graph.replay()
    assert ra.device_status() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    # errors are the cache's: left for device_status(), as by every other call on it
    rd.ring_cache_attend(two.gpu, 0, _i32([2, 7, 0]), n, q, True)
    assert ra.device_status() == ra.RA_ERR_PAGES


# ------------------------------------------------------------------------------------ many sequences
@pytest.mark.parametrize("B,g,T", [(300, 4, 5), (1024, 2, 1), (257, 4, 20), (1024, 64, 1)])
def test_attention_of_many_sequences(ra, B, g, T):  # noqa: F811
    """More entries than a block has threads, ragged, some of them padding."""
    rng = np.random.default_rng(B)
    two = Both(ra, 4 * B + 4, 1, 16, 64, B, 5)
    lengths = [int(x) for x in rng.integers(1, 64, B)]
    perm = [int(s) for s in rng.permutation(B)]
    two.add(perm, lengths)
    slots = [-1 if i % 11 == 5 else s for i, s in enumerate(perm)]
    n_new = [int(min(x, rng.integers(0, T + 1))) for x in lengths]
    n_new[-1], slots[-1] = 1, perm[-1]
    two.attend(slots, n_new, g, T)
    two.attend(slots, n_new, g, T, causal=False, out_dtype=torch.float32)


def test_pages_of_many_sequences(ra):  # noqa: F811
    """Plans over hundreds of entries: shared, partly filled pages whose holders lie in different warps."""
    rng = np.random.default_rng(5)
    N = 600
    two = Both(ra, pages=2500, heads=1, page=16, Dh=64, slots=N, max_pages=6)
    first = list(range(0, 40))
    two.add(first, [int(x) for x in rng.integers(1, 60, 40)])
    dst = [int(s) for s in 40 + rng.permutation(N - 40)[:500]]
    two.fork([int(rng.integers(0, 40)) for _ in dst], dst)
    two.check()
    for step in range(3):
        slots = [int(s) for s in rng.permutation(first + dst)[:450]]
        slots[100], slots[333] = -1, -1
        n = [int(x) for x in rng.integers(0, 9, 450)]
        two.add(slots, n)
        two.check()
        two.trim([int(s) for s in rng.permutation(first + dst)[:200]], [int(x) for x in rng.integers(0, 50, 200)])
        two.check()
        two.compact()
        two.check()
    live = [int(s) for s in np.flatnonzero(two.cpu[0].lens)][:300]
    two.attend(live, [1] * len(live), 2, 1)
