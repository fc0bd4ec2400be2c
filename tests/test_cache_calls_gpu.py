"""Calls on the cache that its documentation allows."""
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
