"""Cache attention of many new tokens (64 rows per key/value head and more take the tcgen05 kernel), with
the oracle, the state and the tolerances of test_cache_gpu.py."""
import numpy as np
import pytest
import torch

from test_cache_gpu import Both, _i32, _randn, check_attend, ra  # noqa: F401

pytestmark = pytest.mark.gpu

# (heads, Hq, T, Dh, page, lengths): one to many items of 256 rows, query heads that do not divide a tile,
# chunks that are the whole sequence, contexts around key tiles of 128, ends inside pages, few rows of a
# long context (every SM has a part), more sequences than SMs
CHUNKS = [(1, 1, 64, 128, 16, [64]), (1, 1, 64, 128, 64, [30000]), (2, 6, 40, 64, 32, [1000, 40, 77]),
          (1, 4, 300, 128, 64, [300, 1500]), (2, 2, 129, 128, 128, [5000, 129, 200, 255, 256, 257]),
          (1, 8, 200, 64, 16, [201, 300]), (4, 20, 64, 128, 64, [2049, 127, 128]), (1, 3, 257, 128, 32, [771]),
          (1, 64, 1, 64, 64, [500, 1]), (1, 64, 2, 128, 16, [17] * 160)]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("heads,Hq,T,Dh,page,lengths", CHUNKS)
def test_chunk_matches_oracle(ra, heads, Hq, T, Dh, page, lengths, causal):  # noqa: F811
    need = [-(-n // page) for n in lengths]
    two = Both(ra, sum(need) + 2, heads, page, Dh, len(lengths), max(need) + 1)
    slots = [int(s) for s in np.random.default_rng(1).permutation(len(lengths))]
    two.add(slots, lengths)
    n_new = [min(T, n) for n in lengths]
    two.attend(slots, n_new, Hq, T, causal=causal, q_scale=2.0)
    two.attend(slots, n_new, Hq, T, causal=causal, scale=0.3, seed=8, out_dtype=torch.float32)


def test_chunks_of_several_lengths_and_padding(ra):  # noqa: F811
    two = Both(ra, 60, 2, 32, 128, 5, 16)
    two.add([0, 1, 2, 4], [300, 90, 10, 200])
    q, o, lse = two.attend([4, -1, 0, 3, 1, 2], [150, 100, 1, 5, 0, 10], Hq=4, T=150, causal=False)
    assert torch.all(o[3, :, :5] == 0) and torch.all(torch.isneginf(lse[3, :, :5]))      # slot 3 holds nothing
    two.attend([4, -1, 0, 1, 2], [150, 100, 64, 0, 10], Hq=4, T=150)


def test_scales_that_differ_from_page_to_page(ra):  # noqa: F811
    """Value scales that grow along the context (the accumulator changes units), shrink, and span most of the
    range; key scales likewise with scores kept moderate; pages of zeros."""
    for Dh, page in ((128, 16), (64, 32)):
        two = Both(ra, 200, 1, page, Dh, 3, 70)
        n = 600
        assert two.reserve([0, 1, 2], [n] * 3)
        k, v = _randn((3, 1, n, Dh), 1), _randn((3, 1, n, Dh), 2)
        grow = torch.exp2(torch.arange(n) // page * 2.0).clamp(max=2.0 ** 60)
        v[0] = v[0] * grow.view(1, n, 1)
        v[1] = v[1] * (1.0 / grow).view(1, n, 1)
        v[2, :, 100:300] = 0
        v[2, :, 300:] *= 1e-6
        k[1] = k[1] * torch.exp2(-(torch.arange(n) // page % 5).float()).view(1, n, 1)
        k[2, :, 50:90] = 0
        two.append([0, 1, 2], [n] * 3, kv=(k, v))
        two.check()
        two.attend([0, 1, 2], [100] * 3, 2, 100)
        two.attend([2, 1], [100] * 2, 1, 100, q_scale=1e-20)
        two.attend([2, 0], [64] * 2, 1, 64, scale=3.0)


def test_values_that_are_not_finite_in_a_chunk(ra):  # noqa: F811
    """As for few tokens: NaN reaches the queries that see it and no others, over several pieces."""
    two = Both(ra, 40, 1, 32, 64, 2, 20)
    two.gpu.k.fill_(0x7f)
    two.gpu.v.fill_(0x7f)
    n, T = 500, 300
    assert two.reserve([0, 1], [n, n])
    k, v = _randn((2, 1, n, 64), 1), _randn((2, 1, n, 64), 2)
    marks = {5: 210, 9: 333, 17: 498, 63: 260}
    for d, t in marks.items():
        v[0, 0, t, d] = float("nan") if d % 2 else float("inf")
    k[1, 0, 400, 3] = float("inf")
    two.append([0, 1], [n, n], kv=(k, v))
    two.check()
    q = _randn((2, 2, T, 64), 3).cuda()
    for _ in range(2):
        o, lse = ra.cache_attend(two.gpu, 0, _i32([0, 1]), None, q)
        assert ra.device_status() == 0
        pos = torch.arange(n - T, n)
        bad = torch.isnan(o[0]).cpu()
        want = torch.zeros((T, 64), dtype=torch.bool)
        for d, t in marks.items():
            want[:, d] = pos >= t
        assert torch.equal(bad, want.expand(2, T, 64)) and torch.isfinite(lse[0]).all()
        hit = pos >= 400
        assert torch.isnan(o[1][:, hit]).all() and torch.isnan(lse[1][:, hit]).all()
        assert torch.isfinite(o[1][:, ~hit]).all() and torch.isfinite(lse[1][:, ~hit]).all()
    # a clean sequence afterwards, in the same launch shapes
    two.trim([0, 1], [0, 0])
    assert two.reserve([0, 1], [n, n])
    two.append([0, 1], [n, n])
    two.attend([0, 1], [T, T], 2, T)


def test_both_kernels_agree_where_they_meet(ra):  # noqa: F811
    two = Both(ra, 200, 2, 32, 128, 1, 190)
    two.add([0], [5000])
    q = _randn((1, 2, 64, 128), 4).cuda()
    o, lse = ra.cache_attend(two.gpu, 0, _i32([0]), None, q)                # 64 rows a head
    a, l = ra.cache_attend(two.gpu, 0, _i32([0]), None, q[:, :, 1:])        # 63
    assert ra.device_status() == 0
    assert (o[:, :, 1:].float() - a.float()).abs().max() <= 2.0 ** -7 * o.float().abs().max()
    assert (lse[:, :, 1:] - l).abs().max() <= 1e-5


def test_chunk_results_do_not_change_from_run_to_run(ra):  # noqa: F811
    two = Both(ra, 400, 2, 16, 64, 3, 200)
    two.add([0, 1, 2], [2000, 333, 1777])
    q = _randn((3, 8, 100, 64), 5).cuda()
    first = [x.clone() for x in ra.cache_attend(two.gpu, 0, _i32([0, 1, 2]), None, q)]
    for _ in range(10):
        for a, b in zip(first, ra.cache_attend(two.gpu, 0, _i32([0, 1, 2]), None, q)):
            assert torch.equal(a, b)


def test_a_prompt_in_chunks_is_the_prompt_at_once(ra):  # noqa: F811
    """Reserve, append and attend chunk by chunk; a page that a later chunk completes may restate older
    codes, so each chunk is compared with the oracle's cache at that time."""
    two = Both(ra, 60, 2, 64, 128, 1, 20)
    for i, n in enumerate([200, 130, 64, 300]):
        two.add([0], [n], size := 1.0 + i)
        two.check()
        two.attend([0], [n], 4, n, q_scale=1.0 / size, seed=20 + i)


def test_chunk_in_a_graph_and_on_two_streams(ra):  # noqa: F811
    two = Both(ra, 60, 1, 32, 128, 2, 25)
    two.add([0, 1], [700, 300])
    q, slots = _randn((2, 4, 90, 128), 6).cuda(), _i32([0, 1])
    want = ra.cache_attend(two.gpu, 0, slots, None, q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = ra.cache_attend(two.gpu, 0, slots, None, q)
    side = [torch.cuda.Stream() for _ in range(2)]
    outs = []
    for s in side:                                           # both calls may be under way at once
        s.wait_stream(torch.cuda.current_stream())
        outs.append(ra.cache_attend(two.gpu, 0, slots, None, q, stream=s))
    g.replay()
    torch.cuda.synchronize()
    assert ra.device_status() == 0
    for o, lse in [got] + outs:
        assert torch.equal(o, want[0]) and torch.equal(lse, want[1])
    check_attend(two.cpu[0], [0, 1], [90, 90], q, *want)
