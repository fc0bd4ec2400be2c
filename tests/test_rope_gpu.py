"""Rotary positions (ring_attn_rope) against the float64 oracle.

Tolerance, from the arithmetic: the phase is exact, the float angle is off by at most half a step at
an eighth of a turn (2^-25 turns, 2^-22 rad), sine and cosine by 2 steps more (2^-22), the two
products and the sum by 2^-23 of their terms: 2^-20 A (|x1| + |x2|) covers them.  Then the output is
rounded once: half a step, 2^-8 |y| in bf16 and 2^-24 |y| in float32."""
import numpy as np
import pytest
import torch

from oracle import cache as oc

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ra():
    from long_context_exact_fwd_b200 import build
    build.ensure_built()
    from long_context_exact_fwd_b200 import ring_attn
    return ring_attn


def _check(got, x, pos, w, inter, amp, inverse=False):
    xd = x.double().cpu().numpy()
    ref = oc.rope(xd, pos, w, inter, amp, inverse)
    r = 2 * len(w)
    i1, i2 = (np.arange(0, r, 2), np.arange(1, r, 2)) if inter else (np.arange(r // 2), np.arange(r // 2, r))
    size = np.zeros_like(xd)
    size[..., i1] = size[..., i2] = np.abs(xd[..., i1]) + np.abs(xd[..., i2])
    half = 2.0 ** -8 if x.dtype == torch.bfloat16 else 2.0 ** -24
    tol = half * np.abs(ref) + 2.0 ** -20 * abs(amp) * size
    err = np.abs(got.double().cpu().numpy() - ref)
    assert np.all(err <= tol), float((err - tol).max())
    assert torch.equal(got[..., r:], x[..., r:])


def _x(shape, dtype, seed):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(shape, generator=g).to(dtype).cuda()


# (B, S, Hq, Hk, Dh, rot): one token, odd lengths, whole and part heads, odd numbers of pairs, widths
# that only single elements fit
SHAPES = [(1, 1, 1, 0, 64, 64), (3, 1, 8, 2, 128, 128), (2, 37, 3, 1, 128, 96), (1, 130, 2, 2, 64, 2), (2, 9, 2, 1, 128, 98),
          (1, 5, 2, 1, 80, 24), (1, 7, 1, 1, 66, 66), (1, 1000, 5, 3, 128, 64), (5, 3, 20, 4, 256, 256)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("B,S,Hq,Hk,Dh,rot", SHAPES)
def test_rope_matches_oracle(ra, B, S, Hq, Hk, Dh, rot, inter, dtype):
    w, amp = ra.rope_inv_freq(rot, scaling="ramp", factor=4.0, original_length=100)
    plan = ra.rope_plan(w, "interleaved" if inter else "half", amp)
    q = _x((B, Hq, S, Dh), dtype, 1)
    pos = torch.randint(-50, 5000, (B, S), generator=torch.Generator().manual_seed(2)).cuda()
    if Hk:
        k = _x((B, Hk, S, Dh), dtype, 3)
        a, b = ra.rope(q, plan, k=k, pos=pos)
        _check(b, k, pos.cpu().numpy(), w.numpy(), inter, amp)
    else:
        a = ra.rope(q, plan, pos=pos)
    _check(a, q, pos.cpu().numpy(), w.numpy(), inter, amp)


@pytest.mark.parametrize("start", [0, 1_000_003, 2 ** 31 + 5, 2 ** 40 + 1, -(2 ** 33) - 7])
def test_far_positions(ra, start):
    """Whole turns are exact: frequencies that are binary fractions of a turn have angles known
    exactly at any position."""
    turns = torch.tensor([0.5, 0.25, 1.0 / 1024, 3.0 / 2 ** 20], dtype=torch.float64)
    plan = ra.rope_plan(turns * 2 * np.pi)
    want = [round(float(t) * 2 ** 64) for t in turns]
    assert all(abs((s - v + 2 ** 63) % 2 ** 64 - 2 ** 63) <= 2 ** 12 for s, v in zip(plan.steps.tolist(), want))
    plan = plan._replace(steps=torch.tensor([v - 2 ** 64 if v >= 2 ** 63 else v for v in want]).cuda())
    q = _x((1, 2, 33, 64), torch.float32, 4)
    y = ra.rope(q, plan, offset=start)
    pos = np.array([[start + i for i in range(33)]], dtype=object)
    small = np.stack([np.array([(int(p) * int(round(float(t) * 2 ** 20))) % 2 ** 20 for p in pos[0]], dtype=np.float64)
                      for t in turns], -1) / 2 ** 20          # fractions of a turn
    x = q.double().cpu().numpy()
    a = 2 * np.pi * small[None, None]
    ref = x.copy()
    ref[..., :4] = x[..., :4] * np.cos(a) - x[..., 4:8] * np.sin(a)
    ref[..., 4:8] = x[..., :4] * np.sin(a) + x[..., 4:8] * np.cos(a)
    assert np.abs(y.double().cpu().numpy() - ref).max() <= 2.0 ** -20 * 2 * np.abs(x).max() + 2.0 ** -24 * np.abs(ref).max()


def test_views_in_place_and_streams(ra):
    """Q and K as columns of one projection, rotated where they lie; then on another stream."""
    B, S, H, Hk, Dh = 2, 19, 6, 2, 128
    w, _ = ra.rope_inv_freq(Dh)
    plan = ra.rope_plan(w)
    rows = _x((B, S, H + 2 * Hk, Dh), torch.bfloat16, 5)
    keep = rows.clone()
    q, k = (rows[:, :, :H].permute(0, 2, 1, 3), rows[:, :, H:H + Hk].permute(0, 2, 1, 3))
    pos = torch.arange(100, 100 + S).cuda()
    want = ra.rope(q, plan, k=k, pos=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ra.rope(q, plan, k=k, pos=pos, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    raw = ra.rope(q, plan, k=k, pos=pos, stream=torch.cuda.current_stream().cuda_stream)
    for a, b, c in zip(want, got, raw):
        assert torch.equal(a, b) and torch.equal(a, c)
    p2 = np.broadcast_to(pos.cpu().numpy(), (B, S))
    _check(want[0], q, p2, w.numpy(), False, 1.0)
    ra.rope(q, plan, k=k, pos=pos, out=q, k_out=k)
    assert torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(rows[:, :, H + Hk:], keep[:, :, H + Hk:])
    # inputs that share a dimension, and odd strides that only single elements fit
    shared = _x((1, 1, S, Dh), torch.float32, 6).expand(B, H, S, Dh)
    _check(ra.rope(shared, plan, pos=pos), shared, p2, w.numpy(), False, 1.0)
    odd = _x((B, H, S, Dh + 3), torch.bfloat16, 7)[..., 1:Dh + 1]
    for name in ("half", "interleaved"):
        _check(ra.rope(odd, ra.rope_plan(w, name), pos=pos), odd, p2, w.numpy(), name != "half", 1.0)


@pytest.mark.parametrize("inter", [False, True])
def test_gradient_is_the_inverse_turn(ra, inter):
    """<g, J dx> with J dx by differences of the (linear) forward equals <J^T g, dx>; and against
    the formula's gradient through torch autograd in float64."""
    w, amp = ra.rope_inv_freq(48, scaling="ramp", factor=2.0, original_length=64)
    plan = ra.rope_plan(w, "interleaved" if inter else "half", amp)
    x, g, dx = (_x((2, 3, 11, 64), torch.float32, s) for s in (8, 9, 10))
    pos = torch.randint(0, 10 ** 6, (2, 11), generator=torch.Generator().manual_seed(11)).cuda()
    back = ra.rope(g, plan, pos=pos, inverse=True)
    diff = (ra.rope(x + dx, plan, pos=pos).double() - ra.rope(x - dx, plan, pos=pos).double()) / 2
    lhs, rhs = (g.double() * diff).sum(), (back.double() * dx.double()).sum()
    # each of the 4224 terms is off by at most 2^-19 of |g| |x|-sized factors
    bound = 2.0 ** -19 * float((g.double().norm() * (dx.double().norm() + x.double().norm())))
    assert abs(float(lhs - rhs)) <= bound
    xd = x.double().cpu().requires_grad_()
    a = pos.cpu().double()[:, None, :, None] * w
    c, s = amp * a.cos(), amp * a.sin()
    x1, x2 = (xd[..., 0:48:2], xd[..., 1:48:2]) if inter else (xd[..., :24], xd[..., 24:48])
    y1, y2 = x1 * c - x2 * s, x1 * s + x2 * c
    y = torch.cat((torch.stack((y1, y2), -1).flatten(-2) if inter else torch.cat((y1, y2), -1), xd[..., 48:]), -1)
    y.backward(g.double().cpu())
    _check(back, g, pos.cpu().numpy(), w.numpy(), inter, amp, inverse=True)
    assert (xd.grad - back.double().cpu()).abs().max() <= 2.0 ** -19 * 2 * amp * float(g.abs().max())


def test_special_values_stay_in_their_pair(ra):
    w, _ = ra.rope_inv_freq(64)
    q = _x((1, 1, 8, 64), torch.bfloat16, 12)
    q[0, 0, 3, 5], q[0, 0, 4, 40] = float("nan"), float("inf")
    y = ra.rope(q, ra.rope_plan(w), offset=3)
    bad = ~torch.isfinite(y[0, 0])
    want = torch.zeros_like(bad)
    want[3, 5] = want[3, 37] = want[4, 8] = want[4, 40] = True
    assert torch.equal(bad, want)


def test_graph_replay_takes_new_positions(ra):
    w, _ = ra.rope_inv_freq(128)
    plan = ra.rope_plan(w)
    q, pos = _x((4, 8, 1, 128), torch.bfloat16, 13), torch.zeros((4, 1), dtype=torch.int64, device="cuda")
    out = torch.empty_like(q)
    ra.rope(q, plan, pos=pos, out=out)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        ra.rope(q, plan, pos=pos, out=out)
    for start in (5, 1000):
        pos.copy_(torch.arange(start, start + 4).view(4, 1))
        g.replay()
        _check(out, q, pos.cpu().numpy(), w.numpy(), False, 1.0)


def test_refusals(ra):
    w, _ = ra.rope_inv_freq(64)
    plan = ra.rope_plan(w)
    q = _x((1, 2, 4, 64), torch.bfloat16, 14)
    with pytest.raises(ValueError):
        ra.rope(q.half(), plan)
    with pytest.raises(ValueError):
        ra.rope(q[..., :32], plan)
    with pytest.raises(ValueError):
        ra.rope(q, plan, pos=torch.zeros(4, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError):
        ra.rope(q, plan, pos=torch.zeros((2, 4), dtype=torch.int64, device="cuda"))
    with pytest.raises(ValueError):
        ra.rope(q, plan, pos=torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        ra.rope(q.transpose(2, 3), plan)
    with pytest.raises(ValueError):
        ra.rope(q, plan, k=q.float())
    with pytest.raises(ra.RingAttnError):
        ra.rope(q, plan, out=q.expand(1, 2, 4, 64).as_strided((1, 2, 4, 64), (0, 0, 64, 1)))
    big = torch.zeros(2 * q.numel(), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(ra.RingAttnError):
        ra.rope(big[:q.numel()].view(q.shape), plan, out=big[64:64 + q.numel()].view(q.shape))
    assert ra.device_status() == 0


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("Dh,rot", [(64, 2), (64, 10), (64, 30), (64, 60), (128, 26), (128, 102), (128, 126), (256, 58), (32, 14),
                                    (8, 6), (1024, 778)])
def test_rotated_widths_that_no_vector_divides(ra, Dh, rot, inter, dtype):
    """Rows start at vectors, the pairs' distance does not: apart and in place, rows of several tokens in one
    warp, more heads than a thread has at once, what a row's neighbours hold not finite."""
    B, S, H, Hk = 2, 5, 5, 2
    w, amp = ra.rope_inv_freq(rot, scaling="ramp", factor=2.0, original_length=50)
    plan = ra.rope_plan(w, "interleaved" if inter else "half", amp)
    rows = _x((B, S, H + 2 * Hk, Dh), dtype, 21)
    rows[:, :, H + Hk:] = float("nan")
    rows[:, 3, 2] = float("inf")
    q, k = (rows[:, :, :H].permute(0, 2, 1, 3), rows[:, :, H:H + Hk].permute(0, 2, 1, 3))
    pos = torch.arange(7, 7 + S).cuda()
    p2 = np.broadcast_to(pos.cpu().numpy(), (B, S))
    for inverse in (False, True):
        a, b = ra.rope(q, plan, k=k, pos=pos, inverse=inverse)
        for got, x in ((a, q), (b, k)):
            ok = [s for s in range(S) if s != 3]
            _check(got[:, :, ok], x[:, :, ok], p2[:, ok], w.numpy(), inter, amp, inverse)
        assert torch.isfinite(a[:, [h for h in range(H) if h != 2], 3]).all()
        assert torch.equal(a[:, 2, 3, rot:], q[:, 2, 3, rot:])
        keep = rows.clone()
        ra.rope(q, plan, k=k, pos=pos, inverse=inverse, out=q, k_out=k)
        for x, want in ((q, a), (k, b)):
            assert torch.equal(x.nan_to_num(nan=5.0), want.nan_to_num(nan=5.0))
        assert torch.equal(rows[:, :, H + Hk:].isnan(), keep[:, :, H + Hk:].isnan())
        rows.copy_(keep)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("shift,rot", [(4, 128), (4, 30), (2, 64), (2, 30), (1, 64), (8, 90)])
def test_rows_that_start_at_smaller_vectors(ra, shift, rot, inter, dtype):
    B, S, H, Dh = 2, 6, 5, 128
    w, _ = ra.rope_inv_freq(rot)
    x = _x((B, H, S, Dh + shift), dtype, 31)[..., shift:]
    p2 = np.broadcast_to(np.arange(50, 50 + S), (B, S))
    y = ra.rope(x, ra.rope_plan(w, "interleaved" if inter else "half"), offset=50)
    _check(y, x, p2, w.numpy(), inter, 1.0)
    ra.rope(x, ra.rope_plan(w, "interleaved" if inter else "half"), offset=50, out=x)
    assert torch.equal(x, y)


@pytest.mark.parametrize("start", [1_000_003, 2 ** 31 + 5, 2 ** 40 + 1, -(2 ** 43) - 7])
@pytest.mark.parametrize("kw", [dict(), dict(scaling="ramp", factor=8.0, original_length=8192)])
def test_far_positions_of_a_plan(ra, start, kw):
    """The plan as it is made: its steps are the nearest, so the phase is off by position 2^-65 turns."""
    from decimal import localcontext
    from test_oracle_cache import exact_turns
    w, amp = ra.rope_inv_freq(64, **kw)
    q = _x((1, 2, 9, 64), torch.float32, 4)
    y = ra.rope(q, ra.rope_plan(w, amplitude=amp), offset=start).double().cpu().numpy()
    # angles in turns, whole ones dropped
    with localcontext() as ctx:
        ctx.prec = 110
        per = [exact_turns(f) for f in w.tolist()]
        turns = np.array([[float(t * (start + i) - (t * (start + i)).to_integral_value()) for t in per] for i in range(9)])
    c, s = amp * np.cos(2 * np.pi * turns), amp * np.sin(2 * np.pi * turns)
    x = q.double().cpu().numpy()
    x1, x2 = x[..., :32], x[..., 32:]
    ref = np.concatenate((x1 * c - x2 * s, x1 * s + x2 * c), -1)
    size = np.tile(np.abs(x1) + np.abs(x2), 2)
    tol = 2.0 ** -24 * np.abs(ref) + (2.0 ** -20 + 2 * np.pi * abs(start) * 2.0 ** -65) * amp * size
    assert np.all(np.abs(y - ref) <= tol), float((np.abs(y - ref) / tol).max())
