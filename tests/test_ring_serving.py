"""Rotary positions in the sequence-sharded rings, and attention over contexts cut across ranks, on CPU: 2 and 3
gloo ranks with the float64 oracle as the block work (the product binds the CUDA library instead)."""
import os
import sys

import numpy as np
import pytest
import torch
import torch.distributed as dist
import torch.multiprocessing as mp

from test_ring_dist import ROOT, _free_port, _full_inputs, _per_head


def _oracle_work():
    import oracle
    from oracle import cache as oc

    def block_fwd(q, k, v, masked):
        return _per_head(lambda a, b, c: oracle.attn_fwd(a, b, c, masked), q, k, v)

    def merge(o_parts, lse_parts):
        o, l = oracle.lse_merge(o_parts.numpy(), lse_parts.numpy())
        return torch.from_numpy(o), torch.from_numpy(l)

    def block_bwd(q, k, v, o, lse, do, masked):
        return _per_head(lambda a, b, c, d, e, f: oracle.attn_bwd_given_stats(a, b, c, d, e, f, masked), q, k, v, o, lse, do)

    def rotate(q, k, plan, pos, inverse):
        p = pos.numpy()[None].repeat(q.shape[0], 0)
        return tuple(torch.from_numpy(oc.rope(x.numpy(), p, plan, True, 1.25, inverse)) for x in (q, k))

    return oracle, oc, block_fwd, merge, block_bwd, rotate


def _start(rank, world, port):
    sys.path.insert(0, ROOT)
    sys.path.insert(0, os.path.join(ROOT, "tests"))
    os.environ.update(MASTER_ADDR="127.0.0.1", MASTER_PORT=str(port))
    from datetime import timedelta
    dist.init_process_group("gloo", rank=rank, world_size=world, timeout=timedelta(seconds=60))


def _rope_rank(rank, world, port, zigzag, out):
    _start(rank, world, port)
    oracle, oc, block_fwd, merge, block_bwd, rotate = _oracle_work()
    from long_context_exact_fwd_b200 import ring_dist as rd
    B, H, c, Dh = 1, 2, 6, 8
    q, k, v, do = _full_inputs(B, H, world * c, Dh, seed=17)
    plan = np.array([1.0, 0.3])
    fwd, bwd = (rd.ring_fwd_zigzag, rd.ring_bwd_zigzag) if zigzag else (rd.ring_fwd, rd.ring_bwd)
    shard = (lambda x: rd.zigzag_shard(x, rank, world)) if zigzag else \
        (lambda x: x[:, :, rank * c:(rank + 1) * c].contiguous())
    o, lse = fwd(shard(q), shard(k), shard(v), True, block_fwd=block_fwd, merge=merge, rope=plan, rotate=rotate)
    got = bwd(shard(q), shard(k), shard(v), o, lse, shard(do), True, block_bwd=block_bwd, rope=plan, rotate=rotate)
    # the whole sequence on one rank, its gradient by autograd
    import torch as t
    qq, kk, vv = (x.clone().requires_grad_() for x in (q, k, v))
    a = t.arange(world * c, dtype=t.float64)[:, None] * t.tensor(plan)

    def turn(x):
        x1, x2 = x[..., 0:4:2], x[..., 1:4:2]
        y = t.stack((x1 * a.cos() - x2 * a.sin(), x1 * a.sin() + x2 * a.cos()), -1).flatten(-2) * 1.25
        return t.cat((y, x[..., 4:]), -1)

    s = turn(qq) @ turn(kk).transpose(2, 3) / Dh ** 0.5
    s = s.masked_fill(t.ones(world * c, world * c, dtype=t.bool).triu(1), float("-inf"))
    O = s.softmax(-1) @ vv
    O.backward(do)
    err = lambda x, y: float((x.double() - shard(y.detach())).abs().max())
    out[rank] = (err(o, O),) + tuple(err(x, y.grad) for x, y in zip(got, (qq, kk, vv)))
    dist.barrier()
    dist.destroy_process_group()


@pytest.mark.parametrize("zigzag", [False, True])
@pytest.mark.parametrize("world", [2, 3])
def test_ring_with_rotary_positions(world, zigzag):
    with mp.Manager() as m:
        out = m.dict()
        mp.spawn(_rope_rank, args=(world, _free_port(), zigzag, out), nprocs=world, join=True)
        for r in range(world):
            assert max(out[r][:1]) < 1e-9 and max(out[r][1:]) < 1e-6, out[r]    # gradients are summed in float32


def _cache_rank(rank, world, port, out):
    _start(rank, world, port)
    oracle, oc, _, merge, _, _ = _oracle_work()
    from long_context_exact_fwd_b200 import ring_dist as rd
    rng = np.random.default_rng(5)
    n, T, H, Dh = 50, 3, 2, 64
    k, v, q = rng.standard_normal((1, 1, n, Dh)), rng.standard_normal((1, 1, n, Dh)), rng.standard_normal((1, H, T, Dh))
    # pages of 16 whole on one rank, so that the parts hold the values that one cache would
    cut = [0, 16, 32, n] if world == 3 else [0, 32, n]

    def cached(a, z):
        c = oc.Cache(8, 1, 16, Dh, 1, 6)
        c.reserve([0], [z - a])
        c.append([0], [z - a], k[:, :, a:z], v[:, :, a:z])
        return c

    def attend(c, layer, slots, n_new, x, causal):
        o, l, _ = c.attend(0, x[0].numpy(), T, causal=causal)
        return torch.from_numpy(o)[None], torch.from_numpy(l)[None]

    mine = cached(cut[rank], cut[rank + 1])
    o, lse = rd.ring_cache_attend(mine, 0, None, None, torch.from_numpy(q), rank == world - 1, attend=attend, merge=merge)
    O, L, _ = cached(0, n).attend(0, q[0], T)
    out[rank] = (float(np.abs(o[0].numpy() - O).max()), float(np.abs(lse[0].numpy() - L).max()))
    dist.barrier()
    dist.destroy_process_group()


@pytest.mark.parametrize("world", [2, 3])
def test_cached_contexts_cut_across_ranks(world):
    with mp.Manager() as m:
        out = m.dict()
        mp.spawn(_cache_rank, args=(world, _free_port(), out), nprocs=world, join=True)
        for r in range(world):
            assert max(out[r]) < 1e-12, out[r]


def test_positions_of_the_assignments():
    from long_context_exact_fwd_b200 import ring_dist as rd
    x = torch.arange(24).view(1, 1, 24, 1)
    for world in (1, 2, 3):
        c = 24 // world
        for r in range(world):
            assert torch.equal(rd.ring_positions(r, world, c), torch.arange(r * c, (r + 1) * c))
            assert torch.equal(rd.zigzag_positions(r, world, c), rd.zigzag_shard(x, r, world).flatten())
    with pytest.raises(ValueError):
        rd.zigzag_positions(0, 2, 5)


# ------------------------------------------------------------------------------------ the library, one GPU
@pytest.mark.gpu
@pytest.mark.parametrize("zigzag", [False, True])
def test_emulated_rings_with_rotary_positions(zigzag):
    """Every rank's work through the library: the ring over blocks with rope equals the single call on the
    rotated whole sequence, forward and backward, at the bf16 bar of the ring tests."""
    from long_context_exact_fwd_b200 import build, ring_dist as rd
    build.ensure_built()
    from long_context_exact_fwd_b200 import ring_attn as ra
    from long_context_exact_fwd_b200.workloads import random_qkv
    from parity import assert_close_bf16
    D, S = 3, 768
    inp = random_qkv(1, 2, S, 128, seed=91, with_do=True)
    q, k, v, do = (inp[n].cuda() for n in ("q", "k", "v", "do"))
    plan = ra.rope_plan(ra.rope_inv_freq(64)[0])
    shard = (lambda x: [rd.zigzag_shard(x, r, D) for r in range(D)]) if zigzag else \
        (lambda x: [b.contiguous() for b in x.chunk(D, dim=2)])
    whole = rd.zigzag_unshard if zigzag else (lambda xs, dim=2: torch.cat(xs, dim=dim))
    fwd, bwd = (rd.ring_fwd_zigzag_emulated, rd.ring_bwd_zigzag_emulated) if zigzag else \
        (rd.ring_fwd_emulated, rd.ring_bwd_emulated)
    outs = fwd(shard(q), shard(k), shard(v), True, rope=plan)
    o, lse = whole([a for a, _ in outs]), whole([b for _, b in outs])
    qr, kr = ra.rope(q, plan, k=k)
    want, want_lse = ra.fwd(qr, kr, v, 1, True)
    got = bwd(shard(q), shard(k), shard(v), [a for a, _ in outs], [b for _, b in outs], shard(do), True, rope=plan)
    dq, dk, dv = ra.bwd(qr, kr, v, want, want_lse, do, 1, True)
    dq, dk = ra.rope(dq, plan, k=dk, inverse=True)
    assert ra.device_status() == 0
    assert (lse - want_lse).abs().max() <= 1e-3
    for name, a, b in (("o", o, want), ("dq", whole(got[0]), dq), ("dk", whole(got[1]), dk), ("dv", whole(got[2]), dv)):
        assert_close_bf16(a.float().cpu().numpy(), b.float().cpu().numpy(), name)


@pytest.mark.gpu
def test_cached_contexts_of_one_rank():
    """ring_cache_attend without a process group is the cache's attention, padding rows empty."""
    from long_context_exact_fwd_b200 import build, ring_dist as rd
    build.ensure_built()
    from long_context_exact_fwd_b200 import ring_attn as ra
    from test_cache_gpu import Both, _i32, _randn, check_attend
    two = Both(ra, 20, 2, 16, 64, 3, 8)
    two.add([0, 2], [100, 37])
    q = _randn((3, 4, 2, 64), 3)
    slots, n_new = _i32([2, -1, 0]), _i32([1, 2, 2])
    o, lse = rd.ring_cache_attend(two.gpu, 0, slots, n_new, q.cuda(), True)
    assert torch.all(o[1] == 0) and torch.all(o[0, :, 1] == 0) and torch.all(torch.isneginf(lse[1]))
    o[1], o[0, :, 1], lse[1], lse[0, :, 1] = 7.0, 7.0, 7.0, 7.0
    check_attend(two.cpu[0], [2, -1, 0], [1, 2, 2], q, o, lse)
