"""Measured cases of the serving and position operators: rotary positions, the 8-bit key/value cache
(append, read back, attention of new queries over it) and the management of its pages.

`run` makes one pass: in plain float32 torch operations (`own` false), or through the library's
entry points (`own` true).  `exact` gives the same outputs in float64 from the definitions.
"""
import math

import torch

own = False

DEV = "cuda"
E_MIN, E_MAX = -117, 120          # exponents a block's scale may take
TOP = 240.0 * 2.0 ** 120          # largest magnitude the cache represents at the largest scale


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one new token in each of 32 running sequences: Q and K straight from a fused projection
        dict(name="rope_step", op="rope", B=32, S=1, Hq=32, Hk=8, Dh=128, rot=128, layout="half", dtype="bf16",
             scaling="ramp", factor=8.0, start=120_000, inverse=False),
        # a 16K-token prompt or training sequence, all heads of Q and K
        dict(name="rope_prompt", op="rope", B=1, S=16384, Hq=16, Hk=16, Dh=128, rot=128, layout="half", dtype="bf16",
             scaling="none", factor=1.0, start=0, inverse=False),
        # gradients of a partly rotated head in float32, odd length, far positions (a later ring block)
        dict(name="rope_grad_f32", op="rope", B=2, S=4099, Hq=8, Hk=2, Dh=128, rot=96, layout="interleaved",
             dtype="f32", scaling="linear", factor=4.0, start=1_000_003, inverse=True),
        # one token appended to each of 64 sequences in the middle of a page, that page read back
        dict(name="append_step", op="append", B=64, T=1, ctx=4096, Hk=8, Dh=128, page=64),
        # an 8K-token prompt written behind a shared prefix that ends inside a page, and read back
        dict(name="append_prompt", op="append", B=2, T=8192, ctx=1000, Hk=16, Dh=128, page=64),
        # the smallest call: one sequence, a short context, one query
        dict(name="attend_short", op="attend", B=1, T=1, ctx=777, Hq=16, Hk=16, Dh=128, page=64, ragged=False),
        # a decoding batch with contexts of very different lengths
        dict(name="attend_batch", op="attend", B=32, T=1, ctx=16384, Hq=32, Hk=8, Dh=128, page=64, ragged=True),
        # one long context, 128K tokens, 8 key/value heads
        dict(name="attend_long", op="attend", B=1, T=1, ctx=131072, Hq=32, Hk=8, Dh=128, page=128, ragged=False),
        # several new tokens a sequence (drafted tokens to be checked), small pages and heads
        dict(name="attend_draft", op="attend", B=16, T=5, ctx=5003, Hq=16, Hk=4, Dh=64, page=16, ragged=True),
        # a chunk of a long prompt against what is cached already
        dict(name="attend_chunk", op="attend", B=1, T=2048, ctx=16384, Hq=16, Hk=4, Dh=128, page=64, ragged=False),
        # sequences ended, others forked in their place, and every fork's shared last page copied
        dict(name="pages_fork", op="fork", slots=64, ctx=4100, layers=2, Hk=8, Dh=128, page=64),
        # a pool with holes brought together
        dict(name="pages_compact", op="compact", slots=48, ctx=4100, layers=2, Hk=8, Dh=128, page=64),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "append", "attend", "attend", "chunk", "fork", "compact"])
    Dh = rng.choice([64, 128])
    page = rng.choice([16, 32, 64, 128])
    Hk = rng.choice([1, 2, 4, 8, 16])
    if op == "rope":
        B, Hq = _log(rng, 1, 48), Hk * rng.choice([1, 2, 3, 4])
        S = max(1, min(_log(rng, 1, 16384), 60_000_000 // (B * (Hq + Hk) * Dh)))
        scaling = rng.choice(["none", "linear", "ramp"])
        return dict(op="rope", B=B, S=S, Hq=Hq, Hk=Hk, Dh=Dh, rot=2 * rng.randint(1, Dh // 2),
                    layout=rng.choice(["half", "interleaved"]), dtype=rng.choice(["bf16", "f32"]), scaling=scaling,
                    factor=1.0 if scaling == "none" else round(rng.uniform(1.5, 16.0), 3),
                    start=_log(rng, 1, 2_000_000), inverse=rng.random() < 0.5)
    if op == "append":
        B = _log(rng, 1, 64)
        T = max(1, min(_log(rng, 1, 8192), 30_000_000 // (B * Hk * Dh)))
        return dict(op="append", B=B, T=T, ctx=_log(rng, 1, 4096), Hk=Hk, Dh=Dh, page=page)
    if op in ("attend", "chunk"):
        g = rng.choice([1, 2, 3, 4, 6, 8])
        if op == "chunk":
            T = _log(rng, 17, 2048)
            B = rng.choice([1, 1, 2, 3])
            ctx = T + _log(rng, 1, 12000)
            B = max(1, min(B, 500_000_000 // (T * ctx * Hk * g)))
            while T * ctx * Hk * g * B > 500_000_000:
                ctx, T = max(ctx // 2, 2), max(T // 2, 1)
        else:
            B, T = _log(rng, 1, 64), rng.choice([1, 1, 1, 2, 3, 5, 8, 13])
            ctx = max(T, min(_log(rng, 1, 131072), 200_000_000 // (B * Hk * Dh)))
        return dict(op="attend", B=B, T=T, ctx=ctx, Hq=g * Hk, Hk=Hk, Dh=Dh, page=page, ragged=rng.random() < 0.6)
    return dict(op=op, slots=2 * _log(rng, 1, 32), ctx=_log(rng, 1, 5000), layers=rng.choice([1, 2, 3]),
                Hk=min(Hk, 8), Dh=Dh, page=page)


def _lengths(case, n):
    """Tokens cached for each of n sequences, from the case alone."""
    ctx, out = case["ctx"], []
    for b in range(n):
        if case.get("ragged"):
            out.append(max(case["T"], ctx * (1 + (b * 40503 + 7919) % 997) // 997))
        elif case["op"] in ("fork", "compact"):
            out.append(max(1, ctx - (b * 37) % max(1, ctx // 2)))
        elif case["op"] == "append":
            out.append(max(0, ctx - 1 - 13 * b) if b % 3 else ctx - ctx % case["page"])
        else:
            out.append(ctx)
    return out


# ------------------------------------------------------------------------------------ inputs
def _frequencies(case):
    """Inverse frequencies of the rotated pairs and the amplitude, scaled for long contexts."""
    rot, f = case["rot"], case["factor"]
    w = torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)
    if case["scaling"] == "linear":
        return w / f, 1.0
    if case["scaling"] == "ramp":        # keep fast pairs, stretch slow ones, blend between
        turns = 8192 * w / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return w / f * (1 - keep) + w * keep, 0.1 * math.log(f) + 1.0
    return w, 1.0


def _exponent(amax):
    """The block scale's exponent e: the least with amax <= 448 * 2^e, within its range."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8).clamp(E_MIN, E_MAX)
    return torch.where(amax > 0, e, torch.full_like(e, E_MIN))


def _two_to(e):
    """2^e in float32, exactly (e within the scale's range)."""
    return ((e + 127) << 23).to(torch.int32).view(torch.float32)


def _codes(x, e):
    """e4m3 codes (as bytes) of float32 x at scale 2^e; what is not finite becomes NaN."""
    y = x.clamp(-TOP, TOP) * _two_to(-e)
    y = torch.where(torch.isfinite(x), y, torch.full_like(y, float("nan")))
    return y.to(torch.float8_e4m3fn).view(torch.uint8)


def _values(codes, scale):
    return codes.view(torch.float8_e4m3fn).float() * scale


def _pool(g, layers, pages, heads, page, Dh):
    """A pool of pages with codes and scales of keys or values, some tokens outliers."""
    codes = torch.empty((layers, pages, heads, page, Dh), dtype=torch.uint8, device=DEV)
    scale = torch.empty((layers, pages, heads), dtype=torch.float32, device=DEV)
    step = max(1, (1 << 26) // (heads * page * Dh))
    for l in range(layers):
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = torch.randn((n, heads, page, Dh), generator=g, device=DEV)
            x = x * torch.where(torch.rand((n, heads, page, 1), generator=g, device=DEV) < 0.002, 6.0, 1.0)
            e = _exponent(x.abs().amax((2, 3)))
            codes[l, p:p + n] = _codes(x, e[..., None, None])
            scale[l, p:p + n] = _two_to(e)
    return codes, scale


def _cache(g, lengths, slots, layers, heads, page, Dh, spare, room):
    """Pools, page table (pages in random order, -1 behind the last), lengths and references."""
    need = [-(-n // page) for n in lengths]
    pages = sum(need) + spare
    M = max(need + [1]) + -(-room // page) + 2
    order = torch.randperm(pages, generator=g, device=DEV).tolist()
    rows, at = [], 0
    for n in need:
        rows.append(order[at:at + n] + [-1] * (M - n))
        at += n
    rows += [[-1] * M] * (slots - len(rows))
    refs = [0] * pages
    for p in order[:at]:
        refs[p] = 1
    k, ks = _pool(g, layers, pages, heads, page, Dh)
    v, vs = _pool(g, layers, pages, heads, page, Dh)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return dict(k=k, v=v, k_scale=ks, v_scale=vs, table=i32(rows), lens=i32(list(lengths) + [0] * (slots - len(lengths))),
                refs=i32(refs))


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    st = dict(case=case)
    if case["op"] == "rope":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        B, S, Hq, Hk, Dh = (case[n] for n in ("B", "S", "Hq", "Hk", "Dh"))
        x = torch.randn((B, S, Hq + Hk, Dh), generator=g, device=DEV).to(dt)     # a fused projection's rows
        q, k = x[:, :, :Hq].permute(0, 2, 1, 3), x[:, :, Hq:].permute(0, 2, 1, 3)
        if case["inverse"]:                                                    # gradients come dense, head by head
            q, k = q.contiguous(), k.contiguous()
        at = torch.randint(0, 1 + case["start"] // 8, (B, 1), generator=g, device=DEV)
        pos = (case["start"] - at + torch.arange(S, device=DEV)).to(torch.int64)
        inv_freq, amplitude = _frequencies(case)
        st.update(q=q, k=k, pos=pos, inv_freq=inv_freq.to(DEV), inv_freq_host=inv_freq, amplitude=amplitude)
        return st
    if case["op"] == "append":
        B, T, page = case["B"], case["T"], case["page"]
        start = _lengths(case, B)
        c = _cache(g, [s + T for s in start], B, 1, case["Hk"], page, case["Dh"], 3, 0)
        new = torch.randn((2, B, T, case["Hk"], case["Dh"]), generator=g, device=DEV)
        new = new * torch.where(torch.rand((2, B, T, 1, 1), generator=g, device=DEV) < 0.02, 12.0, 1.0)
        new = new.to(torch.bfloat16).permute(0, 1, 3, 2, 4)
        st.update(c, slots=torch.randperm(B, generator=g, device=DEV).to(torch.int32), k_new=new[0], v_new=new[1],
                  n_new=torch.full((B,), T, dtype=torch.int32, device=DEV))
        st["from"] = (st["lens"][st["slots"].long()] - T) // page * page        # first token of the first touched page
        return st
    if case["op"] == "attend":
        B, T = case["B"], case["T"]
        c = _cache(g, _lengths(case, B), B, 1, case["Hk"], case["page"], case["Dh"], 3, 0)
        q = 1.5 * torch.randn((B, T, case["Hq"], case["Dh"]), generator=g, device=DEV)
        st.update(c, slots=torch.randperm(B, generator=g, device=DEV).to(torch.int32),
                  q=q.to(torch.bfloat16).permute(0, 2, 1, 3), n_new=torch.full((B,), T, dtype=torch.int32, device=DEV))
        return st
    n = case["slots"]
    c = _cache(g, _lengths(case, n), n, case["layers"], case["Hk"], case["page"], case["Dh"], n, 1)
    order = torch.randperm(n, generator=g, device=DEV).to(torch.int32)
    half = n // 2
    st.update(c, ended=order[:half].contiguous(), kept=order[half:].contiguous(), every=order.contiguous(),
              zeros=torch.zeros((half,), dtype=torch.int32, device=DEV), ones=torch.ones((n,), dtype=torch.int32, device=DEV),
              table0=c["table"].clone(), lens0=c["lens"].clone(), refs0=c["refs"].clone())
    return st


# ------------------------------------------------------------------------------------ plain forms
def _plain_rotate(x, pos, w, amplitude, rot, layout, inverse):
    angle = pos.double()[:, None, :, None] * w                                 # far positions: 64 bits
    c, s = (amplitude * torch.cos(angle)).float(), (amplitude * torch.sin(angle)).float()
    if inverse:
        s = -s
    a = x[..., :rot].float()
    if layout == "half":
        x1, x2 = a[..., : rot // 2], a[..., rot // 2:]
        y = torch.cat((x1 * c - x2 * s, x1 * s + x2 * c), -1)
    else:
        x1, x2 = a[..., 0::2], a[..., 1::2]
        y = torch.stack((x1 * c - x2 * s, x1 * s + x2 * c), -1).flatten(-2)
    return torch.cat((y.to(x.dtype), x[..., rot:]), -1)


def _plain_write(codes, scale, pid, pos, start, x, B, T):
    """New tokens x [B, Hk, T, Dh] into the pages pid [B, N] that hold positions pos [B, N, page]."""
    N, page = pos.shape[1:]
    t = pos - start[:, None, None]                                             # which new token, if any
    is_new, is_old = (t >= 0) & (t < T), t < 0
    bi = torch.arange(B, device=DEV)[:, None, None]
    new = x.permute(0, 2, 1, 3)[bi, t.clamp(0, T - 1)].permute(0, 1, 3, 2, 4).float()     # [B, N, Hk, page, Dh]
    mask_new, mask_old = is_new[:, :, None, :, None], is_old[:, :, None, :, None]
    size = torch.where(mask_new & torch.isfinite(new), new.abs(), torch.zeros((), device=DEV))
    e = _exponent(size.amax((3, 4)))
    old_codes, old_scale = codes[pid], scale[pid]
    e_old = torch.frexp(old_scale)[1] - 1
    e = torch.where(is_old.any(2)[..., None], torch.maximum(e, e_old), e)
    old = old_codes.view(torch.float8_e4m3fn).float() * _two_to((e_old - e).clamp(-126, 0))[..., None, None]
    old = old.to(torch.float8_e4m3fn).view(torch.uint8)
    out = torch.where(mask_new, _codes(new, e[..., None, None]), torch.where(mask_old, old, old_codes))
    codes[pid] = out
    scale[pid] = _two_to(e)


def _plain_append(st):
    case = st["case"]
    B, T, page = case["B"], case["T"], case["page"]
    slots = st["slots"].long()
    start = st["lens"][slots].long() - T
    first, last = start // page, (start + T - 1) // page
    N = (T + page - 2) // page + 1
    at = torch.minimum(first[:, None] + torch.arange(N, device=DEV), last[:, None])   # a page named twice gets the same twice
    pid = st["table"][slots[:, None], at].long()
    pos = at[:, :, None] * page + torch.arange(page, device=DEV)
    _plain_write(st["k"][0], st["k_scale"][0], pid, pos, start, st["k_new"], B, T)
    _plain_write(st["v"][0], st["v_scale"][0], pid, pos, start, st["v_new"], B, T)
    return [_plain_read(st, n, slots, st["from"].long(), _read_length(case)) for n in ("k", "v")]


def _read_length(case):
    return case["page"] if case["T"] == 1 else case["T"] + case["page"]


def _plain_read(st, n, slots, start, length):
    """Positions start .. start + length - 1 of every sequence as bfloat16, zero behind its end."""
    page = st["case"]["page"]
    pos = start[:, None] + torch.arange(length, device=DEV)
    pid = st["table"][slots[:, None], (pos // page).clamp(max=st["table"].shape[1] - 1)].long().clamp(min=0)
    x = st[n][0][pid, :, pos % page].view(torch.float8_e4m3fn).float() * st[n + "_scale"][0][pid][..., None]
    x = torch.where((pos < st["lens"][slots].long()[:, None])[..., None, None], x, torch.zeros((), device=DEV))
    return x.to(torch.bfloat16).permute(0, 2, 1, 3).contiguous()


def _gathered(st, n, slots, length):
    """The sequences' values [B, Hk, length, Dh] in float32."""
    page = st["case"]["page"]
    N = -(-length // page)
    pid = st["table"][slots][:, :N].long().clamp(min=0)
    x = _values(st[n][0][pid], st[n + "_scale"][0][pid][..., None, None])
    return x.permute(0, 2, 1, 3, 4).flatten(2, 3)


def _plain_attend(st):
    case = st["case"]
    B, T, Hq, Hk, Dh = (case[n] for n in ("B", "T", "Hq", "Hk", "Dh"))
    slots = st["slots"].long()
    k, v = _gathered(st, "k", slots, case["ctx"]), _gathered(st, "v", slots, case["ctx"])
    lens = st["lens"][slots].long()
    q = st["q"].float().reshape(B, Hk, Hq // Hk * T, Dh) * Dh ** -0.5
    s = torch.matmul(q, k.transpose(2, 3)).view(B, Hk, Hq // Hk, T, k.shape[2])
    last = lens[:, None] - T + torch.arange(T, device=DEV)
    hidden = torch.arange(k.shape[2], device=DEV) > last[..., None]
    s = s.masked_fill_(hidden[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = (s - m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, Hk, -1, k.shape[2]), v).view(B, Hk, Hq // Hk, T, Dh) / z
    return o.reshape(B, Hq, T, Dh).to(torch.bfloat16), (m + z.log()).reshape(B, Hq, T)


def _plain_trim(st, slots, keep):
    page, slots = st["case"]["page"], slots.long()
    have = st["lens"][slots]
    kept = torch.minimum(have, keep)
    row = st["table"][slots]
    j = torch.arange(row.shape[1], device=DEV)
    gone = (j >= ((kept + page - 1) // page)[:, None]) & (j < ((have + page - 1) // page)[:, None])
    st["refs"].index_add_(0, row.clamp(min=0).flatten(), -gone.to(torch.int32).flatten())
    st["table"][slots] = torch.where(gone, torch.full_like(row, -1), row)
    st["lens"][slots] = kept


def _plain_fork(st, src, dst):
    page = st["case"]["page"]
    src, dst = src.long(), dst.long()
    row, n = st["table"][src], st["lens"][src]
    used = torch.arange(row.shape[1], device=DEV) < ((n + page - 1) // page)[:, None]
    st["table"][dst] = torch.where(used, row, torch.full_like(row, -1))
    st["lens"][dst] = n
    st["refs"].index_add_(0, row.clamp(min=0).flatten(), used.to(torch.int32).flatten())


def _plain_copy(st, src, dst):
    for n in ("k", "v", "k_scale", "v_scale"):
        st[n][:, dst] = st[n][:, src]


def _plain_reserve(st, slots, n_new, most):
    page, slots, P = st["case"]["page"], slots.long(), st["refs"].shape[0]
    n = st["lens"][slots].long()
    have = (n + page - 1) // page
    need = (n + n_new + page - 1) // page - have
    at = (have - 1).clamp(min=0)
    last = st["table"][slots, at].long().clamp(min=0)
    part = (n % page != 0) & (n_new > 0)
    order = torch.arange(P, device=DEV)
    i = torch.arange(len(slots), device=DEV)
    before = ((last[:, None] == last) & part[:, None] & part & (i < i[:, None])).sum(1)
    copied = part & (st["refs"][last] - before > 1)                            # the last one that shares a page keeps it
    free = torch.argsort(order + P * (st["refs"] > 0))                         # lowest free page first
    takes = need + copied
    first = takes.cumsum(0) - takes
    to = torch.where(copied, free[first.clamp(max=P - 1)], last)
    st["table"][slots, at] = torch.where(copied, to.to(torch.int32), st["table"][slots, at])
    one = copied.to(torch.int32)
    st["refs"].index_add_(0, last, -one)
    st["refs"].index_add_(0, to, one)
    _plain_copy(st, last, to)
    j = torch.arange(most, device=DEV)
    got = j < need[:, None]
    pid = free[(first + copied)[:, None].add(j).clamp(max=P - 1)]
    col = have[:, None] + j
    st["table"][slots[:, None], col] = torch.where(got, pid.to(torch.int32), st["table"][slots[:, None], col])
    st["refs"].index_add_(0, pid.flatten(), got.to(torch.int32).flatten())
    st["lens"][slots] += n_new


def _plain_compact(st):
    refs, P = st["refs"], st["refs"].shape[0]
    i = torch.arange(P, device=DEV)
    live = refs > 0
    n_live = live.sum()
    hole, mover = ~live & (i < n_live), live & (i >= n_live)
    holes, movers = torch.argsort(i + P * ~hole)[: P // 2], torch.argsort(i + P * ~mover)[: P // 2]
    used = torch.arange(P // 2, device=DEV) < hole.sum()
    src = torch.where(used, movers, 0)                                         # a pair not used copies page 0 onto itself
    dst = torch.where(used, holes, 0)
    src0 = torch.where(used[:1], movers[:1], 0)
    src = torch.where((dst == 0) & hole[0], src0, src)                         # unless page 0 is filled itself
    _plain_copy(st, src, dst)
    to = i.index_put((src,), dst).to(torch.int32)
    st["table"].copy_(torch.where(st["table"] >= 0, to[st["table"].clamp(min=0).long()], st["table"]))
    moved = refs.index_put((dst,), refs[src])
    refs.copy_(torch.where(i < n_live, moved, torch.zeros_like(moved)))


def _kept(st):
    """What the calls on pages leave: the pools as the values that their codes are, and the books."""
    f8 = torch.float8_e4m3fn
    return [st["k"].view(f8), st["v"].view(f8), st["k_scale"], st["v_scale"], st["table"], st["lens"], st["refs"]]


def _own_cache(st, ra):
    if "cache" not in st:                  # the handle that a program makes once
        st["cache"] = ra.KVCache(*(st[n] for n in ("k", "v", "k_scale", "v_scale", "table", "lens", "refs")))
    return st["cache"]


def run(state):
    st, case = state, state["case"]
    op = case["op"]
    if own:
        from long_context_exact_fwd_b200 import ring_attn as ra
        if op == "rope":
            if "plan" not in st:
                st["plan"] = ra.rope_plan(st["inv_freq_host"], layout=case["layout"], amplitude=st["amplitude"])
            return ra.rope(st["q"], st["plan"], k=st["k"], pos=st["pos"], inverse=case["inverse"])
        cache = _own_cache(st, ra)
        if op == "append":
            ra.cache_append(cache, 0, st["slots"], st["n_new"], st["k_new"], st["v_new"])
            return ra.cache_read(cache, 0, st["slots"], _read_length(case), start=st["from"])
        if op == "attend":
            return ra.cache_attend(cache, 0, st["slots"], st["n_new"], st["q"])
    elif op == "rope":
        w, a = st["inv_freq"], st["amplitude"]
        return [_plain_rotate(st[n], st["pos"], w, a, case["rot"], case["layout"], case["inverse"]) for n in ("q", "k")]
    elif op == "append":
        return _plain_append(st)
    elif op == "attend":
        return _plain_attend(st)
    for n in ("table", "lens", "refs"):    # the books before these calls, so that a pass can follow a pass
        st[n].copy_(st[n + "0"])
    if own:
        ra.cache_trim(cache, st["ended"], st["zeros"])
        if op == "fork":
            ra.cache_fork(cache, st["kept"], st["ended"])
            ra.cache_reserve(cache, st["every"], st["ones"])
        else:
            ra.cache_compact(cache)
    else:
        _plain_trim(st, st["ended"], st["zeros"])
        if op == "fork":
            _plain_fork(st, st["kept"], st["ended"])
            _plain_reserve(st, st["every"], st["ones"], 1)
        else:
            _plain_compact(st)
    return _kept(st)


# ------------------------------------------------------------------------------------ work
def work(case):
    op = case["op"]
    if op == "rope":
        n = case["B"] * case["S"] * (case["Hq"] + case["Hk"])
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": 2 * n * case["Dh"] * size + 8 * case["B"] * case["S"], "flops": 3 * n * case["rot"]}
    Hk, Dh, page = case["Hk"], case["Dh"], case["page"]
    if op == "append":                     # new rows in, codes out; then the codes in, rows out
        n = case["B"] * case["T"] * Hk * Dh * 2
        back = case["B"] * _read_length(case) * Hk * Dh * 2
        return {"bytes": 2 * n + n + back + 2 * back, "flops": 4 * n}
    if op == "attend":
        T, g = case["T"], case["Hq"] // Hk
        lens = _lengths(case, case["B"])
        pairs = sum(T * n - T * (T - 1) // 2 for n in lens) * Hk * g
        rows = case["B"] * case["Hq"] * T
        held = sum(lens) * Hk * 2 * Dh + sum(-(-n // page) for n in lens) * (Hk * 8 + 4)
        return {"bytes": held + rows * (4 * Dh + 4), "flops": 4 * Dh * pairs}
    lens = _lengths(case, case["slots"])
    page_bytes = case["layers"] * Hk * (2 * page * Dh + 8)
    books = 8 * (sum(-(-n // page) for n in lens) + case["slots"])
    half = case["slots"] // 2
    if op == "fork":                       # one page copied for each fork whose last page is partly filled
        part = sum(n % page != 0 for n in lens) / len(lens)
        return {"bytes": 2 * page_bytes * max(1.0, part * half) + books, "flops": 0}
    live = sum(-(-n // page) for n in lens) * (len(lens) - half) / len(lens)
    total = sum(-(-n // page) for n in lens) + case["slots"]
    return {"bytes": 2 * page_bytes * max(1.0, live * (1 - live / total)) + books, "flops": 0}


# ------------------------------------------------------------------------------------ exact
def _e4m3(y):
    """Nearest e4m3 value of float64 y (ties to even), as float64; NaN stays."""
    x = torch.frexp(y.abs())[1].clamp(min=-5).long()                           # y < 2^x; 3 bits behind the leading one
    step = ((x - 4 + 1023) << 52).view(torch.float64)
    return torch.round(y / step) * step


def _exact_block_exponent(a):
    e = E_MIN
    if a > 0:
        e = math.frexp(a / 448.0)
        e = e[1] - 1 if e[0] == 0.5 else e[1]
    return min(max(e, E_MIN), E_MAX)


def _exact_append(st, case):
    """Page by page from the definition; the pools as prepared, this file's state not written."""
    B, T, page, Hk, Dh = (case[n] for n in ("B", "T", "page", "Hk", "Dh"))
    length = _read_length(case)
    slots, lens, table, frm = (st[n].tolist() for n in ("slots", "lens", "table", "from"))
    outs = []
    for n, new in (("k", st["k_new"]), ("v", st["v_new"])):
        out = torch.zeros((B, Hk, length, Dh), dtype=torch.float64, device=DEV)
        exps = torch.log2(st[n + "_scale"][0].double()).round().cpu()
        for b, slot in enumerate(slots):
            p0 = lens[slot] - T
            x = new[b].double()
            lo = frm[b] // page
            for j in range(lo, (lens[slot] - 1) // page + 1):
                pid, a, z = table[slot][j], max(j * page, p0), min((j + 1) * page, lens[slot])
                part = x[:, a - p0:z - p0]
                tops = torch.where(torch.isfinite(part), part.abs(), 0.0).amax((1, 2)).tolist()
                for h in range(Hk):
                    e, e0 = _exact_block_exponent(tops[h]), int(exps[pid, h])
                    n_old = a - j * page
                    e = max(e, e0) if n_old else e
                    at = j * page - frm[b]
                    if n_old:
                        old = st[n][0][pid, h, :n_old].view(torch.float8_e4m3fn).double()
                        end = min(n_old, length - at)
                        out[b, h, at:at + end] = (_e4m3(old * 2.0 ** (e0 - e)) * 2.0 ** e)[:end]
                    end = min(z, frm[b] + length)
                    if end > a:
                        out[b, h, a - frm[b]:end - frm[b]] = (_e4m3(part[h] * 2.0 ** -e) * 2.0 ** e)[: end - a]
        outs.append(out)
    return outs


def _exact_attend(st, case):
    B, T, Hq, Hk, Dh, page = (case[n] for n in ("B", "T", "Hq", "Hk", "Dh", "page"))
    g = Hq // Hk
    o = torch.zeros((B, Hq, T, Dh), dtype=torch.float64, device=DEV)
    lse = torch.zeros((B, Hq, T), dtype=torch.float64, device=DEV)
    slots, lens = st["slots"].tolist(), st["lens"].tolist()
    for b, slot in enumerate(slots):
        n = lens[slot]
        pid = st["table"][slot, : -(-n // page)].long()
        for h in range(Hk):
            kv = [(st[x][0][pid, h].view(torch.float8_e4m3fn).double() * st[x + "_scale"][0][pid, h].double()[:, None, None])
                  .reshape(-1, Dh)[:n] for x in ("k", "v")]
            for t0 in range(0, T, 512):
                t1 = min(T, t0 + 512)
                q = st["q"][b, h * g:(h + 1) * g, t0:t1].double().reshape(-1, Dh)
                s = (q @ kv[0].T).view(g, t1 - t0, n) / math.sqrt(Dh)
                t = torch.arange(t0, t1, device=DEV)
                s.masked_fill_(torch.arange(n, device=DEV) > (n - T + t)[:, None], -math.inf)
                l = torch.logsumexp(s, -1)
                o[b, h * g:(h + 1) * g, t0:t1] = torch.exp(s - l[..., None]) @ kv[1]
                lse[b, h * g:(h + 1) * g, t0:t1] = l
    return o, lse


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rope":
        outs = []
        for x in (st["q"], st["k"]):
            y = x.double().clone()
            turn = torch.polar(torch.full((), float(st["amplitude"]), dtype=torch.float64, device=DEV),
                               st["pos"].double()[:, None, :, None] * st["inv_freq"] * (-1 if case["inverse"] else 1))
            r = case["rot"]
            a, b = (y[..., : r // 2], y[..., r // 2:r]) if case["layout"] == "half" else (y[..., 0:r:2], y[..., 1:r:2])
            z = torch.complex(a.contiguous(), b.contiguous()) * turn
            a.copy_(z.real)
            b.copy_(z.imag)
            outs.append(y)
        return outs
    if case["op"] == "append":
        if case["B"] * case["Hk"] * (case["T"] // case["page"] + 2) > 12000:
            return None
        return _exact_append(st, case)
    if case["op"] == "attend":
        return _exact_attend(st, case)
    return None                            # copies and whole numbers only
