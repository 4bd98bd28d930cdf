"""Cases of the paged 8-bit history cache: its block tables, its append and its attention.

A serving program keeps each user's history as key and value rows in a pool of
fixed-size blocks.  A row is held as int8 codes; every (block, head) has one
fp32 scale for its keys and one for its values, so a row stands for
code * scale.  Three operators work on it:

  reserve    gives the blocks that new rows need to the requests, in order,
             from a stack of free blocks, and lists the slot of every new row;
  append     quantises new key and value rows into their slots.  A block's
             scale is the largest magnitude it has been given over 127; rows
             already in the block are requantised when it grows;
  attention  softmax(q k / sqrt(dh)) v of a request's query rows (its links,
             or its newest rows) over its cached rows, with grouped heads.

``run`` computes them in plain torch where ``own`` is false and with the
library's kernels where it is true.  Cache layout: codes [blocks, Hkv, block,
dh], scales [blocks, Hkv, 2] (keys, values), block table [B, columns].
"""
import math

import torch

own = False

INT8_MAX = 127.0


# ------------------------------------------------------------------- cases

def listed():
    return [
        # one event arrives for each of 256 users: the call of every step, where only latency counts
        dict(name="reserve one row each", op="reserve", B=256, old="lognormal", old_lo=32, old_hi=12000,
             new="uniform", new_lo=1, new_hi=1, block=64, short=False, lens_seed=1),
        # 256 users' whole histories are loaded: the ragged workload's lengths
        dict(name="reserve ragged histories", op="reserve", B=256, old="uniform", old_lo=0, old_hi=0,
             new="lognormal", new_lo=32, new_hi=12000, block=64, short=False, lens_seed=2),
        # a day's trickle over many users, some without any event, from a pool that runs out
        dict(name="reserve many users", op="reserve", B=16384, old="uniform", old_lo=0, old_hi=700,
             new="uniform", new_lo=0, new_hi=8, block=16, short=True, lens_seed=3),
        # one event for each of 64 users: the smallest append
        dict(name="append one row each", op="append", B=64, Hkv=4, dh=32, old="uniform", old_lo=0, old_hi=1023,
             new="uniform", new_lo=1, new_hi=1, block=64, dtype="bf16", lens_seed=4),
        # the ragged workload's histories quantised on their first load
        dict(name="append ragged histories", op="append", B=256, Hkv=4, dh=32, old="uniform", old_lo=0, old_hi=0,
             new="lognormal", new_lo=32, new_hi=12000, block=64, dtype="bf16", lens_seed=2),
        # fp32 rows of odd lengths behind partly filled blocks
        dict(name="append fp32 odd lengths", op="append", B=40, Hkv=8, dh=64, old="uniform", old_lo=0, old_hi=301,
             new="uniform", new_lo=0, new_hi=701, block=32, dtype="f32", lens_seed=5),
        # the tiny workload: four users' links over short histories, one head, fp32
        dict(name="attention tiny fp32", op="attention", B=4, q=32, ragged_q=False, Hq=1, Hkv=1, dh=64, n="uniform",
             n_lo=256, n_hi=256, causal=False, block=16, dtype="f32", lens_seed=6),
        # the standard workload's links over their histories
        dict(name="attention links", op="attention", B=64, q=32, ragged_q=False, Hq=4, Hkv=4, dh=32, n="uniform",
             n_lo=1024, n_hi=1024, causal=False, block=64, dtype="bf16", lens_seed=7),
        # the ragged workload with 64 links: exponentials weigh most
        dict(name="attention ragged 64 links", op="attention", B=256, q=64, ragged_q=False, Hq=4, Hkv=4, dh=32,
             n="lognormal", n_lo=32, n_hi=12000, causal=False, block=64, dtype="bf16", lens_seed=2),
        # the long workload: 16,384 rows for each of 32 users
        dict(name="attention links long", op="attention", B=32, q=32, ragged_q=False, Hq=4, Hkv=4, dh=32, n="uniform",
             n_lo=16384, n_hi=16384, causal=False, block=64, dtype="bf16", lens_seed=8),
        # one token each with grouped heads over long ragged caches: bound by reading the cache
        dict(name="attention single tokens", op="attention", B=64, q=1, ragged_q=False, Hq=32, Hkv=8, dh=128,
             n="uniform", n_lo=1, n_hi=16384, causal=True, block=32, dtype="bf16", lens_seed=9),
        # freshly appended chunks of up to 128 rows, each row seeing the rows up to itself
        dict(name="attention causal chunks", op="attention", B=24, q=128, ragged_q=True, Hq=8, Hkv=2, dh=64,
             n="uniform", n_lo=0, n_hi=4097, causal=True, block=16, dtype="bf16", lens_seed=10),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["reserve", "append", "attention", "attention"])
    block = rng.choice([16, 32, 64, 128])
    seed = rng.randrange(1 << 30)
    if op == "reserve":
        B = _log_int(rng, 1, 16384)
        most = max(1, min(12000, 500000 // B))
        return dict(op=op, B=B, old="uniform", old_lo=0, old_hi=_log_int(rng, 1, most), new="uniform",
                    new_lo=rng.choice([0, 1]), new_hi=_log_int(rng, 1, most), block=block,
                    short=B >= 8 and rng.random() < 0.3, lens_seed=seed)
    Hkv, dh = rng.choice([(1, 64), (2, 64), (4, 32), (8, 16), (8, 64), (4, 128), (8, 128), (1, 32), (3, 32)])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    width = Hkv * dh
    if op == "append":
        B = _log_int(rng, 1, 512)
        most = max(1, min(12000, (1 << 25) // (B * width)))
        return dict(op=op, B=B, Hkv=Hkv, dh=dh, old="uniform", old_lo=0, old_hi=_log_int(rng, 1, most), new="uniform",
                    new_lo=rng.choice([0, 1]), new_hi=_log_int(rng, 1, most), block=block, dtype=dtype,
                    lens_seed=seed)
    B = _log_int(rng, 1, 256)
    G = rng.choice([1, 1, 2, 4, 8])
    q = rng.choice([1, 1, 16, 32, 64, rng.randrange(2, 128)])
    # rows of scores stay below the largest listed case's, and so do cached bytes
    most = max(16, min(16384, (1 << 28) // (B * width), (1 << 28) // (B * Hkv * G * q)))
    hi = _log_int(rng, 16, most)
    return dict(op=op, B=B, q=q, ragged_q=q > 1 and rng.random() < 0.4, Hq=Hkv * G, Hkv=Hkv, dh=dh, n="uniform",
                n_lo=rng.choice([0, 1, hi // 2, hi]), n_hi=hi, causal=rng.random() < 0.4, block=block, dtype=dtype,
                lens_seed=seed)


# ------------------------------------------------------------------ inputs

def _lengths(B, how, lo, hi, seed):
    """B lengths in [lo, hi] on the host; lengths belong to the case, not to the inputs' seed."""
    g = torch.Generator().manual_seed(seed)
    if how == "lognormal":  # median 1,500
        return torch.exp(math.log(1500.0) + torch.randn(B, generator=g)).round().long().clamp(lo, hi)
    return torch.randint(lo, hi + 1, (B,), generator=g)


def _old_new(case):
    old = _lengths(case["B"], case["old"], case["old_lo"], case["old_hi"], case["lens_seed"])
    new = _lengths(case["B"], case["new"], case["new_lo"], case["new_hi"], case["lens_seed"] + 1)
    new[0] = max(1, int(new[0]))          # a call has one new row at least
    return old, new


def _queries(case):
    """Query rows and cached rows of each request.  A request's newest rows are its queries in a causal case."""
    n = _lengths(case["B"], case["n"], case["n_lo"], case["n_hi"], case["lens_seed"])
    q = torch.full_like(n, case["q"])
    if case["ragged_q"]:
        q = _lengths(case["B"], "uniform", 0, case["q"], case["lens_seed"] + 1)
        q[0] = max(1, int(q[0]))          # a call has one query row at least
    return q, n


def _offsets(counts):
    return torch.cat([torch.zeros(1, dtype=torch.int64), counts.long().cumsum(0)])


def _blocks(n, block):
    return (n + block - 1) // block


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _table(counts, columns, order):
    """Block table [B, columns]: counts[u] blocks of `order` for request u, -1 behind them; and the blocks left."""
    col = torch.arange(columns, device=order.device)
    first = counts.cumsum(0) - counts
    at = first[:, None] + col
    live = col < counts[:, None]
    table = torch.where(live, order[at.clamp(max=order.numel() - 1)], -1).to(torch.int32)
    return table, order[int(counts.sum()):].to(torch.int32).contiguous()


def _random_cache(blocks, Hkv, block, dh, g, dev):
    """Codes and scales of rows whose values are about N(0, 1)."""
    codes = [torch.randn(blocks, Hkv, block, dh, generator=g, device=dev).mul_(33.0).round_().clamp_(-127, 127)
             .to(torch.int8) for _ in range(2)]
    scale = torch.exp(0.25 * torch.randn(blocks, Hkv, 2, generator=g, device=dev)) / 32.0
    return codes[0], codes[1], scale


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    op, B, bs = case["op"], case["B"], case["block"]
    s = dict(case=case, B=B, block=bs)
    if op == "attention":
        q, n = _queries(case)
        total_q = int(q.sum())
        Hq, Hkv, dh, dt = case["Hq"], case["Hkv"], case["dh"], _dtype(case)
        nb = _blocks(n, bs)
        columns = max(1, int(nb.max()))
        blocks = int(nb.sum()) + 1
        order = torch.randperm(blocks, generator=g, device=dev)
        table, _ = _table(nb.to(dev), columns, order)
        k, v, scale = _random_cache(blocks, Hkv, bs, dh, g, dev)
        s.update(k=k, v=v, scale=scale, table=table, lens=n.to(dev, torch.int32), q_offsets=_offsets(q).to(dev),
                 total_q=total_q, max_q=int(q.max()), sm_scale=1.0 / math.sqrt(dh), causal=case["causal"],
                 Q=torch.randn(total_q, Hq, dh, generator=g, device=dev).to(dt),
                 O=torch.empty(total_q, Hq, dh, dtype=dt, device=dev),
                 lse=torch.empty(total_q, Hq, dtype=torch.float32, device=dev))
    else:
        old, new = _old_new(case)
        total = int(new.sum())
        before, after = _blocks(old, bs), _blocks(old + new, bs)
        columns = max(1, int(after.max()))
        need, held = int((after - before).sum()), int(before.sum())
        free = need - need // 3 if case.get("short") else need + 7
        blocks = held + free + 64            # 64 blocks belong to requests outside this call
        order = torch.randperm(blocks, generator=g, device=dev)[:held + free]
        table, stack = _table(before.to(dev), columns, order)
        s.update(total=total, blocks=blocks, columns=columns)
        if op == "reserve":
            stack = torch.cat([stack, stack.new_zeros(1)])[:max(1, free)]
            s.update(lens=old.to(dev, torch.int32), new_offsets=_offsets(new).to(dev), table=table, free=stack,
                     n_free=torch.full((1,), free, dtype=torch.int32, device=dev),
                     lens_out=torch.empty(B, dtype=torch.int32, device=dev),
                     n_free_out=torch.empty(1, dtype=torch.int32, device=dev),
                     slots=torch.empty(total, dtype=torch.int64, device=dev))
        else:
            Hkv, dh, dt = case["Hkv"], case["dh"], _dtype(case)
            # the table once the new rows have their blocks, and the slot of every new row
            table, _ = _table(after.to(dev), columns, order)
            u = torch.repeat_interleave(torch.arange(B), new).to(dev)
            pos = old.to(dev)[u] + torch.arange(total, device=dev) - _offsets(new).to(dev)[u]
            k, v, scale = _random_cache(blocks, Hkv, bs, dh, g, dev)
            # one projection leaves keys and values side by side; heads differ in size, a few rows stand out
            kv = torch.randn(total, 2, Hkv, dh, generator=g, device=dev)
            kv *= torch.exp(0.5 * torch.randn(2, Hkv, 1, generator=g, device=dev))
            kv *= 1.0 + 4.0 * (torch.rand(total, 1, 1, 1, generator=g, device=dev) < 0.01)
            s.update(kv=kv.to(dt), new_offsets=_offsets(new).to(dev), k=k, v=v, scale=scale,
                     slots=table[u, pos // bs].long() * bs + pos % bs,
                     k_values=torch.empty(k.shape, dtype=dt, device=dev),
                     v_values=torch.empty(v.shape, dtype=dt, device=dev))
    if own:
        from recsys_decoupled_link_b200 import lime_kv
        if op == "attention":
            dims = lime_kv.make_kv_dims(Hq, Hkv, dh, bs, blocks, columns, dt)
            ws = lime_kv.KvWorkspace(dims, B, total_q)
        elif op == "reserve":
            dims = lime_kv.make_kv_dims(1, 1, 64, bs, blocks, columns, torch.bfloat16)
            ws = lime_kv.KvWorkspace(dims, B, 0)
        else:
            dims = lime_kv.make_kv_dims(Hkv, Hkv, dh, bs, blocks, columns, dt)
            ws = lime_kv.KvWorkspace(dims, B, 0)
        s.update(dims=dims, ws=ws)
    return s


# ------------------------------------------------------------- plain forms

def _reserve_plain(s):
    B, bs, total, columns = s["B"], s["block"], s["total"], s["columns"]
    dev = s["lens"].device
    lens, off, n_free = s["lens"].long(), s["new_offsets"], s["n_free"].long()
    n = off[1:] - off[:-1]
    before, after = _blocks(lens, bs), _blocks(lens + n, bs)
    fits = after <= columns
    need = torch.where(fits, after - before, 0)
    end = need.cumsum(0)
    ok = fits & ((need == 0) | (end <= n_free))
    base = end - need
    taken = torch.where(ok & (need > 0), end, 0).amax()
    u = torch.repeat_interleave(torch.arange(B, device=dev), n, output_size=total)
    pos = lens[u] + torch.arange(total, device=dev) - off[u]
    col = (pos // bs).clamp(max=columns - 1)
    held = s["table"][u, col].long()
    rank = (base[u] + pos // bs - before[u]).clamp(min=0)
    fresh = s["free"][(n_free - 1 - rank).clamp(min=0)].long()
    block = torch.where(pos // bs >= before[u], fresh, held)
    good = ok[u]
    s["table"][u, col] = torch.where(good, block, held).to(torch.int32)
    return {"table": s["table"], "lens": torch.where(ok, lens + n, lens).to(torch.int32),
            "n_free": (n_free - taken).to(torch.int32), "slots": torch.where(good, block * bs + pos % bs, -1)}


def _append_plain(s):
    bs, slots = s["block"], s["slots"]
    block, row = slots // bs, slots % bs
    blocks, dev = s["k"].shape[0], slots.device
    # a request's first new row: its block is the only one that may hold older rows
    head = slots[s["new_offsets"][:-1].clamp(max=slots.numel() - 1)]
    older = torch.arange(bs, device=dev)[:, None] < (head % bs)[:, None, None, None]
    head = head // bs
    touched = torch.zeros(blocks, 1, dtype=torch.bool, device=dev)
    touched[block] = True
    started = torch.zeros(blocks + 1, 1, dtype=torch.bool, device=dev)
    started[torch.where(row == 0, block, blocks)] = True               # a block's first row starts it anew
    for side, cache in ((0, s["k"]), (1, s["v"])):
        x = s["kv"][:, side].float()
        scale = s["scale"][..., side]
        top = torch.zeros_like(scale)
        top.scatter_reduce_(0, block[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
        was = torch.where(started[:blocks], 0.0, scale)
        now = torch.where(touched, torch.maximum(was, (top.double() / INT8_MAX).float()), scale)
        # a quotient next to a border decides the code: in 64 bits
        a, b, codes = was[head].double()[..., None, None], now[head].double()[..., None, None], cache[head].double()
        cache[head] = torch.where((b > a) & older, (codes * a / b).round_(), codes).to(torch.int8)
        by = now.double()[block][..., None]
        code = torch.where(by > 0, x.double() / by, 0.0).round_().clamp_(-127, 127)
        cache[block, :, row] = code.to(torch.int8)
        scale.copy_(now)


def _attention_plain(s):
    c, B, bs = s["case"], s["B"], s["block"]
    Hq, Hkv, dh, max_q = c["Hq"], c["Hkv"], c["dh"], s["max_q"]
    G, dev, dt = Hq // Hkv, s["Q"].device, s["Q"].dtype
    table, lens, off = s["table"].clamp(min=0).long(), s["lens"].long(), s["q_offsets"]
    N = table.shape[1] * bs
    count = off[1:] - off[:-1]
    # rows of all requests padded to the longest: [B, Hkv, keys, dh] and [B, Hkv, G * max_q, dh]
    keys = (s["k"][table].float() * s["scale"][table][..., 0, None, None]).transpose(1, 2).reshape(B, Hkv, N, dh)
    u = torch.repeat_interleave(torch.arange(B, device=dev), count, output_size=s["total_q"])
    i = torch.arange(s["total_q"], device=dev) - off[u]
    q = torch.zeros(B, max_q, Hq, dh, device=dev)
    q[u, i] = s["Q"].float()
    q = q.view(B, max_q, Hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * max_q, dh)
    scores = torch.matmul(q, keys.transpose(-1, -2)).mul_(s["sm_scale"])
    del keys
    limit = lens[:, None].expand(B, max_q)
    if s["causal"]:
        limit = lens[:, None] - count[:, None] + torch.arange(max_q, device=dev) + 1
    hidden = torch.arange(N, device=dev) >= limit[..., None]                       # [B, max_q, keys]
    scores.view(B, Hkv, G, max_q, N).masked_fill_(hidden[:, None, None], -math.inf)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    values = (s["v"][table].float() * s["scale"][table][..., 1, None, None]).transpose(1, 2).reshape(B, Hkv, N, dh)
    out = torch.matmul(p, values) / torch.where(total > 0, total, 1.0)
    lse = (top + total.log()).view(B, Hkv, G, max_q)                               # log 0 = -inf: a row without keys
    out = out.view(B, Hkv, G, max_q, dh).permute(0, 3, 1, 2, 4).reshape(B, max_q, Hq, dh)
    return {"out": out[u, i].to(dt), "lse": lse.permute(0, 3, 1, 2).reshape(B, max_q, Hq)[u, i]}


# --------------------------------------------------------------------- run

def _values(s):
    """What the pool's codes stand for, in the rows' type."""
    torch.mul(s["k"], s["scale"][..., 0, None, None], out=s["k_values"])
    torch.mul(s["v"], s["scale"][..., 1, None, None], out=s["v_values"])
    return {"k": s["k_values"], "v": s["v_values"], "scale": s["scale"]}


def run(s):
    op = s["case"]["op"]
    if op == "reserve":
        if own:
            from recsys_decoupled_link_b200 import lime_kv
            lime_kv.lime_kv_reserve(s["dims"], s["lens"], s["new_offsets"], s["table"], s["free"], s["n_free"],
                                    s["lens_out"], s["n_free_out"], s["slots"], s["ws"])
            return {"table": s["table"], "lens": s["lens_out"], "n_free": s["n_free_out"], "slots": s["slots"]}
        return _reserve_plain(s)
    if op == "append":
        if own:
            from recsys_decoupled_link_b200 import lime_kv
            lime_kv.lime_kv_append(s["dims"], s["kv"][:, 0], s["kv"][:, 1], s["slots"], s["k"], s["v"], s["scale"],
                                   s["ws"])
        else:
            _append_plain(s)
        return _values(s)
    if own:
        from recsys_decoupled_link_b200 import lime_kv
        lime_kv.lime_kv_attention(s["dims"], s["Q"], s["q_offsets"], s["table"], s["lens"], s["k"], s["v"], s["scale"],
                                  s["O"], s["lse"], s["ws"], sm_scale=s["sm_scale"], causal=s["causal"])
        return {"out": s["O"], "lse": s["lse"]}
    return _attention_plain(s)


def work(case):
    """Bytes and operations of one pass: each input read once, each output written once."""
    op, B, bs = case["op"], case["B"], case["block"]
    if op == "reserve":
        old, new = _old_new(case)
        fresh = int((_blocks(old + new, bs) - _blocks(old, bs)).sum())
        if case["short"]:
            fresh -= fresh // 3
        # lengths and offsets in, lengths out, a block read and written for each fresh one, the partly
        # filled block of each request, a slot for each row
        return {"bytes": float(B * (4 + 8 + 4) + 8 * fresh + 4 * B + 8 * int(new.sum())), "flops": 0.0}
    if op == "append":
        old, new = _old_new(case)
        es, width = (2 if case["dtype"] == "bf16" else 4), case["Hkv"] * case["dh"]
        total = int(new.sum())
        pool = (int(_blocks(old + new, bs).sum()) + 71) * bs * width
        # rows and slots in, codes out; then the pool's codes in and the values they stand for out
        return {"bytes": float(total * (2 * width * (es + 1) + 8) + 2 * pool * (1 + es)), "flops": 0.0}
    q, n = _queries(case)
    es, dh, Hq, Hkv = (2 if case["dtype"] == "bf16" else 4), case["dh"], case["Hq"], case["Hkv"]
    if case["causal"]:  # row i of a request sees n - q + i + 1 rows, none where that is negative
        first = (n - q + 1).clamp(min=0)
        seen = torch.where(q > 0, (first + n) * (n - first + 1) // 2, 0)
    else:
        seen = q * n
    live = torch.where(q > 0, n, 0)
    rows = int(q.sum()) * Hq
    bytes_ = rows * (2 * dh * es + 4) + int(live.sum()) * 2 * Hkv * dh + int(_blocks(live, bs).sum()) * (8 * Hkv + 4)
    return {"bytes": float(bytes_ + 12 * B), "flops": float(4 * dh * Hq * int(seen.sum()))}


# ------------------------------------------------------------------- exact

def exact(case, seed):
    """The operators by their definitions, one request at a time, in 64 bits."""
    op, bs = case["op"], case["block"]
    if op == "reserve":
        return None                       # whole numbers
    s = prepare(case, seed)
    if op == "append":
        scale = s["scale"].double()
        out = {}
        for side, name in ((0, "k"), (1, "v")):
            value = s[name].double()                                              # codes, then what they stand for
            start = 0
            for n_old, n in zip(*(t.tolist() for t in _old_new(case))):
                at, x = s["slots"][start:start + n], s["kv"][start:start + n, side].double()
                start += n
                if n == 0:
                    continue
                lead, count = n_old % bs, _blocks(n_old % bs + n, bs)
                rows = x.new_zeros(count * bs, *x.shape[1:])
                rows[lead:lead + n] = x
                rows = rows.view(count, bs, *x.shape[1:])
                ids = at[(torch.arange(count, device=x.device) * bs - lead).clamp(min=0)] // bs
                by = (rows.abs().amax((1, 3)) / 127.0).float().double()           # held in 32 bits: [blocks, Hkv]
                if lead > 0:
                    had = scale[ids[0], :, side]
                    by[0] = torch.maximum(by[0], had)
                    kept = torch.round(value[ids[0], :, :lead] * had[:, None, None] / by[0][:, None, None])
                    value[ids[0], :, :lead] = kept
                per = by[:, None, :, None]
                coded = torch.where(per > 0, torch.round(rows / per), 0.0).clamp(-127, 127)
                value[at // bs, :, at % bs] = coded.reshape(-1, *x.shape[1:])[lead:lead + n]
                scale[ids, :, side] = by
            out[name] = value * scale[..., side, None, None]
        out["scale"] = scale
        return out
    q_counts, n_counts = _queries(case)
    G = case["Hq"] // case["Hkv"]
    out, lse = [], []
    start = 0
    for b, (m, n) in enumerate(zip(q_counts.tolist(), n_counts.tolist())):
        q = s["Q"][start:start + m].double().transpose(0, 1)                      # [Hq, m, dh]
        start += m
        if m == 0:
            continue
        ids = s["table"][b, :_blocks(n, bs)].long()
        k = (s["k"][ids].double() * s["scale"][ids][..., 0, None, None].double()).transpose(0, 1)
        v = (s["v"][ids].double() * s["scale"][ids][..., 1, None, None].double()).transpose(0, 1)
        k = k.reshape(case["Hkv"], -1, case["dh"])[:, :n].repeat_interleave(G, 0)
        v = v.reshape(case["Hkv"], -1, case["dh"])[:, :n].repeat_interleave(G, 0)
        x = torch.einsum("hqd,hkd->hqk", q, k) / math.sqrt(case["dh"])
        if case["causal"]:
            seen = torch.ones(m, n, dtype=torch.bool, device=x.device).tril(n - m)
            x = x.masked_fill(~seen, -math.inf)
        z = torch.logsumexp(x, -1) if n else torch.full(x.shape[:2], -math.inf, dtype=x.dtype, device=x.device)
        w = torch.where(torch.isinf(z)[..., None], torch.zeros_like(x), torch.exp(x - z[..., None]))
        out.append(torch.einsum("hqk,hkd->qhd", w, v))
        lse.append(z.transpose(0, 1))
    return {"out": torch.cat(out), "lse": torch.cat(lse)}
