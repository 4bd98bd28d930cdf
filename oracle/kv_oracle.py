"""fp64 CPU oracle of the paged 8-bit history cache (test infrastructure only).

Plain loops over requests, written from the definitions in include/lime_kv.h;
it shares no code with the GPU path.
"""
from __future__ import annotations

import numpy as np


def blocks_of(n: int, bs: int) -> int:
    return -(-n // bs)


def reserve(lens, new, table, free, n_free, bs):
    """Returns (lens_out, n_free_out, table_out, slots, refused)."""
    lens, table = list(map(int, lens)), np.array(table, dtype=np.int64)
    out, slots, refused = [], [], []
    used = want = 0
    for u, (n, m) in enumerate(zip(lens, map(int, new))):
        held, after = blocks_of(n, bs), blocks_of(n + m, bs)
        need = after - held
        fits = after <= table.shape[1]
        want += need if fits else 0
        if not fits or (need > 0 and want > n_free):
            out.append(n)
            slots += [-1] * m
            refused.append(u)
            continue
        for c in range(held, after):
            table[u, c] = free[n_free - 1 - used]
            used += 1
        out.append(n + m)
        slots += [int(table[u, j // bs]) * bs + j % bs for j in range(n, n + m)]
    return np.array(out), n_free - used, table, np.array(slots, dtype=np.int64), refused


def release(lens, keep, table, free, n_free, bs, n_blocks=None):
    """Returns (lens_out, free_out (the stack's live part), table_out).  With n_blocks, table
    entries outside the pool are dropped."""
    table, stack, out = np.array(table), list(free[:n_free]), []
    for u, n in enumerate(map(int, lens)):
        k = 0 if keep is None else min(max(int(keep[u]), 0), n)
        for c in range(blocks_of(k, bs), blocks_of(n, bs)):
            if n_blocks is None or 0 <= table[u, c] < n_blocks:
                stack.append(int(table[u, c]))
            table[u, c] = -1
        out.append(k)
    return np.array(out), np.array(stack, dtype=np.int64), table


def append(x, slots, codes, scale, bs):
    """x fp64 [n, Hkv, dh] of one side; codes [blocks, Hkv, bs, dh], scale fp64
    holding fp32 values [blocks, Hkv].  Returns new (codes, scale)."""
    codes, scale = codes.astype(np.float64), scale.copy()
    t, n = 0, len(slots)
    while t < n:
        slot = int(slots[t])
        if slot < 0 or slot >= codes.shape[0] * bs:
            t += 1
            continue
        m = 1
        while slot % bs + m < bs and t + m < n and slots[t + m] == slot + m:
            m += 1
        blk, r = divmod(slot, bs)
        for h in range(x.shape[1]):
            rows = x[t:t + m, h]
            finite = np.where(np.isfinite(rows), rows, 0.0)
            had = float(scale[blk, h]) if r else 0.0
            s = max(had, float(np.float32(np.abs(finite).max() / 127.0)))
            if s > had and r:
                codes[blk, h, :r] = np.rint(codes[blk, h, :r] * had / s)
            q = np.clip(np.rint(finite / s), -127, 127) if s > 0 else np.zeros_like(rows)
            q = np.where(np.isposinf(rows), 127.0, np.where(np.isneginf(rows), -127.0, q))
            codes[blk, h, r:r + m] = q if s > 0 else np.zeros_like(rows)
            scale[blk, h] = s
        t += m
    return codes.astype(np.int8), scale


def attention(q, q_counts, table, lens, k, v, scale, bs, sm_scale, causal):
    """q fp64 [n, Hq, dh]; codes and fp64 scale [blocks, Hkv, 2].

    Returns (O, lse, A, S, V): A = sum_j w_j |v_j|, V = max_j |v_j| and S = max_j
    sum_d |q_d k_jd| sm_scale, the magnitudes an error bound of O and lse needs."""
    n_rows, Hq, dh = q.shape
    G = Hq // k.shape[1]
    O, lse = np.zeros((n_rows, Hq, dh)), np.full((n_rows, Hq), -np.inf)
    A, S, V = np.zeros((n_rows, Hq, dh)), np.zeros((n_rows, Hq)), np.zeros((n_rows, Hq, dh))
    i = 0
    for u, m in enumerate(map(int, q_counts)):
        n = int(lens[u])
        for r in range(m):
            seen = n - m + r + 1 if causal else n
            js = [j for j in range(max(0, seen)) if 0 <= table[u][j // bs] < k.shape[0]]
            if js:
                blk, row = np.array([table[u][j // bs] for j in js]), np.array(js) % bs
                for h in range(Hq):
                    kk = k[blk, h // G, row].astype(np.float64) * scale[blk, h // G, 0][:, None]
                    vv = v[blk, h // G, row].astype(np.float64) * scale[blk, h // G, 1][:, None]
                    s = kk @ q[i, h] * sm_scale
                    top = s.max()
                    w = np.exp(s - top)
                    lse[i, h] = top + np.log(w.sum())
                    w /= w.sum()
                    O[i, h], A[i, h], V[i, h] = w @ vv, w @ np.abs(vv), np.abs(vv).max(0)
                    S[i, h] = (np.abs(kk) @ np.abs(q[i, h])).max() * abs(sm_scale)
            i += 1
    return O, lse, A, S, V
