"""Attention over the history cache in 64-bit torch, a request at a time, for sizes that the loops of
oracle.kv_oracle would take minutes over.  Pinned to it in test_kv_host_dense.py."""
import torch


def make_pool(lens, Hkv, dh, bs, seed, device, spare=2):
    """Table, codes and scales of requests with `lens` rows, in shuffled blocks; spare blocks hold NaN scales."""
    g = torch.Generator(device=device).manual_seed(seed)
    lens = torch.as_tensor(lens, dtype=torch.int64, device=device)
    nb = (lens + bs - 1) // bs
    blocks, cols = int(nb.sum()) + spare, max(1, int(nb.max())) + 1
    ids = torch.randperm(blocks, generator=g, device=device)
    col = torch.arange(cols, device=device)
    at = (nb.cumsum(0) - nb)[:, None] + col
    table = torch.where(col < nb[:, None], ids[at.clamp(max=blocks - 1)], -1).to(torch.int32)
    codes = [torch.randn(blocks, Hkv, bs, dh, generator=g, device=device).mul_(33).round_().clamp_(-127, 127)
             .to(torch.int8) for _ in range(2)]
    scale = torch.exp(0.4 * torch.randn(blocks, Hkv, 2, generator=g, device=device)) / 32
    scale[ids[int(nb.sum()):]] = float("nan")
    return table, codes[0], codes[1], scale


def attention(q, counts, table, lens, k, v, scale, bs, sm_scale, causal):
    """As oracle.kv_oracle.attention: (O, lse, A, S, V) as numpy arrays."""
    n_rows, Hq, dh = q.shape
    Hkv = k.shape[1]
    G, dev = Hq // Hkv, q.device
    new = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)
    O, A, V = (new(n_rows, Hq, dh) for _ in range(3))
    S, lse = new(n_rows, Hq), new(n_rows, Hq) - float("inf")
    at = 0
    for u, (m, n) in enumerate(zip(counts, lens)):
        m, n = int(m), int(n)
        rows, at = slice(at, at + m), at + m
        if m == 0 or n == 0:
            continue
        ids = table[u, :-(-n // bs)].long()
        held = (ids >= 0) & (ids < k.shape[0])
        ids = torch.where(held, ids, 0)
        held = held.repeat_interleave(bs)[:n]
        flat = lambda c, side: (c[ids].double() * scale[ids][..., side].double().nan_to_num()[..., None, None]) \
            .transpose(0, 1).reshape(Hkv, -1, dh)[:, :n]
        keys, values = flat(k, 0), flat(v, 1)
        x = q[rows].double().view(m, Hkv, G, dh).permute(1, 2, 0, 3).reshape(Hkv, G * m, dh)
        limit = torch.full((m,), n, device=dev)
        if causal:
            limit = (n - m + 1 + torch.arange(m, device=dev)).clamp(min=0)
        seen = ((torch.arange(n, device=dev) < limit[:, None]) & held).repeat(G, 1)     # [G * m, n]
        s = (x @ keys.transpose(1, 2) * sm_scale).masked_fill(~seen, -float("inf"))
        z = torch.logsumexp(s, -1)
        w = torch.exp(s - torch.where(z.isinf(), 0.0, z)[..., None])
        back = lambda t: t.reshape(Hkv, G, m, -1).permute(2, 0, 1, 3).reshape(m, Hq, -1)
        O[rows], A[rows] = back(w @ values), back(w @ values.abs())
        lse[rows] = back(z)[..., 0]
        big = (x.abs() @ keys.abs().transpose(1, 2) * abs(sm_scale)).masked_fill(~seen, 0.0).amax(-1)
        S[rows] = back(big)[..., 0]
        most = torch.cummax(values.abs() * held[:, None], 1).values                     # [Hkv, n, dh]
        top = most[:, (limit - 1).clamp(min=0)] * (limit > 0)[:, None]                  # [Hkv, m, dh]
        V[rows] = back(top[:, None].expand(-1, G, -1, -1))
    return tuple(t.cpu().numpy() for t in (O, lse, A, S, V))
