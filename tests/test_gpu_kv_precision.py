"""fp32 attention is as exact as the same sums in fp32.

Against the 64-bit attention, relative to the outputs' size (root mean square):
at most 16 fp32 half steps (1e-6), or where torch's own fp32 sums are further
off than that, 1.5 times as far as they are.
"""
import numpy as np
import pytest
import torch

import kv_dense
from recsys_decoupled_link_b200 import lime, lime_kv
from test_gpu_kv import offsets

pytestmark = pytest.mark.gpu


def plain_fp32(q, m, n, table, k, v, scale, bs):
    """Requests of m query rows and n cached rows each, elementary fp32 products throughout."""
    B, Hkv, dh = len(table), k.shape[1], k.shape[3]
    G = q.shape[1] // Hkv
    ids = table[:, :-(-n // bs)].long()
    flat = lambda c, side: (c[ids].float() * scale[ids][..., side, None, None]).transpose(1, 2) \
        .reshape(B, Hkv, -1, dh)[:, :, :n]
    x = q.view(B, m, Hkv, G, dh).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * m, dh)
    s = x @ flat(k, 0).transpose(2, 3) * dh ** -0.5
    p = torch.exp(s - s.amax(-1, keepdim=True))
    out = (p @ flat(v, 1)) / p.sum(-1, keepdim=True)
    return out.view(B, Hkv, G, m, dh).permute(0, 3, 1, 2, 4).reshape(B * m, -1, dh)


@pytest.mark.parametrize("n", [16, 256, 1024, 4096, 16384])
@pytest.mark.parametrize("dh,Hq,Hkv,m", [(16, 4, 4, 1), (32, 4, 4, 1), (32, 4, 4, 32), (64, 8, 2, 1), (64, 1, 1, 32),
                                         (128, 8, 2, 1), (128, 2, 2, 32)])
@pytest.mark.parametrize("seed", [0, 1])
def test_fp32_attention_is_as_exact_as_fp32_sums(n, dh, Hq, Hkv, m, seed):
    assert not torch.backends.cuda.matmul.allow_tf32
    B, bs = 16, 64
    lens, counts = [n] * B, [m] * B
    table, k, v, scale = kv_dense.make_pool(lens, Hkv, dh, bs, seed, "cuda")
    q = torch.randn(B * m, Hq, dh, generator=torch.Generator(device="cuda").manual_seed(seed + 5), device="cuda")
    dims = lime_kv.make_kv_dims(Hq, Hkv, dh, bs, k.shape[0], table.shape[1], "f32")
    ws, O = lime_kv.KvWorkspace(dims, B, B * m), torch.empty_like(q)
    lime_kv.lime_kv_attention(dims, q, offsets(counts), table, torch.full((B,), n, dtype=torch.int32, device="cuda"),
                              k, v, scale, O, None, ws)
    assert lime.lime_get_status(ws) == 0
    ref = kv_dense.attention(q, counts, table, lens, k, v, scale, bs, dh ** -0.5, False)[0]
    off = lambda x: np.linalg.norm(x.double().cpu().numpy() - ref) / np.linalg.norm(ref)
    ours, plain = off(O), off(plain_fp32(q, m, n, table, k, v, scale, bs))
    assert ours <= max(1e-6, 1.5 * plain), (ours, plain)
