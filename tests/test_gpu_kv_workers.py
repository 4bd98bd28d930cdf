"""Attention calls large enough for workers of one warp, and calls just below them.

The kernel gives each warp pairs of its own where ceil(rows * G / R) * Hkv, all
requests' query rows packed together, reaches 8 for every SM; below that four
warps share a pair's tiles.  (G query heads to a key head; R rows of a pair: 32
for bf16 heads of up to 64 with more than 16 rows a head and request, else 16.)
Both kinds, every head size, type, row tile, and blocks smaller and larger than a
softmax step, against the 64-bit attention, within test_gpu_kv.py's bounds.
"""
import numpy as np
import pytest
import torch

import kv_dense
from recsys_decoupled_link_b200 import lime, lime_kv
from test_gpu_kv import DT, assert_near, f64, offsets

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def packed_pairs(counts, Hq, Hkv, dh, dtype):
    total, G = int(np.sum(counts)), Hq // Hkv
    R = 32 if dtype == "bf16" and dh <= 64 and -(-total // len(counts)) * G > 16 else 16
    return -(-total * G // R) * Hkv


class Call:
    def __init__(self, counts, lens, Hq, Hkv, dh, bs, dtype, causal=False, seed=0, strided=False, hook=None):
        self.counts, self.lens, self.dtype, self.bs, self.causal = counts, lens, dtype, bs, causal
        n = int(np.sum(counts))
        self.table, self.k, self.v, self.scale = kv_dense.make_pool(lens, Hkv, dh, bs, seed, "cuda")
        g = torch.Generator(device="cuda").manual_seed(seed + 1)
        q = torch.randn(n, Hq + int(strided), dh, generator=g, device="cuda").to(DT[dtype])
        self.q = q[:, :Hq]
        if hook:
            hook(self)
        self.dims = lime_kv.make_kv_dims(Hq, Hkv, dh, bs, self.k.shape[0], self.table.shape[1], dtype)
        self.ws = lime_kv.KvWorkspace(self.dims, len(lens), n)
        self.off = offsets(counts)
        self.n_rows = torch.tensor(np.asarray(lens), dtype=torch.int32, device="cuda")

    def run(self, with_lse=True):
        O = torch.full(self.q.shape, 7.0, dtype=self.q.dtype, device="cuda")
        lse = torch.full(self.q.shape[:2], 7.0, device="cuda") if with_lse else None
        lime_kv.lime_kv_attention(self.dims, self.q, self.off, self.table, self.n_rows, self.k, self.v, self.scale, O,
                                  lse, self.ws, causal=self.causal)
        return O, lse

    def check(self, want_flags=0):
        O, lse = self.run()
        assert lime.lime_get_status(self.ws) == want_flags
        O2, _ = self.run(with_lse=False)                             # again: the same bits
        assert torch.equal(O2.view(torch.uint8), O.view(torch.uint8))
        assert lime.lime_get_status(self.ws) == want_flags
        dh = self.q.shape[2]
        ref = kv_dense.attention(self.q, self.counts, self.table, self.lens, self.k, self.v, self.scale, self.bs,
                                 dh ** -0.5, self.causal)
        assert_near(O, lse, *ref, max(1, int(np.max(self.lens))), dh, self.dtype)
        return O, lse


def ragged(B, seed, long=9000):
    """Lengths of up to 70 rows, none, one and a full block among them, and one that many workers share."""
    lens = np.random.default_rng(seed).integers(0, 70, B)
    lens[[0, 1, 2, 3, B - 1]] = [0, 1, 64, long, 0]
    return lens


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [16, 32, 64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("above", [True, False])
def test_single_tokens_on_both_sides_of_the_border(sms, dtype, dh, bs, above):
    B = sms * 4 if above else sms * 4 - 4
    counts = np.ones(B, dtype=int)
    assert (packed_pairs(counts, 32, 8, dh, dtype) >= sms * 8) == above
    Call(counts, ragged(B, dh + bs), 32, 8, dh, bs, dtype, causal=bs == 16, seed=bs, strided=bs == 32).check()


@pytest.mark.parametrize("dh", [16, 32, 64])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("G", [1, 3])
@pytest.mark.parametrize("causal", [False, True])
def test_row_tiles_of_32(sms, dh, bs, G, causal):
    B, Hkv = sms, 8
    counts = np.random.default_rng(bs).integers(16 if G == 1 else 5, 64 if G == 1 else 23, B)
    counts[:4] = [1, 0, 90, 64]
    counts[4] = max(0, 32 * sms // G + 40 - int(counts.sum()) + int(counts[4]))
    assert packed_pairs(counts, Hkv * G, Hkv, dh, "bf16") >= sms * 8 and -(-counts.sum() // B) * G > 16
    Call(counts, ragged(B, dh, long=1500), Hkv * G, Hkv, dh, bs, "bf16", causal=causal, seed=bs).check()


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("f32", 16), ("f32", 32), ("f32", 64), ("f32", 128)])
@pytest.mark.parametrize("bs", [16, 64])
@pytest.mark.parametrize("causal", [False, True])
def test_many_row_tiles_of_16(sms, dtype, dh, bs, causal):
    B, Hkv = 40, 8
    counts = np.random.default_rng(bs).integers(20, 100, B)
    counts[:3] = [0, 1, 300]
    counts[3] = max(0, 16 * sms + 40 - int(counts.sum()) + int(counts[3]))
    assert packed_pairs(counts, Hkv, Hkv, dh, dtype) >= sms * 8
    Call(counts, ragged(B, dh, long=2000), Hkv, Hkv, dh, bs, dtype, causal=causal, seed=bs).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,Hq,Hkv", [(32, 8, 2), (64, 5, 5), (128, 16, 1)])
@pytest.mark.parametrize("causal", [False, True])
def test_more_requests_than_a_block_sums(sms, dtype, dh, Hq, Hkv, causal):
    B = 5000                                                         # a kernel of its own adds their weights up
    counts = np.random.default_rng(dh).integers(0, 4, B)
    assert packed_pairs(counts, Hq, Hkv, dh, dtype) >= sms * 8
    Call(counts, ragged(B, dh, long=3000), Hq, Hkv, dh, 16, dtype, causal=causal).check()


def many_tokens(dtype, dh=64, bs=16, B=640, **kw):
    return Call(np.ones(B, dtype=int), ragged(B, 5), 32, 8, dh, bs, dtype, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_bad_table_entries_hide_their_rows(dtype):
    def hook(c):
        c.table[3, 7:500:3] = -1                                     # inside the long request
        c.table[2, 0], c.table[1, 0] = 10 ** 6, 2 ** 31 - 1          # a block of several, a request's only one
    O, lse = many_tokens(dtype, hook=hook).check(want_flags=lime_kv.LIME_FLAG_BAD_BLOCK)
    assert (O[1] == 0).all() and torch.isneginf(lse[1]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_garbage_behind_the_last_row_is_not_used(dtype):
    c = many_tokens(dtype, bs=64)
    clean, lse = c.run()
    last = torch.tensor(np.maximum(c.lens - 1, 0) // 64, device="cuda")
    ids = c.table[torch.arange(len(c.lens), device="cuda"), last].long().clamp(min=0)
    behind = torch.arange(64, device="cuda") >= torch.tensor(c.lens, device="cuda")[:, None] - 64 * last[:, None]
    for cache in (c.k, c.v):
        cache[ids] = torch.where(behind[:, None, :, None] & (c.n_rows > 0)[:, None, None, None], 127, cache[ids])
    c.table[torch.arange(len(c.lens), device="cuda"), -(-c.n_rows.long() // 64)] = 2 ** 31 - 1
    again, lse2 = c.run()
    assert torch.equal(again, clean) and torch.equal(lse2, lse) and lime.lime_get_status(c.ws) == 0


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_in_one_row_stays_there(dtype):
    c = many_tokens(dtype)
    clean, _ = c.run()
    ref = kv_dense.attention(c.q, c.counts, c.table, c.lens, c.k, c.v, c.scale, c.bs, 64 ** -0.5, False)
    rows = [(7, 1), (3, 30), (200, 0)]
    assert all(c.lens[u] > 0 for u, _ in rows)
    for (u, h), x in zip(rows, (float("nan"), float("inf"), float("nan"))):
        c.q[u, h, 3] = x
    bad, lse = c.run()
    assert all(torch.isnan(bad[u, h]).all() for u, h in rows) and not torch.isnan(clean).any()
    # the other rows of its pair (the query heads of its key head) bring their references up to date when
    # it asks for that, so they are summed in other steps: within the bounds; all others bit by bit
    others, pair = np.ones(bad.shape[:2], dtype=bool), np.zeros(bad.shape[:2], dtype=bool)
    for u, h in rows:
        pair[u, h // 4 * 4:h // 4 * 4 + 4] = True
        others[u, h // 4 * 4:h // 4 * 4 + 4] = False
    for u, h in rows:
        pair[u, h] = False
    on = torch.tensor(others, device="cuda")
    assert torch.equal(bad[on], clean[on])
    on = torch.tensor(pair, device="cuda")
    assert_near(bad[on], lse[on], *(r[pair] for r in ref), int(np.max(c.lens)), 64, dtype)


def test_bad_lengths_and_offsets_stay_in_bounds():
    def whole(c):
        c.scale.nan_to_num_(0.01)
        c.table.clamp_(min=0)
    c = many_tokens("bf16", hook=whole)
    c.n_rows[10], c.n_rows[11] = -1, 10 ** 6
    c.run()
    assert lime.lime_get_status(c.ws) == lime.LIME_FLAG_BAD_OFFSETS
    c.n_rows[10:12] = 20
    c.off = offsets([3] + [1] * 637 + [900, -300])
    c.run()
    assert lime.lime_get_status(c.ws) == lime.LIME_FLAG_BAD_OFFSETS
    c.off = offsets([1] * 600 + [0] * 40)                            # rows of nobody are left as they were
    O, lse = c.run()
    assert lime.lime_get_status(c.ws) == lime.LIME_FLAG_BAD_OFFSETS
    assert (O[600:] == 7.0).all() and (lse[600:] == 7.0).all() and (O[4:600] != 7.0).any()


@pytest.mark.parametrize("B", [640, 2500])
def test_captured_and_replayed(B):
    c = many_tokens("bf16", B=B)
    want, want_lse = c.run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        O, lse = c.run()
        O2, lse2 = c.run()                                           # two calls share the workspace
    for _ in range(3):
        O.zero_(), O2.zero_(), lse.zero_(), lse2.zero_()
        graph.replay()
        assert torch.equal(O, want) and torch.equal(O2, want) and torch.equal(lse, want_lse) \
            and torch.equal(lse2, want_lse)
    assert lime.lime_get_status(c.ws) == 0
