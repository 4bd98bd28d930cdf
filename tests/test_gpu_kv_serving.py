"""The history cache as a serving loop holds it: captured calls beside eager ones."""
import pytest
import torch

from recsys_decoupled_link_b200 import lime_kv
from test_gpu_kv import offsets

pytestmark = pytest.mark.gpu


def rows(*shape, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


def capture(fn):
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = fn()
    return graph, out


@pytest.mark.parametrize("dh,n_rows", [(32, 40), (128, 2000)])
def test_captured_attention_outlives_a_larger_eager_one(dh, n_rows):
    # the graph's workspace stays the cache's, whatever is called, allocated and filled in between
    dims = lime_kv.make_kv_dims(4, 2, dh, 16, 300, 130, "bf16")
    cache = lime_kv.HistoryCache(dims, 2, max_q=8)
    x = rows(2 * n_rows, 2, 2, dh, seed=1)
    cache.append(x[:, 0], x[:, 1], offsets([n_rows, n_rows]))
    q, off = rows(8, 4, dh, seed=2), offsets([4, 4])
    want = cache.attend(q, off).clone()
    graph, out = capture(lambda: cache.attend(q, off))
    big = rows(4000, 4, dh, seed=3)
    cache.attend(big, offsets([2000, 2000]))
    fillers = [torch.full((n,), 7, dtype=torch.uint8, device="cuda") for n in (1 << 12, 1 << 20, 48 << 20, 48 << 20)]
    out.zero_()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(bool((f == 7).all()) for f in fillers)
    assert cache.status() == 0 and torch.equal(cache.attend(q, off), want)


def test_a_single_row_of_any_pitch():
    # the only row of a wider buffer whose width is no multiple of 16 bytes
    dims = lime_kv.make_kv_dims(2, 2, 32, 16, 4, 2, "bf16")
    outs = []
    for pitch in (64, 65, 3):
        cache = lime_kv.HistoryCache(dims, 1, max_q=1)
        at = lambda seed: rows(64, seed=seed).as_strided((1, 2, 32), (pitch, 32, 1))
        cache.append(at(1), at(2), offsets([1]))
        outs.append(cache.attend(at(3), offsets([1])))
        assert cache.status() == 0
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]) and bool((outs[0] != 0).any())


def test_a_step_without_new_rows():
    dims = lime_kv.make_kv_dims(4, 2, 32, 16, 10, 4, "bf16")
    cache = lime_kv.HistoryCache(dims, 2, max_q=4)
    x = rows(5, 2, 2, 32, seed=1)
    cache.append(x[:, 0], x[:, 1], offsets([5, 0]))
    none = torch.zeros(0, 2, 2, 32, dtype=torch.bfloat16)
    assert cache.append(none[:, 0].cuda(), none[:, 1].cuda(), offsets([0, 0])).numel() == 0
    assert cache.lens.tolist() == [5, 0] and int(cache.n_free) == 9 and cache.status() == 0
    out = cache.attend(rows(0, 4, 32, seed=2), offsets([0, 0]))
    assert out.shape == (0, 4, 32) and cache.status() == 0
