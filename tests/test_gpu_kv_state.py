"""A captured call of HistoryCache works on the cache as it stands at each replay."""
import pytest
import torch

from recsys_decoupled_link_b200 import lime_kv
from test_gpu_kv import i32, offsets
from test_gpu_kv_serving import capture, rows

pytestmark = pytest.mark.gpu


@pytest.fixture
def dims():
    return lime_kv.make_kv_dims(4, 2, 32, 16, 60, 12, "bf16")


@pytest.mark.parametrize("causal", [False, True])
def test_captured_attention_follows_the_cache(dims, causal):
    cache = lime_kv.HistoryCache(dims, 3, max_q=6)
    q, off = rows(6, 4, 32, seed=1), offsets([2, 2, 2])
    graph, out = capture(lambda: cache.attend(q, off, causal=causal))
    lens = [0, 0, 0]
    for step, counts in enumerate(([20, 1, 40], [1, 1, 1], [0, 30, 5], [17, 0, 0], [2, 2, 2])):
        x = rows(sum(counts), 2, 2, 32, seed=10 + step)
        cache.append(x[:, 0], x[:, 1], offsets(counts))
        lens = [a + b for a, b in zip(lens, counts)]
        assert cache.lens.tolist() == lens
        out.zero_()
        graph.replay()
        assert torch.equal(out, cache.attend(q, off, causal=causal))
    cache.release(i32([3, 100, 0]))
    graph.replay()
    assert cache.lens.tolist() == [3, min(100, lens[1]), 0]
    assert torch.equal(out, cache.attend(q, off, causal=causal)) and (out[4:] == 0).all() and (out[:4] != 0).any()
    assert cache.status() == 0


@pytest.mark.parametrize("shorten", [False, True])
def test_captured_steps_advance_the_cache(dims, shorten):
    # replays of a captured step against the same steps made eagerly
    cache, eager = lime_kv.HistoryCache(dims, 3, max_q=6), lime_kv.HistoryCache(dims, 3)
    x, q, off = rows(3, 2, 2, 32, seed=2), rows(3, 4, 32, seed=3), offsets([1, 1, 1])
    keep = i32([64, 20, 1000])
    first = rows(50, 2, 2, 32, seed=4)
    for c in (cache, eager):
        c.append(first[:, 0], first[:, 1], offsets([20, 30, 0]))

    def step(c):
        slots = c.append(x[:, 0], x[:, 1], off)
        out = c.attend(q, off, causal=True)
        if shorten:
            c.release(keep)
        return slots, out

    graph, (slots, out) = capture(lambda: step(cache))
    assert cache.lens.tolist() == [20, 30, 0]                        # nothing has run yet
    for i in range(21):
        x.copy_(rows(3, 2, 2, 32, seed=100 + i))
        q.copy_(rows(3, 4, 32, seed=200 + i))
        graph.replay()
        want_slots, want = step(eager)
        assert torch.equal(slots, want_slots) and torch.equal(out, want)
        assert torch.equal(cache.lens, eager.lens) and torch.equal(cache.n_free, eager.n_free)
        assert torch.equal(cache.table, eager.table)
    assert cache.lens.tolist() == [41, 20 if shorten else 51, 21]
    want_slots, want = step(eager)                                   # and an eager step after the replays
    got_slots, got = step(cache)
    assert torch.equal(got_slots, want_slots) and torch.equal(got, want)
    assert cache.status() == eager.status() == 0


def test_cache_state_stays_where_it_is(dims):
    cache = lime_kv.HistoryCache(dims, 3)
    lens, n_free = cache.lens, cache.n_free
    x = rows(7, 2, 2, 32, seed=5)
    for n in range(1, 4):
        cache.append(x[:, 0], x[:, 1], offsets([7, 0, 0]))
        assert cache.lens is lens and cache.n_free is n_free and lens.tolist() == [7 * n, 0, 0]
    cache.release()
    assert cache.lens is lens and cache.n_free is n_free and lens.tolist() == [0, 0, 0] and int(n_free) == 60
