"""Release of tables that hold ids outside the pool: they stay off the free stack."""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from recsys_decoupled_link_b200 import lime, lime_kv
from test_gpu_kv import i32, offsets, pool_case
from test_gpu_kv_serving import rows

pytestmark = pytest.mark.gpu


def run_release(lens, keep, table, free, cap, n_blocks, bs=16):
    B = len(lens)
    dims = lime_kv.make_kv_dims(1, 1, 16, bs, n_blocks, table.shape[1], "bf16")
    ws = lime_kv.KvWorkspace(dims, B, 0)
    tab, st = i32(table), torch.full((cap,), -9, dtype=torch.int32, device="cuda")
    st[:len(free)] = i32(free)
    out, nfo = i32(np.full(B, -7)), i32([-7])
    lime_kv.lime_kv_release(dims, i32(lens), None if keep is None else i32(keep), tab, st, i32([len(free)]), out, nfo,
                            ws)
    return out.cpu().numpy(), int(nfo), tab.cpu().numpy(), st.cpu().numpy(), lime.lime_get_status(ws)


@pytest.mark.parametrize("B", [1, 3, 70, 1025, 3000])
@pytest.mark.parametrize("how", ["all", "some"])
@pytest.mark.parametrize("old_hi", [100, 900])
def test_release_drops_ids_outside_the_pool(B, how, old_hi):
    rng = np.random.default_rng(B)
    lens, _, table, free, n_blocks = pool_case(rng, B, 16, old_hi, 30)
    lens[0] = max(lens[0], 1)
    bad = (rng.random(table.shape) < 0.3) & (np.arange(table.shape[1]) < -(-lens // 16)[:, None])
    bad[0, 0] = True
    table = np.where(bad, rng.choice([-1, -5, n_blocks, n_blocks + 9, 2 ** 31 - 1, -2 ** 31], table.shape), table)
    keep = None if how == "all" else np.where(np.arange(B) == 0, 0, rng.integers(-3, old_hi, B))
    out, nfo, tab, st, flags = run_release(lens, keep, table, free, n_blocks, n_blocks)
    w_lens, w_stack, w_table = K.release(lens, keep, table, free, len(free), 16, n_blocks)
    assert flags == lime_kv.LIME_FLAG_BAD_BLOCK
    np.testing.assert_array_equal(out, w_lens)
    np.testing.assert_array_equal(tab, w_table)
    assert nfo == len(w_stack)
    np.testing.assert_array_equal(st[:nfo], w_stack)
    assert (st[nfo:] == -9).all()


def test_release_of_bad_ids_and_past_the_stack():
    # five good ids of eight, room for three
    table = np.array([[4, -1, 99, 6], [8, 7, 3, -1]])
    out, nfo, tab, st, flags = run_release([64, 64], None, table, [0], 4, 8)
    assert flags == lime_kv.LIME_FLAG_BAD_BLOCK and nfo == 4
    assert st.tolist() == [0, 4, 6, 7] and (tab == -1).all() and (out == 0).all()


def test_a_bad_id_on_the_stack_leaves_the_cache_with_its_first_owner():
    dims = lime_kv.make_kv_dims(2, 2, 32, 16, 8, 4, "bf16")
    cache = lime_kv.HistoryCache(dims, 2)
    assert cache.free.tolist() == [7, 6, 5, 4, 3, 2, 1, 0]
    cache.free[6] = 99                                               # the second block to be taken: block 1 is lost
    x = rows(40, 2, 2, 32, seed=1)
    slots = cache.append(x[:, 0], x[:, 1], offsets([40, 0]))
    assert cache.status() == lime_kv.LIME_FLAG_BAD_BLOCK
    assert (slots[16:32] == -1).all() and (slots[:16] >= 0).all() and (slots[32:] >= 0).all()
    cache.release()
    assert cache.status() == lime_kv.LIME_FLAG_BAD_BLOCK
    n = int(cache.n_free)
    assert n == 7 and sorted(cache.free[:n].tolist()) == [0, 2, 3, 4, 5, 6, 7]
    slots = cache.append(x[:, 0], x[:, 1], offsets([0, 40]))         # every block it hands out is whole again
    assert (slots >= 0).all() and cache.status() == 0
