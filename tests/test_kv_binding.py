"""CPU-only checks of the history cache's binding: what it passes on, keeps and
refuses.  The library's entry points are replaced by recorders, and host tensors
stand for the current device's."""
import pytest
import torch

from recsys_decoupled_link_b200 import build as lime_build


class Recorder:
    """Stands for the library: answers the size queries, records every other call."""

    def __init__(self, lib):
        self.lib, self.calls = lib, []

    def __getattr__(self, name):
        if name.endswith("_bytes"):
            return getattr(self.lib, name)

        def call(*args):
            self.calls.append((name, args))
            return 0
        return call

    def names(self):
        return [n for n, _ in self.calls]


@pytest.fixture
def kv(monkeypatch):
    lime_build.build()
    from recsys_decoupled_link_b200 import lime_kv as m
    monkeypatch.setattr(m, "_lib", Recorder(m._lib))
    monkeypatch.setattr(m, "_device", lambda: -1)                    # a host tensor's get_device()
    monkeypatch.setattr(m, "_raw_stream", lambda stream, dev: 0)
    return m


@pytest.fixture
def capturing(monkeypatch):
    state = {"on": False}
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: state["on"])
    return state


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def i64(*shape):
    return torch.zeros(*shape, dtype=torch.int64)


# ------------------------------------------------------------ history cache

def make_cache(kv, B=2, **kw):
    return kv.HistoryCache(kv.make_kv_dims(4, 2, 32, 16, 10, 4, "bf16"), B, device="cpu", **kw)


def rows(n, heads):
    return torch.zeros(n, heads, 32, dtype=torch.bfloat16)


def test_workspace_of_one_query_row_serves_any_number(kv):
    for B in (1, 2048, 2049, 100_000):
        for dims in (kv.make_kv_dims(4, 2, 32, 16, 10, 4, "bf16"), kv.make_kv_dims(8, 8, 128, 64, 10, 4, "f32")):
            one = kv.lime_kv_workspace_bytes(dims, B, 1)
            assert one > 0
            for n in (2, 1000, 2 ** 31 - 1):
                assert kv.lime_kv_workspace_bytes(dims, B, n) == one


@pytest.mark.parametrize("max_q", [0, 4])
def test_cache_keeps_one_workspace(kv, capturing, max_q):
    # what a captured call writes to must outlive every later call, whatever its size
    cache = make_cache(kv, max_q=max_q)
    ws, address = cache.ws, cache.ws.address
    for n in (1, 4, 5, 300, 7):
        cache.attend(rows(n, 4), i64(3))
        assert cache.ws is ws and cache.ws.address == address == cache.ws.buf.data_ptr()
    assert cache.max_q == 300
    assert [n for n in kv._lib.names() if n != "lime_kv_attention"] == ["lime_kv_workspace_init"]
    name, args = kv._lib.calls[-1]
    assert args[-3] == address and args[-2] == ws.nbytes


def test_cache_in_a_capture(kv, capturing):
    cache = make_cache(kv, max_q=6)
    capturing["on"] = True
    cache.attend(rows(6, 4), i64(3))
    with pytest.raises(ValueError, match="max_q"):
        cache.attend(rows(7, 4), i64(3))
    assert cache.max_q == 6


def test_cache_state_stays_where_it_is(kv):
    cache = make_cache(kv)
    lens, n_free = cache.lens, cache.n_free
    at = lens.data_ptr(), n_free.data_ptr()
    assert lens.tolist() == [0, 0] and n_free.tolist() == [10]
    for step in range(1, 4):
        cache._next.copy_(torch.tensor([step, 2 * step, 10 - step]))  # what the call would write
        if step < 3:
            cache.append(rows(5, 2), rows(5, 2), i64(3))
        else:
            cache.release()
        assert cache.lens is lens and cache.n_free is n_free and at == (lens.data_ptr(), n_free.data_ptr())
        assert lens.tolist() == [step, 2 * step] and n_free.tolist() == [10 - step]
    fn, args = kv._lib.calls[-1]
    assert fn == "lime_kv_release" and args[2] == at[0] and args[7] == at[1]


# --------------------------------------------------------- tensors of a call

class Space:
    """A workspace beside the host tensors that stand for device ones."""
    device, address, nbytes = -1, 1 << 20, 1 << 30


def call(kv, fn, **change):
    """Calls `fn` with B = 3 requests; returns what reached the library, if anything did."""
    d = kv.make_kv_dims(4, 2, 32, 16, 8, 5, "bf16")
    pool = dict(k_cache=torch.zeros(8, 2, 16, 32, dtype=torch.int8), scale=torch.zeros(8, 2, 2))
    pool["v_cache"] = pool["k_cache"].clone()
    table = dict(block_table=i32(3, 5))
    stack = dict(free_blocks=i32(8), n_free=i32(1), lens_out=i32(3), n_free_out=i32(1))
    args = {"lime_kv_reserve": dict(lens=i32(3), new_offsets=i64(4), **table, **stack, slot_map=i64(6)),
            "lime_kv_release": dict(lens=i32(3), keep=i32(3), **table, **stack),
            "lime_kv_append": dict(K=rows(6, 2), V=rows(6, 2), slot_map=i64(6), **pool),
            "lime_kv_attention": dict(Q=rows(6, 4), q_offsets=i64(4), **table, lens=i32(3), **pool, O=rows(6, 4),
                                      lse=torch.zeros(6, 4))}[fn]
    assert set(change) <= set(args)
    args.update(change)
    kv._lib.calls.clear()
    getattr(kv, fn)(d, ws=Space, **args)
    return kv._lib.calls


CALLS = ["lime_kv_reserve", "lime_kv_release", "lime_kv_append", "lime_kv_attention"]


@pytest.mark.parametrize("fn", CALLS)
def test_calls_pass_on_what_they_document(kv, fn):
    assert [n for n, _ in call(kv, fn)] == [fn]


WRONG_SHAPES = {
    "lens": [(3, 2), (6,), (1, 3), (3, 1)],
    "new_offsets": [(3,), (1, 4), (4, 1), (2, 2)],
    "q_offsets": [(3,), (1, 4), (4, 1), (2, 2)],
    "block_table": [(5, 3), (15,), (3, 5, 1), (3, 4), (4, 5)],
    "free_blocks": [(8, 1), (2, 4)],
    "n_free": [(), (1, 1), (2,)],
    "n_free_out": [(), (1, 1), (2,)],
    "lens_out": [(3, 1), (1, 3), (4,)],
    "keep": [(3, 1), (3, 2), (4,)],
    "slot_map": [(6, 1), (1, 6)],
    "lse": [(4, 6), (24,)],
}


@pytest.mark.parametrize("fn,name,shape", [(fn, name, shape) for fn, names in (
    ("lime_kv_reserve", "lens new_offsets block_table free_blocks n_free n_free_out lens_out slot_map"),
    ("lime_kv_release", "lens keep block_table free_blocks n_free n_free_out lens_out"),
    ("lime_kv_append", "slot_map"),
    ("lime_kv_attention", "lens q_offsets block_table lse")) for name in names.split() for shape in WRONG_SHAPES[name]])
def test_calls_refuse_other_shapes(kv, fn, name, shape):
    # among them shapes of as many elements, which would be read in another order
    dtype = {"new_offsets": torch.int64, "q_offsets": torch.int64, "slot_map": torch.int64,
             "lse": torch.float32}.get(name, torch.int32)
    with pytest.raises(ValueError):
        call(kv, fn, **{name: torch.zeros(shape, dtype=dtype)})
    assert kv._lib.calls == []


def test_a_workspace_is_initialised_on_its_own_device(kv, monkeypatch):
    # from another device's stream it would be cleared beside the calls that use it
    dims, cache = kv.make_kv_dims(4, 2, 32, 16, 10, 4, "bf16"), make_cache(kv)
    monkeypatch.setattr(kv, "lime_get_status", lambda ws, stream: 3)
    assert kv._lib.names() == ["lime_kv_workspace_init"] and cache.status() == 3
    monkeypatch.setattr(kv, "_device", lambda: 1)
    for make in (lambda: kv.KvWorkspace(dims, 2, 1, device="cpu"), lambda: make_cache(kv), cache.status):
        with pytest.raises(ValueError, match="current device"):
            make()
    assert kv._lib.names() == ["lime_kv_workspace_init"]


@pytest.mark.parametrize("pitch", [0, 3, 64, 65, 2 ** 33])
def test_the_pitch_of_a_single_row_does_not_matter(kv, pitch):
    one = torch.zeros(64, dtype=torch.bfloat16).as_strided((1, 2, 32), (pitch, 32, 1))
    assert kv._pitch("K", one, 2, 32) == 64
    (_, args), = call(kv, "lime_kv_append", K=one, V=one, slot_map=i64(1))
    assert args[2] == args[4] == 64
    q = torch.zeros(128, dtype=torch.bfloat16).as_strided((1, 4, 32), (pitch, 32, 1))
    (_, args), = call(kv, "lime_kv_attention", Q=q, O=rows(1, 4), lse=torch.zeros(1, 4))
    assert args[3] == 128


def test_the_strides_of_no_rows_do_not_matter(kv):
    # a slice of nothing, brought to another device, has strides of its own
    none = torch.zeros(0, 2, 4, 32, dtype=torch.bfloat16)[:, 1].transpose(0, 1).contiguous().transpose(0, 1)
    odd = torch.zeros(64, dtype=torch.bfloat16).as_strided((0, 4, 32), (1, 1, 7))
    for q in (none, odd):
        (_, args), = call(kv, "lime_kv_attention", Q=q, O=rows(0, 4), lse=torch.zeros(0, 4))
        assert args[3] == 128 and args[5] == 0
        (_, args), = call(kv, "lime_kv_append", K=q[:, :2], V=q[:, :2], slot_map=i64(0))
        assert args[2] == args[4] == 64 and args[5] == 0
    with pytest.raises(ValueError, match="contiguous"):
        call(kv, "lime_kv_append", K=rows(6, 4)[:, ::2], V=rows(6, 2))
