"""CPU-only checks of the history cache: its C ABI and host-side refusals (they
return before any CUDA call), and the oracle's pins against torch."""
import ctypes
import os
import re
import subprocess

import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from recsys_decoupled_link_b200 import build as lime_build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def kv():
    lime_build.build()
    from recsys_decoupled_link_b200 import lime_kv as m
    return m


def declared_functions():
    text = open(os.path.join(ROOT, "include", "lime_kv.h")).read()
    return sorted(set(re.findall(r"^\s*(?:int|size_t)\s+(lime_kv_\w+)\s*\(", text, re.M)))


def test_header_and_library_agree(kv):
    out = subprocess.run(["nm", "-D", "--defined-only", kv._lib._name], capture_output=True,
                         text=True, check=True).stdout
    exported = set(re.findall(r"\sT\s+(lime_kv_\w+)$", out, re.M))
    assert exported == set(declared_functions()) == set(kv.EXPORTED)


def test_header_compiles_as_c():
    src = '#include "lime_kv.h"\nint main(void){ lime_kv_dims d = {8,2,64,16,10,LIME_BF16,100};' \
          ' return (int)lime_kv_workspace_bytes(&d, 1, 1) == 0; }\n'
    r = subprocess.run(["gcc", "-std=c99", "-fsyntax-only", "-x", "c", "-",
                        "-I", os.path.join(ROOT, "include"), "-I", "/usr/local/cuda/include"],
                       input=src, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_workspace_bytes(kv):
    ok = kv.make_kv_dims(8, 2, 64, 16, 100, 10, "bf16")
    assert kv.lime_kv_workspace_bytes(ok, 0, 0) >= 256
    assert kv.lime_kv_workspace_bytes(ok, 4, 100) <= kv.lime_kv_workspace_bytes(ok, 400, 10000)
    for args in ((8, 3, 64, 16, 100, 10), (8, 2, 48, 16, 100, 10), (8, 2, 64, 8, 100, 10),
                 (8, 2, 64, 16, 100, 0), (0, 1, 64, 16, 100, 10), (2048, 2, 64, 16, 100, 10),
                 (8, 2, 64, 16, -1, 10), (8, 2, 64, 16, 2 ** 30, 10),
                 (8, 2, 64, 16, 100, 2 ** 27)):
        assert kv.lime_kv_workspace_bytes(kv.make_kv_dims(*args, "bf16"), 1, 1) == 0, args
    assert kv.lime_kv_workspace_bytes(kv.lime_kv_dims(8, 2, 64, 16, 10, 7, 100), 1, 1) == 0
    assert kv.lime_kv_workspace_bytes(ok, -1, 1) == 0


WS = 0x10000000


def test_workspace_init_refuses(kv):
    f = kv._lib.lime_kv_workspace_init
    for args in ((None, 1 << 20), (WS + 64, 1 << 20), (WS, 64)):
        assert f(*args, None) == kv_err(kv, "ARG"), args


def _call(kv, fn, dims, names, base, **change):
    a = dict(base)
    a.update(change)
    return getattr(kv._lib, fn)(ctypes.byref(dims), *[a[n] for n in names], None)


def test_reserve_refuses(kv):
    d = kv.make_kv_dims(8, 2, 64, 16, 100, 10, "bf16")
    names = ("B", "lens", "off", "total", "table", "free", "cap", "n_free", "lens_out",
             "n_free_out", "slots", "ws", "nws")
    base = dict(B=4, lens=0x1000, off=0x2000, total=9, table=0x3000, free=0x4000, cap=50,
                n_free=0x5000, lens_out=0x6000, n_free_out=0x7000, slots=0x8000, ws=WS,
                nws=kv.lime_kv_workspace_bytes(d, 4, 0))
    call = lambda dims=d, **c: _call(kv, "lime_kv_reserve", dims, names, base, **c)
    for change in (dict(lens=None), dict(off=None), dict(table=None), dict(n_free=None),
                   dict(lens_out=None), dict(n_free_out=None), dict(slots=None), dict(free=None),
                   dict(ws=None), dict(ws=WS + 16), dict(nws=64), dict(B=-1), dict(total=-1),
                   dict(cap=-1), dict(off=0x2004), dict(slots=0x8004), dict(lens=0x1002),
                   dict(B=0), dict(total=2 ** 31)):
        assert call(**change) == kv_err(kv, "ARG"), change
    for change in (dict(lens_out=0x1000), dict(n_free_out=0x5000), dict(slots=0x3000 + 16),
                   dict(table=0x4000), dict(slots=0x2000), dict(lens_out=WS + 64)):
        assert call(**change) == kv_err(kv, "ALIAS"), change
    assert call(kv.make_kv_dims(8, 2, 64, 24, 100, 10, "bf16")) == kv_err(kv, "SHAPE")


def kv_err(kv, name):
    from recsys_decoupled_link_b200 import lime
    return getattr(lime, "LIME_ERR_" + name)


def test_release_refuses(kv):
    d = kv.make_kv_dims(8, 2, 64, 16, 100, 10, "bf16")
    names = ("B", "lens", "keep", "table", "free", "cap", "n_free", "lens_out", "n_free_out", "ws",
             "nws")
    base = dict(B=4, lens=0x1000, keep=0x2000, table=0x3000, free=0x4000, cap=50, n_free=0x5000,
                lens_out=0x6000, n_free_out=0x7000, ws=WS,
                nws=kv.lime_kv_workspace_bytes(d, 4, 0))
    call = lambda **c: _call(kv, "lime_kv_release", d, names, base, **c)
    for change in (dict(lens=None), dict(table=None), dict(free=None), dict(n_free=None),
                   dict(lens_out=None), dict(ws=WS + 8), dict(nws=0), dict(B=-3),
                   dict(keep=0x2001)):
        assert call(**change) == kv_err(kv, "ARG"), change
    for change in (dict(lens_out=0x1000), dict(lens_out=0x2000), dict(n_free_out=0x5000),
                   dict(free=0x3000)):
        assert call(**change) == kv_err(kv, "ALIAS"), change


def test_append_refuses(kv):
    d = kv.make_kv_dims(8, 2, 64, 16, 100, 10, "bf16")
    names = ("K", "ldk", "V", "ldv", "total", "slots", "kc", "vc", "scale", "ws", "nws")
    base = dict(K=0x100000, ldk=128, V=0x200000, ldv=128, total=5, slots=0x300000, kc=0x400000,
                vc=0x800000, scale=0xc00000, ws=WS, nws=kv.lime_kv_workspace_bytes(d, 0, 0))
    call = lambda **c: _call(kv, "lime_kv_append", d, names, base, **c)
    for change in (dict(K=None), dict(V=None), dict(slots=None), dict(kc=None), dict(vc=None),
                   dict(scale=None), dict(ldk=120), dict(ldv=132), dict(K=0x100008),
                   dict(kc=0x400008), dict(total=-1), dict(nws=64), dict(ws=WS + 128)):
        assert call(**change) == kv_err(kv, "ARG"), change
    for change in (dict(kc=0x100000), dict(vc=0x400000 + 64), dict(scale=0x300000)):
        assert call(**change) == kv_err(kv, "ALIAS"), change
    assert call(total=0) == 0


def test_attention_refuses(kv):
    d = kv.make_kv_dims(8, 2, 64, 16, 100, 10, "bf16")
    names = ("B", "Q", "ldq", "off", "total", "table", "lens", "kc", "vc", "scale", "sm", "causal",
             "O", "lse", "ws", "nws")
    base = dict(B=2, Q=0x100000, ldq=512, off=0x200000, total=6, table=0x300000, lens=0x310000,
                kc=0x400000, vc=0x800000, scale=0xc00000, sm=ctypes.c_float(0.125), causal=0,
                O=0xd00000, lse=0xe00000, ws=WS, nws=kv.lime_kv_workspace_bytes(d, 2, 6))
    call = lambda **c: _call(kv, "lime_kv_attention", d, names, base, **c)
    for change in (dict(Q=None), dict(off=None), dict(table=None), dict(lens=None), dict(kc=None),
                   dict(scale=None), dict(O=None), dict(ldq=511), dict(ldq=516), dict(Q=0x100002),
                   dict(O=0xd00008), dict(lse=0xe00001), dict(causal=2), dict(B=0), dict(B=-1),
                   dict(total=2 ** 30), dict(nws=256), dict(sm=ctypes.c_float(float("nan")))):
        assert call(**change) == kv_err(kv, "ARG"), change
    for change in (dict(O=0x100000), dict(lse=0xd00000), dict(O=0x400000)):
        assert call(**change) == kv_err(kv, "ALIAS"), change
    assert call(total=0) == 0


def test_binding_checks_types_and_shapes(kv):
    d = kv.make_kv_dims(4, 2, 16, 16, 8, 4, "bf16")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)
    with pytest.raises(ValueError):
        kv.lime_kv_reserve(d, torch.zeros(3), torch.zeros(4, dtype=torch.int64), i32(3, 4), i32(8),
                           i32(1), i32(3), i32(1), torch.zeros(2, dtype=torch.int64), None)
    with pytest.raises(ValueError):     # a table of other width
        kv.lime_kv_reserve(d, i32(3), torch.zeros(4, dtype=torch.int64), i32(3, 5), i32(8),
                           i32(1), i32(3), i32(1), torch.zeros(2, dtype=torch.int64), None)
    x = torch.zeros(5, 2, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):     # host tensors
        kv.lime_kv_append(d, x, x, torch.zeros(5, dtype=torch.int64), None, None, None, None)
    with pytest.raises(ValueError):     # another type than the dims'
        kv.lime_kv_append(d, x.float(), x.float(), torch.zeros(5, dtype=torch.int64), None, None,
                          None, None)


# ------------------------------------------------------------- oracle pins

def test_oracle_attention_is_torch_attention():
    g = np.random.default_rng(0)
    bs, Hq, Hkv, dh, n, m = 16, 4, 2, 16, 37, 5
    k = g.integers(-127, 128, (6, Hkv, bs, dh)).astype(np.int8)
    v = g.integers(-127, 128, (6, Hkv, bs, dh)).astype(np.int8)
    scale = g.uniform(0.01, 0.03, (6, Hkv, 2))
    table, q = [[5, 0, 3]], g.standard_normal((m, Hq, dh))
    flat = lambda c, side: torch.tensor(
        (c[table[0]] * scale[table[0], :, side][..., None, None]).transpose(1, 0, 2, 3)
        .reshape(Hkv, -1, dh)[:, :n]).repeat_interleave(Hq // Hkv, 0)
    for causal in (False, True):
        mask = torch.ones(m, n, dtype=torch.bool)
        if causal:
            mask = mask.tril(n - m)
        ref = torch.nn.functional.scaled_dot_product_attention(
            torch.tensor(q).transpose(0, 1), flat(k, 0), flat(v, 1), attn_mask=mask)
        got, lse, A, S, V = K.attention(q, [m], table, [n], k, v, scale, bs, dh ** -0.5, causal)
        np.testing.assert_allclose(got, ref.transpose(0, 1).numpy(), rtol=1e-12, atol=1e-12)
        s = torch.tensor(q).transpose(0, 1) @ flat(k, 0).transpose(1, 2) * dh ** -0.5
        s = s.masked_fill(~mask, -np.inf).logsumexp(-1).T.numpy()
        np.testing.assert_allclose(lse, s, rtol=1e-12)
        assert (A >= np.abs(got) - 1e-12).all()


def test_oracle_attention_without_keys():
    q = np.ones((4, 1, 16))
    k = np.ones((1, 1, 16, 16), dtype=np.int8)
    O, lse, *_ = K.attention(q, [3, 1], [[0], [0]], [2, 0], k, k, np.ones((1, 1, 2)), 16, 1.0, True)
    assert (O[0] == 0).all() and np.isneginf(lse[0]).all()          # 3 queries, 2 rows: none seen
    np.testing.assert_allclose(O[1], 1.0)
    assert (O[3] == 0).all() and np.isneginf(lse[3]).all()          # an empty history


def test_oracle_append_quantises():
    codes = np.zeros((2, 1, 16, 2), dtype=np.int8)
    scale = np.zeros((2, 1))
    x = np.array([[[127.0, -63.5]], [[1.5, 2.5]]])                  # scale 1: ties to even
    c, s = K.append(x, np.array([16, 17]), codes, scale, 16)
    assert s[1, 0] == 1.0 and c[1, 0, :2].tolist() == [[127, -64], [2, 2]]
    c, s = K.append(np.array([[[254.0, 0.0]]]), np.array([18]), c, s, 16)
    assert s[1, 0] == 2.0 and c[1, 0, :3].tolist() == [[64, -32], [1, 1], [127, 0]]
    c, s = K.append(np.array([[[np.nan, np.inf]], [[4.0, -np.inf]]]), np.array([0, 1]), c, s, 16)
    assert c[0, 0, :2].tolist() == [[0, 127], [127, -127]]


def test_oracle_reserve_takes_from_the_top():
    table = -np.ones((3, 4), dtype=np.int64)
    table[0, 0] = 9
    lens, n_free, table, slots, refused = K.reserve([10, 0, 0], [10, 0, 40], table, [1, 2, 3, 4], 4, 16)
    assert table[0].tolist() == [9, 4, -1, -1] and table[2].tolist() == [3, 2, 1, -1]
    assert lens.tolist() == [20, 0, 40] and n_free == 0 and not refused
    assert slots[:10].tolist() == [9 * 16 + r for r in range(10, 16)] + [4 * 16 + r for r in range(4)]
    lens, n_free, table, slots, refused = K.reserve(lens, [1, 1, 1], table, [], 0, 16)
    assert refused == [1] and slots.tolist() == [4 * 16 + 4, -1, 1 * 16 + 8]
