"""The paged 8-bit history cache on the GPU against the fp64 oracle.

Tolerances.  Reserve, release and append are exact: block ids, slots, codes
and scales have to be equal (the quotient that decides a code is rounded
exactly, include/lime_kv.h).  Attention, per output element, with
  A = sum_j w_j |v_j|,  S = max_j sum_d |q_d k_jd| sm_scale  (oracle),
n keys and u = 2^-24 (half an fp32 step, relative):
  a score is off by at most ds = S ((dh + 8) 2u) (fp32 accumulation of dh exact
  products, a tensor core's adds may truncate: 2u each; eight more for the
  scales), its weight by a factor 1 + 2 ds + 8u (the exponential), the
  weighted sum by n 2u more, and the probability's rounding adds 2^-11 (one
  fp16 term, bf16 rows) or 2^-21 (two terms, fp32 rows).  The weights' sum in
  the denominator is off by the same, so
  |err| <= 2 A (2 ds + 8u + 2u n + p) + n 2^-39 V + half a step of the output type |O|;
  V = max_j |v_j|: a probability enters fp16 times 2^14, so one below fp16's normal range is off by half its
  smallest step, 2^-25 / 2^14 = 2^-39 of the row's largest, whatever its own size (include/lime_kv.h).
  |err lse| <= 2 ds + 8u + 2u n + 4u |lse|.
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from recsys_decoupled_link_b200 import lime, lime_kv

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def offsets(counts):
    return torch.tensor(np.concatenate([[0], np.cumsum(counts)]), dtype=torch.int64, device="cuda")


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def f64(t):
    return t.detach().to("cpu", torch.float64).numpy()


# ---------------------------------------------------------------- reserve

def run_reserve(lens, new, table, free, bs, n_blocks, n_free=None):
    B, cols = table.shape
    dims = lime_kv.make_kv_dims(1, 1, 16, bs, n_blocks, cols, "bf16")
    ws = lime_kv.KvWorkspace(dims, B, 0)
    tab, out = i32(table), torch.full((B,), -7, dtype=torch.int32, device="cuda")
    nfo = torch.full((1,), -7, dtype=torch.int32, device="cuda")
    slots = torch.full((int(np.sum(new)),), -7, dtype=torch.int64, device="cuda")
    lime_kv.lime_kv_reserve(dims, i32(lens), offsets(new), tab, i32(free),
                            i32([len(free) if n_free is None else n_free]), out, nfo, slots, ws)
    flags = lime.lime_get_status(ws)
    return (out.cpu().numpy(), int(nfo), tab.cpu().numpy(), slots.cpu().numpy()), flags


def pool_case(rng, B, bs, old_hi, new_hi, short=1.0, cols=None):
    lens, new = rng.integers(0, old_hi + 1, B), rng.integers(0, new_hi + 1, B)
    held = -(-lens // bs)
    need = int((-(-(lens + new) // bs) - held).sum())
    cols = int(max(1, (-(-(lens + new) // bs)).max())) if cols is None else cols
    lens = np.minimum(lens, cols * bs)
    held = -(-lens // bs)
    free = int(need * short) + (3 if short >= 1 else 0)
    ids = rng.permutation(int(held.sum()) + free + 5)
    table = np.full((B, cols), -1)
    at = 0
    for u in range(B):
        table[u, :held[u]] = ids[at:at + held[u]]
        at += held[u]
    return lens, new, table, ids[at:at + free], len(ids)


@pytest.mark.parametrize("B", [1, 2, 31, 256, 1023, 2048, 2049, 5000])
@pytest.mark.parametrize("bs,old_hi,new_hi,short", [(16, 100, 40, 1), (64, 0, 300, 1),
                                                    (32, 70, 1, 1), (16, 50, 60, 0.5),
                                                    (128, 700, 0, 1)])
def test_reserve_equals_the_oracle(B, bs, old_hi, new_hi, short):
    rng = np.random.default_rng(B * 1000 + bs + old_hi)
    lens, new, table, free, n_blocks = pool_case(rng, B, bs, old_hi, new_hi, short)
    got, flags = run_reserve(lens, new, table, free, bs, n_blocks)
    *want, refused = K.reserve(lens, new, table, free, len(free), bs)
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)
    assert flags == (lime_kv.LIME_FLAG_NO_BLOCKS if refused else 0)


def test_reserve_long_rows_and_narrow_tables():
    rng = np.random.default_rng(5)
    # a table too narrow for some requests: they alone are refused
    lens, new, table, free, n_blocks = pool_case(rng, 300, 16, 90, 90, cols=8)
    got, flags = run_reserve(lens, new, table, free, 16, n_blocks)
    *want, refused = K.reserve(lens, new, table, free, len(free), 16)
    assert refused and flags == lime_kv.LIME_FLAG_NO_BLOCKS
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)
    # few requests, many rows
    lens, new, table, free, n_blocks = pool_case(rng, 3, 128, 10, 200_000)
    got, flags = run_reserve(lens, new, table, free, 128, n_blocks)
    *want, refused = K.reserve(lens, new, table, free, len(free), 128)
    assert flags == 0
    for g, w in zip(got, want):
        np.testing.assert_array_equal(g, w)


def test_reserve_nothing_to_do():
    got, flags = run_reserve([0, 17, 3], [0, 0, 0], np.array([[-1, -1], [2, 1], [0, -1]]), [3, 4], 16, 5)
    np.testing.assert_array_equal(got[0], [0, 17, 3])
    assert got[1] == 2 and flags == 0


def test_reserve_bad_values_stay_in_bounds():
    table = np.full((3, 2), -1)
    # lengths and a free count outside their ranges, a free id outside the pool
    got, flags = run_reserve([-5, 40, 0], [1, 1, 1], table, [1, 99], 16, 4, n_free=7)
    assert flags & lime.LIME_FLAG_BAD_OFFSETS and flags & lime_kv.LIME_FLAG_BAD_BLOCK
    assert ((got[3] >= -1) & (got[3] < 4 * 16)).all()
    assert got[3][0] == -1                                           # its block was id 99


@pytest.mark.parametrize("B", [3, 2500])
def test_reserve_rows_of_nobody_get_no_slot(B):
    # offsets that end before the packed rows do: flagged, and those rows stay out of every block
    dims = lime_kv.make_kv_dims(1, 1, 16, 16, 3 * B, 2, "bf16")
    ws = lime_kv.KvWorkspace(dims, B, 0)
    tab, out, nfo = i32(np.full((B, 2), -1)), i32(np.zeros(B)), i32([0])
    slots = torch.full((B + 9,), -7, dtype=torch.int64, device="cuda")
    lime_kv.lime_kv_reserve(dims, i32(np.zeros(B)), offsets([1] * B), tab, i32(np.arange(3 * B)), i32([3 * B]), out,
                            nfo, slots, ws)
    assert lime.lime_get_status(ws) == lime.LIME_FLAG_BAD_OFFSETS
    assert (slots[B:] == -1).all() and (slots[:B] >= 0).all() and (tab[:, 1] == -1).all()
    # and offsets that begin behind row 0
    late = offsets([1] * B) + 9
    slots.fill_(-7)
    lime_kv.lime_kv_reserve(dims, i32(np.zeros(B)), late, tab, i32(np.arange(3 * B)), i32([3 * B]), out, nfo, slots, ws)
    assert lime.lime_get_status(ws) == lime.LIME_FLAG_BAD_OFFSETS
    assert (slots[:9] == -1).all() and (slots[9:] >= 0).all()


def test_reserve_many_rows_behind_rows_of_nobody():
    # 80,000 rows: the first request begins at row 3, inside the rows that one thread places, and holds 5 rows
    B, n, bs = 3, 80_000, 128
    dims = lime_kv.make_kv_dims(1, 1, 16, bs, 700, 300, "bf16")
    ws = lime_kv.KvWorkspace(dims, B, 0)
    counts, lens = np.array([26_667, 26_665, 26_665]), np.array([5, 6, 128])
    table = np.full((B, 300), -1)
    table[:, 0] = [690, 691, 692]
    tab, out, nfo = i32(table), i32(np.zeros(B)), i32([0])
    slots = torch.full((n,), -7, dtype=torch.int64, device="cuda")
    lime_kv.lime_kv_reserve(dims, i32(lens), offsets(counts) + 3, tab, i32(np.arange(690)), i32([690]), out, nfo,
                            slots, ws)
    assert lime.lime_get_status(ws) == lime.LIME_FLAG_BAD_OFFSETS
    lens_w, nf_w, tab_w, slots_w, _ = K.reserve(lens, counts, table, np.arange(690), 690, bs)
    np.testing.assert_array_equal(slots.cpu()[3:], slots_w)
    assert (slots[:3] == -1).all() and int(nfo) == nf_w
    np.testing.assert_array_equal(tab.cpu(), tab_w)
    np.testing.assert_array_equal(out.cpu(), lens_w)


def test_calls_without_requests():
    dims = lime_kv.make_kv_dims(2, 2, 16, 16, 8, 2, "bf16")
    ws = lime_kv.KvWorkspace(dims, 0, 4)
    none, n_free, out = torch.zeros(0, dtype=torch.int32, device="cuda"), i32([5]), i32([0])
    off = torch.zeros(1, dtype=torch.int64, device="cuda")
    table = torch.zeros(0, 2, dtype=torch.int32, device="cuda")
    lime_kv.lime_kv_reserve(dims, none, off, table, i32(np.arange(8)), n_free, none.clone(), out,
                            torch.zeros(0, dtype=torch.int64, device="cuda"), ws)
    assert int(out) == 5
    lime_kv.lime_kv_release(dims, none, None, table, i32(np.arange(8)), n_free, none.clone(), out, ws)
    assert int(out) == 5
    k = torch.zeros(8, 2, 16, 16, dtype=torch.int8, device="cuda")
    x, scale = torch.zeros(0, 2, 16, dtype=torch.bfloat16, device="cuda"), torch.zeros(8, 2, 2, device="cuda")
    lime_kv.lime_kv_append(dims, x, x, torch.zeros(0, dtype=torch.int64, device="cuda"), k, k.clone(), scale, ws)
    lime_kv.lime_kv_attention(dims, x, off, table, none, k, k.clone(), scale, x.clone(), None, ws)
    assert lime.lime_get_status(ws) == 0


@pytest.mark.parametrize("B", [1, 70, 3000])
@pytest.mark.parametrize("how", ["all", "some"])
def test_release_equals_the_oracle(B, how):
    rng = np.random.default_rng(B)
    lens, _, table, free, n_blocks = pool_case(rng, B, 16, 100, 30)
    dims = lime_kv.make_kv_dims(1, 1, 16, 16, n_blocks, table.shape[1], "bf16")
    ws = lime_kv.KvWorkspace(dims, B, 0)
    keep = None if how == "all" else rng.integers(-3, 120, B)
    stack = np.concatenate([free, np.full(n_blocks - len(free), -9)])
    tab, st = i32(table), i32(stack)
    out, nfo = i32(np.zeros(B)), i32([0])
    lime_kv.lime_kv_release(dims, i32(lens), None if keep is None else i32(keep), tab, st,
                            i32([len(free)]), out, nfo, ws)
    assert lime.lime_get_status(ws) == 0
    w_lens, w_stack, w_table = K.release(lens, keep, table, free, len(free), 16)
    np.testing.assert_array_equal(out.cpu(), w_lens)
    np.testing.assert_array_equal(tab.cpu(), w_table)
    assert int(nfo) == len(w_stack)
    np.testing.assert_array_equal(st.cpu()[:len(w_stack)], w_stack)


def test_release_past_the_stack_is_flagged():
    dims = lime_kv.make_kv_dims(1, 1, 16, 16, 8, 4, "bf16")
    ws = lime_kv.KvWorkspace(dims, 1, 0)
    st, out, nfo = i32([0, 0]), i32([0]), i32([0])
    lime_kv.lime_kv_release(dims, i32([64]), None, i32([[4, 5, 6, 7]]), st, i32([0]), out, nfo, ws)
    assert lime.lime_get_status(ws) == lime_kv.LIME_FLAG_BAD_BLOCK
    assert int(nfo) == 2 and st.tolist() == [4, 5]


# ----------------------------------------------------------------- append

def append_case(rng, counts, olds, Hkv, dh, bs, dtype, spread=1.0):
    """Slots of new rows behind `olds` rows, in shuffled blocks; random pool."""
    nb = [-(-(o + c) // bs) for o, c in zip(olds, counts)]
    blocks = sum(nb) + 3
    ids, at, slots = rng.permutation(blocks), 0, []
    for o, c, k in zip(olds, counts, nb):
        slots += [int(ids[at + j // bs]) * bs + j % bs for j in range(o, o + c)]
        at += k
    codes = rng.integers(-127, 128, (2, blocks, Hkv, bs, dh)).astype(np.int8)
    scale = rng.uniform(0.2, 1.5, (blocks, Hkv, 2)).astype(np.float32) * spread / 32
    x = torch.tensor(rng.standard_normal((2, len(slots), Hkv, dh)) * spread).to(DT[dtype])
    return x, np.array(slots, dtype=np.int64), codes, scale


def run_append(x, slots, codes, scale, bs, dtype, strided=False):
    _, n, Hkv, dh = x.shape
    dims = lime_kv.make_kv_dims(Hkv, Hkv, dh, bs, codes.shape[1], 1, dtype)
    ws = lime_kv.KvWorkspace(dims, 0, 0)
    kc, vc = torch.tensor(codes[0], device="cuda"), torch.tensor(codes[1], device="cuda")
    sc = torch.tensor(scale, device="cuda")
    if strided:   # slices of one projection's output, rows further apart than their width
        wide = torch.zeros(n, 3, Hkv, dh, dtype=x.dtype, device="cuda")
        wide[:, 1], wide[:, 2] = x[0].cuda(), x[1].cuda()
        k, v = wide[:, 1], wide[:, 2]
    else:
        k, v = x[0].cuda().contiguous(), x[1].cuda().contiguous()
    lime_kv.lime_kv_append(dims, k, v, torch.tensor(slots, device="cuda"), kc, vc, sc, ws)
    return kc.cpu().numpy(), vc.cpu().numpy(), sc.cpu().numpy(), lime.lime_get_status(ws)


def check_append(x, slots, codes, scale, bs, dtype, strided=False, want_flags=0):
    kc, vc, sc, flags = run_append(x, slots, codes, scale, bs, dtype, strided)
    for side, got in ((0, kc), (1, vc)):
        wc, wsc = K.append(f64(x[side]), slots, codes[side], scale[..., side].astype(np.float64), bs)
        np.testing.assert_array_equal(sc[..., side].astype(np.float64), wsc)
        np.testing.assert_array_equal(got, wc)
    assert flags == want_flags


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [16, 32, 64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_append_equals_the_oracle(dtype, dh, bs):
    rng = np.random.default_rng(dh * bs)
    counts = [1, 0, 5, bs, bs + 1, 3 * bs - 1, 1, 17]
    olds = [0, 3, bs - 1, 0, 7, bs // 2, 5 * bs + 3, bs]
    args = append_case(rng, counts, olds, 3, dh, bs, dtype)
    check_append(*args, bs, dtype, strided=bs != 32)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("Hkv", [1, 2, 8])
def test_append_one_row_each(dtype, Hkv):
    rng = np.random.default_rng(Hkv)
    olds = rng.integers(0, 200, 150)
    args = append_case(rng, [1] * 150, olds, Hkv, 64, 64, dtype)
    check_append(*args, 64, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("spread", [1e-38, 1e-30, 1e30, 1e36])
def test_append_extreme_magnitudes(dtype, spread):
    rng = np.random.default_rng(3)
    args = append_case(rng, [20, 3], [0, 9], 2, 32, 16, dtype, spread)
    check_append(*args, 16, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_ties_and_zeros(dtype):
    # scale 1 (a 127 in every group): halves round to even; scale 2^-6 likewise
    rng = np.random.default_rng(4)
    x, slots, codes, scale = append_case(rng, [16, 32], [0, 0], 2, 64, 16, dtype)
    x = torch.tensor(rng.integers(-253, 254, x.shape) / 2.0).clamp(-126.5, 126.5)
    x[:, :, :, 0] = 127.0
    x[1] /= 64.0
    x[:, 40:48, 1] = 0.0
    check_append(x.to(DT[dtype]), slots, codes, scale, 16, dtype)
    # an all-zero block has scale 0 and codes 0
    check_append(torch.zeros_like(x).to(DT[dtype]), slots, codes, scale, 16, dtype)


def test_append_near_ties_fp32():
    # values one fp32 step beside a code's border, for scales that are not powers of two
    rng = np.random.default_rng(6)
    x, slots, codes, scale = append_case(rng, [64] * 4, [0] * 4, 4, 64, 64, "f32")
    top = rng.uniform(0.5, 2.0, x.shape[:3] + (1,)).astype(np.float32)
    top[:] = top[:, :1]                                  # one top value per block's head
    s = (top.astype(np.float64) / 127.0).astype(np.float32).astype(np.float64)
    r = rng.integers(-126, 126, x.shape) + 0.5
    v = (r * s).astype(np.float32)
    v = np.where(rng.random(x.shape) < 0.5, np.nextafter(v, np.float32(9)), np.nextafter(v, np.float32(-9)))
    v[..., :1] = top
    check_append(torch.tensor(v), slots, codes, scale, 64, "f32")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_append_nan_and_infinity(dtype):
    rng = np.random.default_rng(8)
    x, slots, codes, scale = append_case(rng, [20, 1, 1], [0, 5, 0], 2, 32, 16, dtype)
    x[0, 3, 0, 5], x[0, 4, 1, 0], x[1, 19, 0, 31] = np.nan, np.inf, -np.inf
    x[1, 20, 1, :], x[0, 21, 0, :] = np.inf, np.nan
    check_append(x, slots, codes, scale, 16, dtype, want_flags=lime_kv.LIME_FLAG_NONFINITE)


def test_append_skips_rows_without_a_slot():
    rng = np.random.default_rng(9)
    x, slots, codes, scale = append_case(rng, [40, 9], [3, 0], 2, 32, 16, "bf16")
    slots[13:29] = -1                                   # the rows of one block found no room
    check_append(x, slots, codes, scale, 16, "bf16")
    slots[40] = codes.shape[1] * 16                     # behind the pool
    slots[41] = -2
    check_append(x, slots, codes, scale, 16, "bf16", want_flags=lime_kv.LIME_FLAG_BAD_BLOCK)


def test_append_twice_changes_nothing_more():
    rng = np.random.default_rng(10)
    x, slots, codes, scale = append_case(rng, [40, 1, 7], [3, 20, 0], 2, 64, 32, "bf16")
    k1, v1, s1, _ = run_append(x, slots, codes, scale, 32, "bf16")
    k2, v2, s2, _ = run_append(x, slots, np.stack([k1, v1]), s1, 32, "bf16")
    assert (k1 == k2).all() and (v1 == v2).all() and (s1 == s2).all()


def test_append_many_rows():
    rng = np.random.default_rng(11)
    args = append_case(rng, [2000, 1, 777], [0, 63, 5], 4, 32, 64, "bf16")
    check_append(*args, 64, "bf16")


# -------------------------------------------------------------- attention

def make_pool(rng, lens, Hkv, dh, bs, spare=2):
    nb = [-(-n // bs) for n in lens]
    blocks = sum(nb) + spare
    ids = rng.permutation(blocks)
    cols = max(1, max(nb)) + 1
    table = np.full((len(lens), cols), -1)
    at = 0
    for u, k in enumerate(nb):
        table[u, :k] = ids[at:at + k]
        at += k
    codes = np.clip(np.rint(rng.standard_normal((2, blocks, Hkv, bs, dh)) * 33), -127, 127).astype(np.int8)
    scale = (np.exp(0.4 * rng.standard_normal((blocks, Hkv, 2))) / 32).astype(np.float32)
    scale[ids[at:]] = np.nan                            # blocks of nobody
    return table, codes, scale


def check_attention(counts, lens, Hq, Hkv, dh, bs, dtype, causal=False, q_gain=1.0, seed=0, hook=None,
                    want_flags=0, strided=False, sm_scale=None):
    rng = np.random.default_rng(seed)
    table, codes, scale = make_pool(rng, lens, Hkv, dh, bs)
    n = int(np.sum(counts))
    q = torch.tensor(rng.standard_normal((n, Hq, dh)) * q_gain).to(DT[dtype])
    if hook:
        hook(table, codes, scale, q)
    dims = lime_kv.make_kv_dims(Hq, Hkv, dh, bs, codes.shape[1], table.shape[1], dtype)
    ws = lime_kv.KvWorkspace(dims, len(lens), n)
    qd = q.cuda()
    if strided:
        wide = torch.full((n, Hq + 1, dh), float("nan"), dtype=q.dtype, device="cuda")
        wide[:, :Hq] = qd
        qd = wide[:, :Hq]
    O = torch.full((n, Hq, dh), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((n, Hq), 7.0, device="cuda")
    args = (dims, qd, offsets(counts), i32(table), i32(lens), torch.tensor(codes[0], device="cuda"),
            torch.tensor(codes[1], device="cuda"), torch.tensor(scale, device="cuda"))
    sm = dh ** -0.5 if sm_scale is None else sm_scale
    lime_kv.lime_kv_attention(*args, O, lse, ws, sm_scale=sm_scale, causal=causal)
    assert lime.lime_get_status(ws) == want_flags
    # a second pass, without lse, gives the same bits
    O2 = torch.empty_like(O)
    lime_kv.lime_kv_attention(*args, O2, None, ws, sm_scale=sm_scale, causal=causal)
    assert torch.equal(O2.view(torch.uint8), O.view(torch.uint8))
    lime.lime_get_status(ws)
    ref, rl, A, S, V = K.attention(f64(q), counts, table, lens, codes[0], codes[1],
                                np.nan_to_num(scale).astype(np.float64), bs, sm, causal)
    assert_near(O, lse, ref, rl, A, S, V, max([1] + list(lens)), dh, dtype)
    return O, lse


def assert_near(O, lse, ref, rl, A, S, V, n, dh, dtype):
    ds = S * (dh + 8) * 2 * U
    p, half = (2.0 ** -11, 2.0 ** -8) if dtype == "bf16" else (2.0 ** -21, U)
    rel = 2 * ds + 8 * U + 2 * U * n
    err = np.abs(f64(O) - ref)
    tol = 2 * A * (rel[..., None] + p) + n * 2.0 ** -39 * V + half * np.abs(ref) + 1e-38
    assert (err <= tol).all(), (err / tol).max()
    got = f64(lse)
    empty = np.isneginf(rl)
    assert np.isneginf(got[empty]).all() and (f64(O)[empty] == 0).all()
    e = np.abs(got[~empty] - rl[~empty])
    t = rel[~empty] + 4 * U * np.abs(rl[~empty])
    assert (e <= t).all(), (e / t).max()


LENS = [0, 1, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 300]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [16, 32, 64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
def test_attention_single_rows(dtype, dh, bs):
    check_attention([1] * len(LENS), LENS, 4, 2, dh, bs, dtype, causal=bs == 16)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh,Hq,Hkv,l", [(32, 4, 4, 32), (32, 4, 4, 64), (64, 1, 1, 32), (16, 2, 2, 16),
                                         (128, 2, 1, 33), (64, 3, 3, 100), (32, 2, 2, 128)])
def test_attention_links(dtype, dh, Hq, Hkv, l):
    lens = [70, 0, 1, 200, 64]
    check_attention([l] * len(lens), lens, Hq, Hkv, dh, 64, dtype, strided=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("B,Hq,Hkv,dh,q", [(700, 2, 2, 32, 1), (2100, 1, 1, 16, 1), (2500, 2, 1, 128, 1),
                                           (2200, 1, 1, 32, 3), (600, 2, 2, 64, 2)])
def test_attention_many_requests(B, Hq, Hkv, dh, q, dtype):
    # a warp to a pair, and more requests than a thread block sums by itself
    rng = np.random.default_rng(B)
    lens = rng.integers(0, 70, B)
    counts = rng.integers(0, q + 1, B) if q > 1 else np.ones(B, dtype=int)
    lens[5], lens[B - 1] = 900, 0
    check_attention(counts, lens, Hq, Hkv, dh, 16, dtype, causal=q > 1)


def test_attention_rows_behind_the_last_request_are_left():
    rng = np.random.default_rng(3)
    table, codes, scale = make_pool(rng, [40], 1, 32, 16)
    dims = lime_kv.make_kv_dims(1, 1, 32, 16, codes.shape[1], table.shape[1], "bf16")
    ws = lime_kv.KvWorkspace(dims, 1, 5)
    q = torch.ones(5, 1, 32, dtype=torch.bfloat16, device="cuda")
    O, lse = torch.full_like(q, 9.0), torch.full((5, 1), 9.0, device="cuda")
    lime_kv.lime_kv_attention(dims, q, offsets([3]), i32(table), i32([40]), torch.tensor(codes[0], device="cuda"),
                              torch.tensor(codes[1], device="cuda"), torch.tensor(scale, device="cuda"), O, lse, ws)
    assert lime.lime_get_status(ws) == lime.LIME_FLAG_BAD_OFFSETS
    assert (O[3:] == 9.0).all() and (lse[3:] == 9.0).all() and (O[:3] != 9.0).any()


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("dh,Hq,Hkv,l", [(32, 4, 4, 32), (32, 8, 4, 20), (32, 2, 2, 64), (32, 3, 3, 128), (64, 2, 2, 64),
                                         (64, 6, 6, 40), (64, 5, 1, 30), (128, 1, 1, 90)])
def test_attention_many_rows(bs, dh, Hq, Hkv, l):
    # one to four heads to a tensor-core tile, full and partly filled, one tile of rows and several
    lens = [70, 0, 1, 200, 64, 129]
    counts = [l, l, l - 3, l + 7, 3 * l + 1, 0]
    check_attention(counts, lens, Hq, Hkv, dh, bs, "bf16", strided=True)
    check_attention(counts, lens, Hq, Hkv, dh, bs, "bf16", causal=True, seed=1)


def test_attention_many_rows_split_over_the_gpu():
    check_attention([32], [7001], 4, 4, 32, 64, "bf16")
    check_attention([64, 70], [3000, 129], 2, 2, 64, 16, "bf16", causal=True)


def test_attention_many_rows_sharp_and_flat():
    for gain, sm in ((20.0, None), (0.0, None), (1.0, -0.3), (1.0, 0.0), (1e30, 1e-30), (1e-30, 1e29)):
        check_attention([32, 32], [300, 90], 4, 4, 32, 64, "bf16", q_gain=gain, sm_scale=sm)


def test_attention_many_rows_bad_pages_and_uneven_scales():
    def bad(table, codes, scale, q):
        table[0, 1], table[1, 0] = 10 ** 6, -1
        scale[table[2, 1], :, 1] *= 2.0 ** 40
        scale[table[2, 2], :, 1] = 0.0
        codes[1, table[2, 2]] = 0
        table[:, -1] = 2 ** 31 - 1
    O, lse = check_attention([32, 32, 32], [150, 9, 190], 4, 4, 32, 16, "bf16", hook=bad,
                             want_flags=lime_kv.LIME_FLAG_BAD_BLOCK)
    assert (O[32:64] == 0).all() and torch.isneginf(lse[32:64]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [16, 32, 64, 128])
@pytest.mark.parametrize("G", [1, 2, 4, 8])
def test_attention_causal_chunks(dtype, dh, G):
    # more queries than rows (the first see nothing), as many, fewer, none; a chunk over many tiles
    counts, lens = [5, 17, 40, 0, 3, 1, 70], [3, 17, 100, 50, 0, 90, 150]
    check_attention(counts, lens, 2 * G, 2, dh, 16, dtype, causal=True)


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hkv,dh", [(32, 8, 128), (8, 1, 64), (24, 2, 32), (5, 1, 16), (64, 1, 128)])
def test_attention_head_layouts(causal, Hq, Hkv, dh):
    check_attention([1, 3, 2], [130, 37, 64], Hq, Hkv, dh, 32, "bf16", causal=causal)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_long_rows_split_over_the_gpu(dtype):
    # one request: its rows are split over many thread blocks and joined
    check_attention([2], [9000], 2, 1, 64, 64, dtype)
    check_attention([1, 1, 1], [5003, 1, 2500], 4, 1, 128, 16, dtype, causal=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_attention_sharp_and_flat_rows(dtype):
    check_attention([4, 4], [300, 90], 4, 2, 64, 64, dtype, q_gain=20.0)
    check_attention([4, 4], [300, 90], 4, 2, 64, 64, dtype, q_gain=0.0)
    check_attention([4, 4], [300, 90], 4, 2, 64, 64, dtype, sm_scale=-0.3)
    check_attention([4, 4], [300, 90], 4, 2, 64, 64, dtype, sm_scale=0.0)
    check_attention([4, 4], [300, 90], 4, 2, 64, 64, dtype, q_gain=1e30, sm_scale=1e-30)
    check_attention([4, 4], [300, 90], 4, 2, 64, 64, dtype, q_gain=1e-30, sm_scale=1e29)


def test_attention_scales_of_very_different_size():
    # a block whose values are 2^40 times the others', one whose keys or values are all zero
    def hook(table, codes, scale, q):
        scale[table[0, 1], :, 1] *= 2.0 ** 40
        scale[table[0, 2], :, 1] = 0.0
        codes[1, table[0, 2]] = 0
        scale[table[0, 3], :, 0] = 0.0
        codes[0, table[0, 3]] = 0
    for dtype in DT:
        check_attention([3, 1], [100, 20], 4, 2, 32, 16, dtype, hook=hook)


def test_attention_a_sink_row_with_a_small_value():
    # one row holds nearly all weight and a value 0: the output is the sum of the others' tiny weights
    def hook(table, codes, scale, q):
        q[:, :, 0] = 30.0
        codes[0, :, :, :, 0] = 0
        codes[0, table[0, 0], :, 0, 0] = 127
        codes[1, table[0, 0], :, 0] = 0
    for dtype in DT:
        check_attention([2], [1000], 2, 2, 32, 64, dtype, hook=hook)


def test_attention_garbage_behind_the_last_row_is_not_used():
    def hook(table, codes, scale, q):
        table[:, -1] = 2 ** 31 - 1                      # columns behind the last block
        codes[:, table[0, 1], :, 5:] = 127              # rows behind the last one
    check_attention([2, 1], [21, 16], 2, 2, 32, 16, "bf16", hook=hook)


def test_attention_bad_table_entries_hide_their_rows():
    def hook(table, codes, scale, q):
        table[0, 1], table[1, 0] = 10 ** 6, -1          # one block of several; a request's only one
    O, lse = check_attention([2, 2, 1], [80, 9, 40], 2, 1, 64, 16, "bf16", hook=hook,
                             want_flags=lime_kv.LIME_FLAG_BAD_BLOCK)
    assert (O[2:4] == 0).all() and torch.isneginf(lse[2:4]).all()


def test_attention_nan_in_one_row_stays_there():
    rng = np.random.default_rng(1)
    table, codes, scale = make_pool(rng, [100], 2, 32, 16)
    q = torch.tensor(rng.standard_normal((40, 4, 32))).to(torch.bfloat16).cuda()
    dims = lime_kv.make_kv_dims(4, 2, 32, 16, codes.shape[1], table.shape[1], "bf16")
    ws = lime_kv.KvWorkspace(dims, 1, 40)
    run = lambda q: _attend(dims, q, [40], table, [100], codes, scale, ws)
    clean = run(q)
    q[7, 1, 3], q[9, 2, 0] = float("nan"), float("inf")
    bad = run(q)
    assert torch.isnan(bad[7, 1]).all() and torch.isnan(bad[9, 2]).all()
    keep = torch.ones(40, 4, dtype=torch.bool)
    keep[7, 1] = keep[9, 2] = False
    assert torch.equal(bad.cpu()[keep], clean.cpu()[keep])


def _attend(dims, q, counts, table, lens, codes, scale, ws, **kw):
    O = torch.empty_like(q)
    lime_kv.lime_kv_attention(dims, q, offsets(counts), i32(table), i32(lens), torch.tensor(codes[0], device="cuda"),
                              torch.tensor(codes[1], device="cuda"), torch.tensor(scale, device="cuda"), O, None, ws,
                              **kw)
    return O


def test_attention_bad_lengths_and_offsets_stay_in_bounds():
    rng = np.random.default_rng(2)
    table, codes, scale = make_pool(rng, [64, 64], 1, 32, 16)
    table[:, -1] = 0
    scale = np.nan_to_num(scale)
    dims = lime_kv.make_kv_dims(1, 1, 32, 16, codes.shape[1], table.shape[1], "bf16")
    ws = lime_kv.KvWorkspace(dims, 2, 4)
    q = torch.ones(4, 1, 32, dtype=torch.bfloat16, device="cuda")
    _attend(dims, q, [2, 2], table, [-1, 10 ** 6], codes, scale, ws)
    assert lime.lime_get_status(ws) == lime.LIME_FLAG_BAD_OFFSETS
    _attend(dims, q, [3, 9], table, [64, 64], codes, scale, ws)
    assert lime.lime_get_status(ws) == lime.LIME_FLAG_BAD_OFFSETS
    _attend(dims, q, [10, -10], table, [64, 64], codes, scale, ws)
    assert lime.lime_get_status(ws) == lime.LIME_FLAG_BAD_OFFSETS


def test_cache_past_four_gigabytes():
    # 2^32 bytes of keys: only the blocks in use are written and read
    Hkv, dh, bs = 2, 128, 128
    n_blocks = (1 << 32) // (Hkv * dh * bs) + 7
    dims = lime_kv.make_kv_dims(2, Hkv, dh, bs, n_blocks, 2, "bf16")
    kc, vc = (torch.empty(n_blocks, Hkv, bs, dh, dtype=torch.int8, device="cuda") for _ in range(2))
    scale = torch.zeros(n_blocks, Hkv, 2, device="cuda")
    ws = lime_kv.KvWorkspace(dims, 1, 3)
    rng = np.random.default_rng(3)
    x = torch.tensor(rng.standard_normal((2, 140, Hkv, dh))).to(torch.bfloat16)
    table = np.array([[n_blocks - 1, n_blocks - 3]])
    slots = np.array([int(table[0, j // bs]) * bs + j % bs for j in range(140)])
    lime_kv.lime_kv_append(dims, x[0].cuda(), x[1].cuda(), torch.tensor(slots, device="cuda"), kc, vc, scale, ws)
    q = torch.tensor(rng.standard_normal((3, 2, dh))).to(torch.bfloat16)
    O, lse = torch.empty(3, 2, dh, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 2, device="cuda")
    lime_kv.lime_kv_attention(dims, q.cuda(), offsets([3]), i32(table), i32([140]), kc, vc, scale, O, lse, ws)
    assert lime.lime_get_status(ws) == 0
    ids = table[0]
    small = [K.append(f64(x[s]), slots % bs + bs * (slots // bs == ids[1]),
                      np.zeros((2, Hkv, bs, dh), dtype=np.int8), np.zeros((2, Hkv)), bs) for s in (0, 1)]
    for s, cache in ((0, kc), (1, vc)):
        got = cache[torch.tensor(ids, device="cuda")].cpu().numpy()
        assert (got[0] == small[s][0][0]).all() and (got[1, :, :12] == small[s][0][1, :, :12]).all()
    both = np.stack([small[0][1], small[1][1]], -1)
    ref, rl, A, S, V = K.attention(f64(q), [3], np.array([[0, 1]]), [140], small[0][0], small[1][0], both, bs,
                                dh ** -0.5, False)
    assert_near(O, lse, ref, rl, A, S, V, 140, dh, "bf16")


# --------------------------------------------------------------- together

def test_cache_serves_a_growing_history():
    """Append, attend, append again, release: the outputs are the attention over the values that the
    oracle's own quantisation of the same rows gives, and near the unquantised rows' attention."""
    rng = np.random.default_rng(12)
    B, Hq, Hkv, dh, bs = 5, 4, 2, 32, 16
    dims = lime_kv.make_kv_dims(Hq, Hkv, dh, bs, 64, 16, "bf16")
    cache = lime_kv.HistoryCache(dims, B)
    codes = np.zeros((2, 64, Hkv, bs, dh), dtype=np.int8)
    scale = np.zeros((64, Hkv, 2))
    lens, free, n_free = np.zeros(B, dtype=int), np.arange(63, -1, -1), 64
    table = np.full((B, 16), -1)
    full = [np.zeros((0, 2, Hkv, dh)) for _ in range(B)]

    def step(counts):
        nonlocal lens, n_free, table, scale
        n = int(np.sum(counts))
        x = torch.tensor(rng.standard_normal((n, 2, Hkv, dh))).to(torch.bfloat16)
        slots = cache.append(x[:, 0].cuda(), x[:, 1].cuda(), offsets(counts))
        lens, n_free, table, want, refused = K.reserve(lens, counts, table, free, n_free, bs)
        assert not refused
        np.testing.assert_array_equal(slots.cpu(), want)
        new_scale = scale.copy()
        for s in (0, 1):
            codes[s], new_scale[..., s] = K.append(f64(x[:, s]), want, codes[s], scale[..., s], bs)
        scale = new_scale
        at = 0
        for u, c in enumerate(counts):
            full[u] = np.concatenate([full[u], f64(x[at:at + c])])
            at += c

    def attend(counts, causal):
        q = torch.tensor(rng.standard_normal((int(np.sum(counts)), Hq, dh))).to(torch.bfloat16)
        lse = torch.empty(q.shape[:2], device="cuda")
        O = cache.attend(q.cuda(), offsets(counts), causal=causal, lse=lse)
        assert cache.status() == 0
        ref, rl, A, S, V = K.attention(f64(q), counts, table, lens, codes[0], codes[1], scale, bs, dh ** -0.5, causal)
        assert_near(O, lse, ref, rl, A, S, V, int(lens.max()), dh, "bf16")
        # against the rows themselves: a key or value is off by half a code, at most its block's scale / 2
        # per element, and by as much again each time the scale grew
        i = 0
        for u, m in enumerate(counts):
            for r in range(m):
                seen = int(lens[u]) - m + r + 1 if causal else int(lens[u])
                if seen > 0 and not causal:
                    k, v = full[u][:seen, 0], full[u][:seen, 1]
                    for h in range(Hq):
                        s = k[:, h // 2] @ f64(q[i, h]) * dh ** -0.5
                        w = np.exp(s - s.max())
                        dk = 4 * scale[..., 0].max() / 2 * np.abs(f64(q[i, h])).sum() * dh ** -0.5
                        dv = 4 * scale[..., 1].max() / 2
                        out = (w / w.sum()) @ v[:, h // 2]
                        mag = (w / w.sum()) @ np.abs(v[:, h // 2])
                        tol = (np.exp(2 * dk) - 1) * mag + np.exp(2 * dk) * dv + 2.0 ** -7 * mag + 1e-3
                        assert (np.abs(f64(O[i, h]) - out) <= tol).all()
                i += 1

    step([40, 0, 1, 100, 16])
    attend([8, 8, 8, 8, 8], False)
    step([1, 1, 1, 1, 1])
    attend([1, 1, 1, 1, 1], True)
    step([0, 30, 5, 33, 0])
    attend([0, 30, 5, 33, 0], True)
    attend([8, 0, 3, 1, 2], False)
    keep = [10, 0, 500, 64, 0]
    cache.release(i32(keep))
    lens, stack, table = K.release(lens, keep, table, free, n_free, bs)
    free, n_free = stack, len(stack)
    full = [f[:n] for f, n in zip(full, lens)]
    np.testing.assert_array_equal(cache.table.cpu(), table)
    step([20, 20, 2, 0, 1])
    attend([4, 4, 4, 4, 4], False)


def test_cache_refused_rows_change_nothing():
    dims = lime_kv.make_kv_dims(2, 2, 32, 16, 20, 4, "bf16")
    cache, other = lime_kv.HistoryCache(dims, 2), lime_kv.HistoryCache(dims, 2)
    x = torch.randn(50, 2, 2, 32, device="cuda").to(torch.bfloat16)
    for bad in (x[:, 1].float(), x[:49, 1], x.transpose(0, 1)[1].transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(ValueError):
            cache.append(x[:, 0], bad, offsets([20, 30]))
    with pytest.raises(lime.LimeError):                              # row pitch of 65 elements
        cache.append(x[:, 0], torch.zeros(50 * 65, dtype=torch.bfloat16, device="cuda").as_strided(
            (50, 2, 32), (65, 32, 1)), offsets([20, 30]))
    assert cache.lens.tolist() == [0, 0] and int(cache.n_free) == 20
    for c in (cache, other):
        c.append(x[:, 0], x[:, 1], offsets([20, 30]))
    assert cache.lens.tolist() == [20, 30] and cache.status() == 0
    q = torch.randn(8, 2, 32, device="cuda").to(torch.bfloat16)
    assert torch.equal(cache.attend(q, offsets([4, 4])), other.attend(q, offsets([4, 4])))


def test_cache_keeps_its_flags_when_its_workspace_grows():
    dims = lime_kv.make_kv_dims(2, 2, 32, 16, 2, 4, "bf16")
    cache = lime_kv.HistoryCache(dims, 2)
    x = torch.randn(50, 2, 2, 32, device="cuda").to(torch.bfloat16)
    cache.append(x[:, 0], x[:, 1], offsets([20, 30]))                # two blocks: the second request is refused
    q = torch.randn(8, 2, 32, device="cuda").to(torch.bfloat16)
    O = cache.attend(q, offsets([4, 4]))
    assert cache.status() == lime_kv.LIME_FLAG_NO_BLOCKS and cache.status() == 0
    assert cache.lens.tolist() == [20, 0] and (O[4:] == 0).all() and (O[:4] != 0).any()
    graph = torch.cuda.CUDAGraph()
    more = torch.randn(80, 2, 32, device="cuda").to(torch.bfloat16)
    off = offsets([40, 40])
    with pytest.raises(ValueError, match="max_q"):                   # its workspace would belong to the graph
        with torch.cuda.graph(graph):
            cache.attend(more, off)
    assert torch.equal(cache.attend(more, off)[:1], cache.attend(more, off)[:1])


def test_calls_on_another_stream_and_in_a_graph():
    rng = np.random.default_rng(13)
    B, Hq, Hkv, dh, bs = 3, 4, 2, 64, 16
    dims = lime_kv.make_kv_dims(Hq, Hkv, dh, bs, 40, 12, "bf16")
    c = lime_kv.HistoryCache(dims, B, max_q=3 * B)
    x = torch.tensor(rng.standard_normal((60, 2, Hkv, dh))).to(torch.bfloat16).cuda()
    q = torch.tensor(rng.standard_normal((3 * B, Hq, dh))).to(torch.bfloat16).cuda()
    off, qoff = offsets([20, 39, 1]), offsets([3, 3, 3])
    slots = torch.empty(60, dtype=torch.int64, device="cuda")
    O, lens2, nf2 = torch.empty_like(q), c._lens, c._n_free

    def calls():
        lime_kv.lime_kv_reserve(dims, c.lens, off, c.table, c.free, c.n_free, lens2, nf2, slots, c.ws)
        lime_kv.lime_kv_append(dims, x[:, 0], x[:, 1], slots, c.k, c.v, c.scale, c.ws)
        lime_kv.lime_kv_attention(dims, q, qoff, c.table, lens2, c.k, c.v, c.scale, O, None, c.ws, causal=True)

    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        calls()
    side.synchronize()
    first = O.clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        calls()
    O.zero_()
    x.mul_(1.0)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, first)
    q.neg_()                                            # the graph reads what the tensors hold now
    g.replay()
    torch.cuda.synchronize()
    assert not torch.equal(O, first)
    calls()
    second = O.clone()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(O, second)
    assert c.status() == 0


_CAPTURE_FIRST = r"""
import torch
from recsys_decoupled_link_b200 import lime_kv

dims = lime_kv.make_kv_dims(4, 2, 32, 16, 40, 12, "bf16")
c = lime_kv.HistoryCache(dims, 3, max_q=96)
g = torch.Generator(device="cuda").manual_seed(1)
x = torch.randn(60, 2, 2, 32, device="cuda", generator=g).to(torch.bfloat16)
q = torch.randn(96, 4, 32, device="cuda", generator=g).to(torch.bfloat16)
off = torch.tensor([0, 20, 59, 60], device="cuda")
qoff = torch.tensor([0, 32, 64, 96], device="cuda")
slots, O = torch.empty(60, dtype=torch.int64, device="cuda"), torch.empty_like(q)

def calls():
    lime_kv.lime_kv_reserve(dims, c.lens, off, c.table, c.free, c.n_free, c._lens, c._n_free, slots, c.ws)
    lime_kv.lime_kv_append(dims, x[:, 0], x[:, 1], slots, c.k, c.v, c.scale, c.ws)
    lime_kv.lime_kv_attention(dims, q, qoff, c.table, c._lens, c.k, c.v, c.scale, O, None, c.ws)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls()
graph.replay()
torch.cuda.synchronize()
first = O.clone()
O.zero_()
calls()
assert c.status() == 0 and torch.equal(O, first) and bool((O != 0).any())
print("capture-first ok")
"""


def test_calls_captured_before_any_eager_call():
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    env = dict(os.environ, PYTHONPATH=root + os.pathsep + os.environ.get("PYTHONPATH", ""),
               CUDA_MODULE_LOADING="EAGER")
    r = subprocess.run([sys.executable, "-c", _CAPTURE_FIRST], cwd=root, env=env, capture_output=True, text=True,
                       timeout=600)
    assert r.returncode == 0 and "capture-first ok" in r.stdout, r.stdout + r.stderr
