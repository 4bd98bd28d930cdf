"""Attention over scales at the ends of fp32's range, against the fp64 oracle.

Tolerances are those of test_gpu_kv.py's module text; where outputs are near or
below fp32's smallest normal number, each of the value's few roundings (a join
of four warps' parts, the scale, the last product) may lose half of fp32's
smallest step besides: 16 of them are allowed, and half of the output type's.
"""
import numpy as np
import pytest
import torch

from oracle import kv_oracle as K
from recsys_decoupled_link_b200 import lime, lime_kv
from test_gpu_kv import DT, U, assert_near, check_attention, f64, i32, make_pool, offsets

pytestmark = pytest.mark.gpu


def near_the_largest(low):
    """Codes of at most 3 keep the outputs finite; one block of request 0 and all of request 1 lie near
    the largest float, the others at `low`."""
    def hook(table, codes, scale, q):
        codes[1] = np.clip(codes[1], -3, 3)
        held = table[0][table[0] >= 0]
        scale[held, :, 1] = np.float32(low)
        scale[held[len(held) // 2], :, 1] = 1.1e38
        if len(table) > 1:
            scale[table[1][table[1] >= 0], :, 1] = 1e38
    return hook


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", [9e37, 1e30, 1.0])
def test_attention_value_scales_near_the_largest_float(dtype, low):
    for n, m, dh in ((100, 5, 32), (13, 40, 32), (100, 1, 128), (200, 3, 64)):
        check_attention([m], [n], 4, 2, dh, 16, dtype, hook=near_the_largest(low))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("low", [9e37, 1e30, 1.0])
def test_attention_joins_values_near_the_largest_float(dtype, low):
    # rows cut at workers' borders: short ones, and one over many workers (more than are joined at a time)
    check_attention([5, 40], [100, 13], 4, 2, 32, 16, dtype, hook=near_the_largest(low))
    check_attention([1, 1], [100, 13], 4, 2, 128, 16, dtype, hook=near_the_largest(low), seed=1)
    check_attention([3], [7001], 4, 2, 64, 64, dtype, hook=near_the_largest(low), seed=2)
    check_attention([2, 33], [9000, 70], 2, 1, 32, 64, dtype, hook=near_the_largest(low), seed=3, causal=True)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("dh", [32, 128])
@pytest.mark.parametrize("unit,low", [(1e-39, 1e-39), (1e-39, 1e-41), (3e-38, 1e-39), (1e-41, 1e-42)])
def test_attention_value_scales_below_the_normal_range(dtype, dh, unit, low):
    rng = np.random.default_rng(7)
    counts, lens, bs = [3, 1], [50, 9], 16
    table, codes, scale = make_pool(rng, lens, 2, dh, bs)
    scale[table[0, :4], :, 1] = np.float32(low)
    scale[table[0, 1], :, 1] = scale[table[1, 0], :, 1] = np.float32(unit)
    scale = np.nan_to_num(scale)
    q = torch.tensor(rng.standard_normal((4, 4, dh))).to(DT[dtype])
    dims = lime_kv.make_kv_dims(4, 2, dh, bs, codes.shape[1], table.shape[1], dtype)
    ws = lime_kv.KvWorkspace(dims, 2, 4)
    O, lse = torch.empty(4, 4, dh, dtype=q.dtype, device="cuda"), torch.empty(4, 4, device="cuda")
    lime_kv.lime_kv_attention(dims, q.cuda(), offsets(counts), i32(table), i32(lens),
                              torch.tensor(codes[0], device="cuda"), torch.tensor(codes[1], device="cuda"),
                              torch.tensor(scale, device="cuda"), O, lse, ws)
    assert lime.lime_get_status(ws) == 0
    ref, rl, A, S, V = K.attention(f64(q), counts, table, lens, codes[0], codes[1], scale.astype(np.float64), bs,
                                   dh ** -0.5, False)
    ds = S * (dh + 8) * 2 * U
    p, half, least = (2.0 ** -11, 2.0 ** -8, 2.0 ** -134) if dtype == "bf16" else (2.0 ** -21, U, 2.0 ** -150)
    tol = 2 * A * ((2 * ds + 8 * U + 2 * U * 50)[..., None] + p) + 50 * 2.0 ** -39 * V + half * np.abs(ref) \
        + 16 * 2.0 ** -150 + least
    err = np.abs(f64(O) - ref)
    assert (err <= tol).all(), (err / tol).max()
    assert np.abs(ref).max() > 0.3 * unit


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("top,exact", [(2.0 ** 20, True), (2.0 ** 30, False), (2.0 ** 33, False)])
def test_attention_one_huge_query_dim_over_zero_keys(dtype, causal, top, exact):
    """A row's largest element m sets the step of all others: 2^-39 m at most, which moves a score by
    sm_scale 2^-39 m sum_d |k_d| although the keys are 0 there.  bf16 elements from 2^-31 m on are exact."""
    rng = np.random.default_rng(11)
    counts, lens, bs, dh, Hq, Hkv = [20, 1, 7], [300, 40, 5], 16, 32, 4, 2
    table, codes, scale = make_pool(rng, lens, Hkv, dh, bs)
    codes[0, ..., 3] = 0
    q = rng.standard_normal((28, Hq, dh))
    q = np.sign(q) * (0.25 + np.abs(q))
    q[..., 3] = top * rng.choice([-1.0, 1.0], (28, Hq))
    q = torch.tensor(q).to(DT[dtype])
    dims = lime_kv.make_kv_dims(Hq, Hkv, dh, bs, codes.shape[1], table.shape[1], dtype)
    ws = lime_kv.KvWorkspace(dims, 3, 28)
    O, lse = torch.empty(28, Hq, dh, dtype=q.dtype, device="cuda"), torch.empty(28, Hq, device="cuda")
    lime_kv.lime_kv_attention(dims, q.cuda(), offsets(counts), i32(table), i32(lens),
                              torch.tensor(codes[0], device="cuda"), torch.tensor(codes[1], device="cuda"),
                              torch.tensor(scale, device="cuda"), O, lse, ws, causal=causal)
    assert lime.lime_get_status(ws) == 0
    finite = np.nan_to_num(scale).astype(np.float64)
    ref, rl, A, S, V = K.attention(f64(q), counts, table, lens, codes[0], codes[1], finite, bs, dh ** -0.5, causal)
    # |k_d| summed over the dims: S of a query of ones
    ones = K.attention(np.ones((28, Hq, dh)), counts, table, lens, codes[0], codes[1], finite, bs, dh ** -0.5,
                       causal)[3]
    step = np.zeros_like(S) if exact and dtype == "bf16" else 2.0 ** -39 * top * ones
    # test_gpu_kv.py's bound takes a score to be off by S (dh + 8) 2u
    assert_near(O, lse, ref, rl, A, S + step / ((dh + 8) * 2 * U), V, max(lens), dh, dtype)
