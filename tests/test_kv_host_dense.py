"""The dense 64-bit attention of the large GPU tests against the oracle's loops."""
import numpy as np
import pytest
import torch

import kv_dense
from oracle import kv_oracle as K


@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("Hq,Hkv", [(4, 4), (6, 2)])
def test_dense_attention_is_the_oracles(causal, Hq, Hkv):
    counts, lens, bs, dh = [3, 0, 40, 1, 7], [50, 9, 17, 0, 33], 16, 16
    table, k, v, scale = kv_dense.make_pool(lens, Hkv, dh, bs, 1, "cpu")
    table[0, 1], table[4, 0] = -1, 10 ** 6
    q = torch.randn(sum(counts), Hq, dh, generator=torch.Generator().manual_seed(2))
    args = (bs, -0.3, causal)
    got = kv_dense.attention(q, counts, table, lens, k, v, scale, *args)
    want = K.attention(q.double().numpy(), counts, table.numpy(), lens, k.numpy(), v.numpy(),
                       np.nan_to_num(scale.numpy()).astype(np.float64), *args)
    for name, g, w in zip(("O", "lse", "A", "S", "V"), got, want):
        np.testing.assert_allclose(g, w, rtol=1e-12, atol=1e-13, err_msg=name)
