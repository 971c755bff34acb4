"""An infinite or NaN value appended to one request leaves the attention of the others, bit for bit."""
import pytest
import torch

from layer_wise_mixed_b200 import kvq

from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("val", [float("inf"), -float("inf"), float("nan"), 3e38, -7e4])
@pytest.mark.parametrize("kmode", [0, 1])
def test_other_requests_keep_their_bits(kmode, val):
    L, T = 70, 6
    c = Case([L, L, L], T, kmode=kmode, bits=(8, 8), seed=4)
    c.V[1].mul_(2.0 ** -6)   # (small scales: a scaling of the layer would cost them bits)
    kvq.kvq_reset_sequences(c.cache.h, [0, 1, 2])
    c.cache.append(0, c.K, c.V)
    tree = c.cache.tree_attn(0, c.q, c.Kd, c.Vd)
    Kn, Vn = c.K[:, :, :1].contiguous(), c.V[:, :, :1].contiguous()
    Vn[0, 0, 0, 5] = val
    Kn[0, 1, 0, 7] = val
    c.cache.append_ragged(0, Kn, Vn, [1, 0, 0])
    assert torch.equal(c.cache.tree_attn(0, c.q, c.Kd, c.Vd)[1:], tree[1:])
    assert kvq.kvq_device_status(c.cache.h) == 0
