"""What a row of kvq_tree_attn sees comes out the same whatever the number of splits: NaN and
infinite drafted values whose weight is far below the row's largest."""
import pytest
import torch

from layer_wise_mixed_b200 import kvq

from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [3, 70])
@pytest.mark.parametrize("val", [float("inf"), -float("inf"), float("nan")])
def test_non_finite_values_of_little_weight(val, T):
    """The cached keys score 256 above the drafted ones (the weights' ratio is below fp32's
    smallest number): a drafted infinity still reaches the rows that see it, in its channel only,
    split or not."""
    L, D = 600, 64
    c = Case([L], T, Hkv=1, G=2, D=D, bits=(8, 8), kmode=1, seed=T)
    kvq.kvq_reset_sequences(c.cache.h, [0])
    c.cache.append(0, torch.full_like(c.K, 4.0), c.V)
    c.q.fill_(4.0)
    c.Kd.fill_(-4.0)
    at = 1
    c.Vd[:, :, at, 7] = val
    sees = torch.arange(T, device="cuda") >= at
    first = None
    for S in (1, 2, 3, 5):
        kvq.kvq_set_num_splits(c.cache.h, S)
        out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, out_fp32=True)[0]
        hit, rest = out[sees][:, :, 7], out.clone()
        assert (torch.isnan(hit) if val != val else hit == val).all(), S
        rest[sees, :, 7] = 0.0
        assert torch.isfinite(rest).all(), S
        first = rest if first is None else first
        # (the splits' partial sums differ by fp32 roundings of values up to 8)
        assert (rest - first).abs().max() <= 2.0 ** -18, S
    assert kvq.kvq_device_status(c.cache.h) == 0


def test_a_key_that_is_nan_reaches_every_split():
    """A visible NaN score makes its row NaN, split or not, and no other row."""
    c = Case([600], 5, Hkv=1, G=2, D=64, bits=(8, 8), kmode=1, seed=9)
    c.Kd[:, :, 2] = float("nan")
    for S in (1, 3):
        kvq.kvq_set_num_splits(c.cache.h, S)
        out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, out_fp32=True)[0]
        assert torch.isfinite(out[:2]).all() and torch.isnan(out[2:]).all(), S
