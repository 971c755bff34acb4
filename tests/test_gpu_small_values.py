"""Drafted values far below fp16's normal numbers, alone, beside ordinary ones in other tiles, and
beside cached tokens of either size: kvq_tree_attn keeps them to 2^-11, or to 2^-20 of the largest
value of their request and kv head."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import kvq

import exact_attention as exact
import step_reference as ref
from test_gpu_softcap import check, f64
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


def run(c, L, what, mask=None, splits=(1, 2, 3)):
    T = c.T
    Kh, Vh = ref.cached_values(c.K[0], c.V[0], L, *c.bits, c.kmode)
    K, V = np.concatenate([Kh, f64(c.Kd[0])], 1), np.concatenate([Vh, f64(c.Vd[0])], 1)
    tri = np.tril(np.ones((T, T), bool)) if mask is None else ref.mask_rows(mask[0], T)
    see = np.concatenate([np.ones((T, L), bool), tri], 1)
    pos = np.arange(float(L + T))
    # cached values are fp16 to 2^-11 or exact; drafted ones to the lesser of 2^-25 and 2^-20 of the
    # largest that the kernel looks at: all drafted ones and the open group's
    top = np.abs(np.concatenate([Vh[:, L // 32 * 32:], f64(c.Vd[0])], 1)).max()
    vstep = np.zeros(L + T)
    vstep[L:] = min(2.0 ** -25, 2.0 ** -20 * top)
    r, e = exact.attention(f64(c.q[0]), K, V, see, pos[L:], pos, c.G, vstep=vstep)
    for S in splits:
        kvq.kvq_set_num_splits(c.cache.h, S)
        out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, mask=mask, out_fp32=True)
        check(out[0], r, e, f"{what} splits {S}")
    kvq.kvq_set_num_splits(c.cache.h, 0)
    assert kvq.kvq_device_status(c.cache.h) == 0


@pytest.mark.parametrize("T,D", [(1, 128), (5, 64), (12, 128), (30, 64), (70, 128)])
@pytest.mark.parametrize("p", [-10, -20, -60, -110])
def test_alone(T, D, p):
    """No cached token: the output is a mean of the drafted values, whatever their size."""
    c = Case([0], T, Hkv=1, D=D, seed=T)
    c.Vd.mul_(2.0 ** p)
    run(c, 0, f"2^{p}")


@pytest.mark.parametrize("kmode", [0, 1])
@pytest.mark.parametrize("L", [77, 96, 300])
@pytest.mark.parametrize("cached,drafted", [(0, -20), (-12, -20), (-20, -20), (-20, 0), (-20, -60), (-20, 13)])
def test_beside_cached_tokens(cached, drafted, L, kmode):
    """Cached values of one size, drafted ones of another; with and without an open key group."""
    for T in (3, 40):
        c = Case([L], T, Hkv=1, kmode=kmode, bits=(8, 8), seed=L + T)
        c.V.mul_(2.0 ** cached)
        c.Vd.mul_(2.0 ** drafted)
        kvq.kvq_reset_sequences(c.cache.h, [0])
        c.cache.append(0, c.K, c.V)
        run(c, L, f"cached 2^{cached}, drafted 2^{drafted}, T={T}")


@pytest.mark.parametrize("T,G", [(300, 1), (300, 4), (140, 8)])
@pytest.mark.parametrize("sizes", [(-20, 0, -30), (0, -20, 3), (-40, -20, -3), (-110, -110, 12)])
def test_tiles_of_different_sizes(sizes, T, G):
    """The open tiles' exponent follows the largest value so far; zeros change nothing."""
    L = 50
    c = Case([L], T, Hkv=1, G=G, D=64, seed=T + G)
    c.Vd[:, :, :100].mul_(2.0 ** sizes[0])
    c.Vd[:, :, 100:230].mul_(2.0 ** sizes[1])
    c.Vd[:, :, 230:].mul_(2.0 ** sizes[2])
    run(c, L, str(sizes), splits=(1, 3))
    c.Vd[:, :, :128] = 0
    run(c, L, f"zeros, {sizes}", splits=(1, 3))


def test_non_finite_values_do_not_count():
    """An infinite value that no row sees leaves the small ones as they are."""
    c = Case([0], 20, Hkv=1, seed=2)
    c.Vd.mul_(2.0 ** -20)
    vis = np.tril(np.ones((1, 20, 20), bool))
    vis[:, :, 6] = False
    vis[:, 6, 5] = True
    mask = ref.pack_mask(vis)
    run(c, 0, "finite", mask)
    first = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, mask=mask)
    c.Vd[:, :, 6] = float("inf")
    assert torch.equal(c.cache.tree_attn(0, c.q, c.Kd, c.Vd, mask=mask), first)
