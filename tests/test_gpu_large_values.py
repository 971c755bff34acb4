"""Caches with groups whose zero and scale are finite in fp16 but whose values are not (60000 ..
70000), or of a range of 2^17: the tree attention's fp16 operands have to be scaled down, whether the
values came by an append, a selected append or a fused step; tokens that a window hides have no
influence."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import kvq

import exact_attention as exact
import step_reference as ref
from test_gpu_softcap import check, f64
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


def step(x):
    """Half an fp16 step of the scaled operands: the exponent e is that of a group's |zero| + scale
    (2^b - 1), which is below 3.1 times the largest value (the zero and the range of min .. max).
    The scales and zeros of these inputs (above 2^-10, or zero) are scaled by 2^-e exactly."""
    return 2.0 ** (max(0, int(np.floor(np.log2(3.1 * np.abs(x).max()))) - 14) - 25)


def run(c, Kc, Vc, L, what, window=0, depth=None):
    """tree_attn against 64 bits over the oracle's values of the cached tokens Kc, Vc [Hkv, L, D]."""
    T = c.T
    Kh, Vh = ref.cached_values(Kc, Vc, L, *c.bits, c.kmode)
    assert np.isfinite(Kh).all() and np.isfinite(Vh).all()
    K, V = np.concatenate([Kh, f64(c.Kd[0])], 1), np.concatenate([Vh, f64(c.Vd[0])], 1)
    see = np.concatenate([np.ones((T, L), bool), np.tril(np.ones((T, T), bool))], 1)
    d = np.arange(T) if depth is None else f64(depth[0])
    pos = np.concatenate([np.arange(float(L)), L + d])
    r, e = exact.attention(f64(c.q[0]), K, V, see, pos[L:], pos, c.G, window=window, vstep=step(Vh), kstep=step(Kh))
    for S in (1, 2):
        kvq.kvq_set_num_splits(c.cache.h, S)
        out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, depth=depth, opts=kvq.ScoreOpts(window=window), out_fp32=True)
        check(out[0], r, e, f"{what} splits {S}")
    kvq.kvq_set_num_splits(c.cache.h, 0)
    assert kvq.kvq_device_status(c.cache.h) == 0


def ramp(shape, lo, hi, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (lo + (hi - lo) * torch.rand(shape, generator=g, device="cuda")).to(torch.bfloat16)


def refill(c, L):
    kvq.kvq_reset_sequences(c.cache.h, [0])
    c.cache.append(0, c.K[:, :, :L].contiguous(), c.V[:, :, :L].contiguous())


@pytest.mark.parametrize("bits", [(8, 8), (4, 2), (2, 4)])
@pytest.mark.parametrize("D,kmode,T", [(128, 0, 3), (64, 1, 12), (128, 1, 40), (64, 0, 20)])
def test_values(D, kmode, T, bits):
    L = 150
    c = Case([L], T, Hkv=1, D=D, bits=bits, kmode=kmode, seed=5)
    c.V[:, :, 20:60, :32] = ramp((1, 1, 40, 32), 60000, 70000, 1)
    c.V[:, :, 100:101, 32:64] = ramp((1, 1, 1, 32), -65000, 70000, 2)
    refill(c, L)
    run(c, c.K[0], c.V[0], L, "values")
    # the rows of a window that starts behind the large values get what the others hold
    run(c, c.K[0], c.V[0], L, "window", window=L - 101)


@pytest.mark.parametrize("bits", [(8, 8), (4, 2), (2, 4)])
@pytest.mark.parametrize("D,kmode,T", [(128, 0, 3), (64, 1, 12), (128, 1, 40), (64, 0, 20)])
def test_keys(D, kmode, T, bits):
    """Scores of order one: the queries are small, and zero in most of the large channels."""
    L = 150
    c = Case([L], T, Hkv=1, D=D, bits=bits, kmode=kmode, seed=6)
    c.K[:, :, 32:96, :8] = ramp((1, 1, 64, 8), 60000, 70000, 3)
    c.q[..., :8] = 0
    c.q[..., 3] = 2.0 ** -14
    refill(c, L)
    run(c, c.K[0], c.V[0], L, "keys")


@pytest.mark.parametrize("kmode", [0, 1])
def test_by_selected_append_and_fused_step(kmode):
    """A layer learns of its large values from every way in."""
    L, T, D = 70, 5, 128
    for way in ("selected", "fused"):
        c = Case([L], T, Hkv=1, D=D, bits=(8, 4), kmode=kmode, seed=7)
        Kn, Vn = (torch.randn((1, 1, 1, D), device="cuda").to(torch.bfloat16) for _ in range(2))
        Vn[..., :32] = ramp((1, 1, 1, 32), 60000, 70000, 4)
        if way == "selected":
            c.cache.append_selected(0, Kn, Vn, torch.zeros((1, 1), dtype=torch.int32, device="cuda"))
        else:
            out = c.cache.append_decode(0, Kn, Vn, c.q[:, 0].contiguous(), out_fp32=True)
            assert torch.isfinite(out).all()
        run(c, torch.cat([c.K[0], Kn[0]], 1), torch.cat([c.V[0], Vn[0]], 1), L + 1, way)


def test_layers_keep_their_own_bounds():
    """Large values in one layer leave another layer's bits as they were."""
    B, Hkv, G, D, L, T = 1, 1, 4, 128, 90, 4
    c = Case([L], T, Hkv=1, seed=8)
    cache = kvq.Cache(3, B, Hkv, Hkv * G, D, L + T, [(4, 2)] * 3)
    for layer in range(3):
        cache.append(layer, c.K, c.V)
    first = cache.tree_attn(1, c.q, c.Kd, c.Vd)
    big = c.V.clone()
    big[..., :32] = ramp((1, 1, L, 32), 60000, 70000, 5)
    for layer in (0, 2):
        kvq.kvq_truncate(cache.h, layer, 0)
        cache.append(layer, c.K, big)
        assert torch.isfinite(cache.tree_attn(layer, c.q, c.Kd, c.Vd)).all()
    assert torch.equal(cache.tree_attn(1, c.q, c.Kd, c.Vd), first)
