"""Capped scores at caps from below the scores to far above them: the error may not grow with
the cap.  Attention far below the cap is attention without it."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import kvq

import exact_attention as exact
import step_reference as ref
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu

CAPS = [0.5, 20.0, 64.0, 65.0, 1e3, 1e5, 1e7, 1e30, 3.3e38, 1e-30, 1e-42]


def f64(x):
    return x.double().cpu().numpy()


def check(out, r, bound, what):
    o, half = f64(out), torch.finfo(out.dtype).eps / 2
    tol = bound * (1 + half) + half * np.abs(r)
    assert (np.abs(o - r) <= tol).all(), (what, float((np.abs(o - r) / np.maximum(tol, 1e-30)).max()))


@pytest.mark.parametrize("T,D,kmode", [(3, 128, 0), (9, 64, 1), (20, 128, 1), (40, 128, 0), (70, 64, 0)])
def test_tree(T, D, kmode):
    """Four, two and one copies of the rows, two row tiles; cached, open and drafted keys."""
    c = Case([203], T, Hkv=1, D=D, bits=(8, 4), kmode=kmode, seed=T)
    Kh, Vh = ref.cached_values(c.K[0], c.V[0], 203, 8, 4, kmode)
    K, V = np.concatenate([Kh, f64(c.Kd[0])], 1), np.concatenate([Vh, f64(c.Vd[0])], 1)
    see = np.concatenate([np.ones((T, 203), bool), np.tril(np.ones((T, T), bool))], 1)
    pos = np.concatenate([np.arange(203.0), 203 + np.arange(T)])
    for cap in CAPS:
        r, e = exact.attention(f64(c.q[0]), K, V, see, pos[203:], pos, c.G, cap=np.float64(np.float32(cap)),
                               vstep=2.0 ** -25)
        for S in (0, 2):
            kvq.kvq_set_num_splits(c.cache.h, S)
            out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, opts=kvq.ScoreOpts(cap), out_fp32=True)
            check(out[0], r, e, f"cap {cap} splits {S}")
    kvq.kvq_set_num_splits(c.cache.h, 0)
    assert kvq.kvq_device_status(c.cache.h) == 0


@pytest.mark.parametrize("G,D,kmode", [(4, 128, 0), (8, 64, 0), (4, 64, 1)])
def test_scored_decode(G, D, kmode):
    L = 203
    c = Case([L], 1, Hkv=1, G=G, D=D, bits=(8, 4), kmode=kmode, seed=G)
    Kh, Vh = ref.cached_values(c.K[0], c.V[0], L, 8, 4, kmode)
    kmax, vmax = np.abs(Kh).max(1), np.broadcast_to(np.abs(Vh).max((1, 2))[:, None], (1, D))
    if kmode:   # groups run over 32 channels of a token
        kmax = np.broadcast_to(np.abs(Kh).max((1, 2))[:, None], (1, D))
    for cap in CAPS:
        r, e = exact.attention(f64(c.q[0]), Kh, Vh, np.ones((1, L), bool), np.array([L - 1.0]), np.arange(float(L)), G,
                               cap=np.float64(np.float32(cap)), operands="fp32", kmax=kmax, vmax=vmax)
        out = c.cache.decode_attn_scored(0, c.q[:, 0].contiguous(), kvq.ScoreOpts(cap), out_fp32=True)
        check(out, r, e, f"cap {cap}")
