"""kvq_norm_rope against the formula in 64 bits: head layouts, lengths, pair orders, partial
rotation, padded rows, far positions, ragged requests."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import kvq

import step_reference as ref

pytestmark = pytest.mark.gpu


def run(B, n, Hkv, G, D, lens, rot, inter, norm, far=None, pad=0, seed=0):
    Hq, W = Hkv * G, (Hkv * G + 2 * Hkv) * D
    g = torch.Generator(device="cuda").manual_seed(seed)
    cache = kvq.Cache(1, B, Hkv, Hq, D, max(max(lens), 1), [(2, 2)])
    if max(lens):
        z = torch.zeros((B, Hkv, max(lens), D), dtype=torch.bfloat16, device="cuda")
        cache.append_ragged(0, z, z, lens)
    x = torch.randn((B, n, W + pad), generator=g, device="cuda").to(torch.bfloat16)
    inv = (1e4 ** (-torch.arange(0, max(rot, 2), 2, device="cuda", dtype=torch.float64) / max(rot, 2))).float()
    wq = 1 + 0.3 * torch.randn(D, generator=g, device="cuda") if norm else None
    wk = 1 + 0.3 * torch.randn(D, generator=g, device="cuda") if norm else None
    off = None
    if far is not None:
        off = torch.randint(far, far + 50, (B, n), generator=g, device="cuda", dtype=torch.int32)
    rope = kvq.Rope(rot, inv, wq, wk, 1e-6, inter)
    q, K, V = cache.norm_rope(0, x[:, :, :W], rope, off)
    torch.cuda.synchronize()
    f = lambda t: t.double().cpu().numpy()
    xr = f(x[:, :, :W]).reshape(B, n, Hq + 2 * Hkv, D)
    pos = np.array(lens, np.float64)[:, None] + (np.arange(n)[None] if off is None else f(off))
    qr = ref.norm_rope(xr[:, :, :Hq], None if wq is None else f(wq), pos[:, :, None], f(inv), rot, inter, 1e-6)
    kr = ref.norm_rope(xr[:, :, Hq:Hq + Hkv], None if wk is None else f(wk), pos[:, :, None], f(inv), rot, inter, 1e-6)
    # One rounding to bf16 (2^-8 of the value at most, half a step) on top of fp32 work: the
    # norm's factor and products are off by less than 2^-19 of the pair's size, an angle by
    # less than 2^-20 (fp32 of the reduced turns, sine and cosine within 2 ulp)
    def close(a, r, size):
        assert (np.abs(f(a) - r) <= 2.0 ** -8 * np.abs(r) + 2.0 ** -18 * size).all(), np.abs(f(a) - r).max()
    close(q, qr, np.abs(qr).max())
    close(K, kr.transpose(0, 2, 1, 3), np.abs(kr).max())
    assert torch.equal(V, x[:, :, :W].reshape(B, n, -1, D)[:, :, Hq + Hkv:].transpose(1, 2))
    if not norm:   # channels behind the rotated ones come out as they went in
        assert torch.equal(q[..., rot:], x[:, :, :W].reshape(B, n, -1, D)[:, :, :Hq, rot:])


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 32, 48, 64, 128])
def test_rotation(D, inter, norm, rot):
    if rot <= D:
        run(2, 5, 2, 4, D, [37, 37], rot, inter, norm, seed=rot)


@pytest.mark.parametrize("Hkv,G", [(1, 1), (1, 8), (2, 3), (4, 7), (8, 4), (16, 1), (1, 5)])
@pytest.mark.parametrize("n", [1, 3, 40])
def test_head_layouts(Hkv, G, n):
    run(3, n, Hkv, G, 128, [9, 0, 200], 128, False, True, pad=24, seed=n)
    run(1, n, Hkv, G, 64, [65], 32, True, False, seed=n)


@pytest.mark.parametrize("far", [0, 4095, 131072, 2 ** 30 - 100])
def test_far_positions(far):
    run(2, 6, 2, 2, 128, [3, 3], 128, False, True, far=far, seed=far & 1023)


def test_large_batch_ragged():
    rng = np.random.default_rng(0)
    run(70, 2, 1, 2, 64, [int(v) for v in rng.integers(0, 90, 70)], 64, False, True)


def test_long_prompt():
    run(2, 3001, 2, 4, 128, [0, 0], 128, False, True)


def test_strided_rows_of_a_larger_buffer():
    """Rows of every second token of a buffer (token stride twice the row), and one buffer
    row shared by all requests of a batch (batch stride 0 is the caller's right in C)."""
    B, n, Hkv, G, D = 2, 4, 1, 2, 64
    W = (Hkv * G + 2 * Hkv) * D
    cache = kvq.Cache(1, B, Hkv, Hkv * G, D, 8, [(2, 2)])
    x = torch.randn((B, 2 * n, W), device="cuda").to(torch.bfloat16)
    rope = kvq.Rope(64, torch.rand(32, device="cuda"))
    a = cache.norm_rope(0, x[:, ::2], rope)
    b = cache.norm_rope(0, x[:, ::2].contiguous(), rope)
    assert all(torch.equal(u, v) for u, v in zip(a, b))
    q, K, V = (torch.empty_like(t) for t in a)
    kvq.kvq_norm_rope(cache.h, 0, x[0, ::2], 0, 2 * W, n, None, rope, q, K, V)
    both = cache.norm_rope(0, x[:1, ::2].expand(B, -1, -1).contiguous(), rope)
    assert all(torch.equal(u, v) for u, v in zip((q, K, V), both))
