"""kvq_append_selected and kvq_read, and a run of the step operators together: the cache
after a selected append is byte-equal to one that got the same tokens in order, reads
equal the oracle's values rounded to bf16."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import inputs, kvq

import step_reference as ref
from test_gpu_parity import workload

pytestmark = pytest.mark.gpu


def as_bf16(x):
    """float64 numpy (exact values) -> bf16, by way of the format's fp32 FMA result."""
    return torch.from_numpy(x).float().to(torch.bfloat16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kmode", [0, 1])
@pytest.mark.parametrize("bk", [2, 4, 8])
@pytest.mark.parametrize("bv", [2, 4, 8])
def test_read_every_format(D, kmode, bk, bv):
    B, Hkv, L = 2, 3, 75
    wl = workload(B, Hkv, 1, D, name=f"read{D}{kmode}{bk}{bv}")
    K, V = inputs.layer_kv(wl, 0, L, "cuda")
    cache = kvq.Cache(1, B, Hkv, Hkv, D, L, [(bk, bv)], kmodes=[kmode])
    cache.append(0, K, V)
    Ko, Vo = cache.read(0, 0, L)
    for b in range(B):
        Kh, Vh = ref.cached_values(K[b], V[b], L, bk, bv, kmode)
        assert torch.equal(Ko[b].cpu(), as_bf16(Kh)) and torch.equal(Vo[b].cpu(), as_bf16(Vh))


@pytest.mark.parametrize("pool", [0, 60])
@pytest.mark.parametrize("kmode", [0, 1])
def test_read_ranges_of_ragged_requests(kmode, pool):
    lens = [200, 33, 0, 64, 131]
    B, Hkv, D = 5, 2, 128
    wl = workload(B, Hkv, 2, D, name="readrange")
    K, V = inputs.layer_kv(wl, 0, 200, "cuda")
    cache = kvq.Cache(1, B, Hkv, 2 * Hkv, D, 224, [(4, 2)], kmodes=[kmode], pool_blocks=pool)
    cache.append_ragged(0, K, V, lens)
    vals = [ref.cached_values(K[b], V[b], lens[b], 4, 2, kmode) for b in range(B)]
    for t0, n in ((0, 200), (0, 1), (199, 1), (31, 2), (32, 32), (17, 100), (130, 70), (63, 65)):
        Ko = torch.full((B, Hkv, n, D), 9.0, dtype=torch.bfloat16, device="cuda")
        Vo = torch.full_like(Ko, 9.0)
        cache.read(0, t0, n, Ko, Vo)
        K1 = torch.full_like(Ko, 9.0)
        kvq.kvq_read(cache.h, 0, t0, n, K1, None)
        assert torch.equal(K1, Ko)
        for b in range(B):
            m = max(0, min(lens[b] - t0, n))
            assert torch.equal(Ko[b, :, :m].cpu(), as_bf16(vals[b][0][:, t0:t0 + m]))
            assert torch.equal(Vo[b, :, :m].cpu(), as_bf16(vals[b][1][:, t0:t0 + m]))
            assert (Ko[b, :, m:] == 9.0).all() and (Vo[b, :, m:] == 9.0).all()


@pytest.mark.parametrize("kmode,pool", [(0, 0), (1, 0), (0, 40)])
def test_selected_append_equals_plain_append(kmode, pool):
    """Gathered appends (out of order, the same slot twice, none at all, group completions)
    give the bytes of appending the gathered tokens."""
    B, Hkv, D, n_src, n_max = 4, 2, 128, 50, 40
    wl = workload(B, Hkv, 2, D, name="selected")
    K, V = inputs.layer_kv(wl, 0, 100, "cuda")
    Ks, Vs = inputs.layer_kv(wl, 0, n_src, "cuda", tag="src")
    caches = [kvq.Cache(1, B, Hkv, 2 * Hkv, D, 260, [(4, 8)], kmodes=[kmode], pool_blocks=pool) for _ in range(2)]
    for c in caches:
        c.append_ragged(0, K, V, [100, 3, 0, 60])
    rng = np.random.default_rng(kmode)
    for counts in ([3, 0, 40, 5], [1, 1, 1, 1], [40, 33, 0, 7], None):
        index = torch.from_numpy(rng.integers(0, n_src, (B, n_max)).astype(np.int32)).cuda()
        caches[0].append_selected(0, Ks, Vs, index, counts)
        rows = index.long()[:, None, :, None].expand(B, Hkv, n_max, D)
        caches[1].append_ragged(0, Ks.gather(2, rows), Vs.gather(2, rows), [n_max] * B if counts is None else counts)
        assert np.array_equal(caches[0].export_layer(0), caches[1].export_layer(0))
        assert list(caches[0].seq_lens(0)) == list(caches[1].seq_lens(0))
    assert kvq.kvq_device_status(caches[0].h) == 0


def test_selected_append_above_the_parameter_tables():
    B, Hkv, D = 70, 1, 64
    wl = workload(B, Hkv, 1, D, name="selected70")
    Ks, Vs = inputs.layer_kv(wl, 0, 9, "cuda")
    rng = np.random.default_rng(1)
    index = torch.from_numpy(rng.integers(0, 9, (B, 6)).astype(np.int32)).cuda()
    counts = [int(x) for x in rng.integers(0, 7, B)]
    a, b = (kvq.Cache(1, B, Hkv, Hkv, D, 32, [(8, 8)]) for _ in range(2))
    a.append_selected(0, Ks, Vs, index, counts)
    rows = index.long()[:, None, :, None].expand(B, Hkv, 6, D)
    b.append_ragged(0, Ks.gather(2, rows), Vs.gather(2, rows), counts)
    assert np.array_equal(a.export_layer(0), b.export_layer(0))


def test_slot_outside_its_source_is_reported():
    """The kernel bounds-checks every slot: a bad one is reported and slot 0 taken."""
    B, Hkv, D = 1, 1, 64
    wl = workload(B, Hkv, 1, D, name="badslot")
    Ks, Vs = inputs.layer_kv(wl, 0, 4, "cuda")
    for bad in (4, -1, 2 ** 31 - 1):
        a, b = (kvq.Cache(1, B, Hkv, Hkv, D, 32, [(8, 8)]) for _ in range(2))
        a.append_selected(0, Ks, Vs, torch.tensor([[1, bad, 2]], dtype=torch.int32, device="cuda"))
        with pytest.raises(kvq.KvqError) as e:
            kvq.kvq_device_status(a.h)
        assert e.value.code == kvq.KVQ_EDEVICE and "slot" in str(e.value)
        assert kvq.kvq_device_status(a.h) == 0
        b.append_selected(0, Ks, Vs, torch.tensor([[1, 0, 2]], dtype=torch.int32, device="cuda"))
        assert np.array_equal(a.export_layer(0), b.export_layer(0))


@pytest.mark.parametrize("kmode", [0, 1])
def test_a_run_of_steps(kmode):
    """Three speculative steps over two layers as a serving loop makes them: norm + rotation
    of the drafted tokens, tree attention, append of the accepted path, then a plain decode
    step; attention within its bound, the cache equal to one that was fed the accepted
    tokens, the read-back equal to the oracle's values."""
    B, Hkv, G, D, T, NL = 2, 2, 4, 128, 12, 2
    Hq, W = Hkv * G, (Hkv * G + 2 * Hkv) * D
    g = torch.Generator(device="cuda").manual_seed(kmode)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
    bits = [(8, 4), (4, 2)]
    cache = kvq.Cache(NL, B, Hkv, Hq, D, 200, bits, kmodes=[kmode] * NL)
    inv = (1e4 ** (-torch.arange(0, D, 2, device="cuda") / D)).float()
    w = torch.ones(D, device="cuda")
    rope = kvq.Rope(D, inv, w, w)
    hist = [[[rnd(0, 0), rnd(0, 0)] for _ in range(B)] for _ in range(NL)]
    lens = [40, 61]
    for l in range(NL):
        _, K, V = cache.norm_rope(l, rnd(B, 61, W), rope)
        cache.append_ragged(l, K, V, lens)
        for b in range(B):
            hist[l][b] = [K[b, :, :lens[b]], V[b, :, :lens[b]]]
    rng = np.random.default_rng(kmode)
    for step in range(3):
        mask, depth = ref.random_tree(B, T, step)
        paths = []
        for b in range(B):   # accept the ancestors of some drafted token
            leaf = int(rng.integers(0, T))
            paths.append(np.flatnonzero(ref.mask_rows(mask[b], T)[leaf]))
        n_new = [len(x) for x in paths]
        index = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        for b in range(B):
            index[b, :n_new[b]] = torch.from_numpy(paths[b].astype(np.int32)).cuda()
        for l in range(NL):
            q, K, V = cache.norm_rope(l, rnd(B, T, W), rope, depth)
            out = cache.tree_attn(l, q, K, V, None, mask, depth)
            for b in range(B):
                Kh, Vh = ref.cached_values(*hist[l][b], lens[b], *bits[l], kmode)
                f = lambda x: x.double().cpu().numpy()
                d = f(depth[b])
                r, e = ref.attention(f(q[b]), Kh, Vh, f(K[b]), f(V[b]), ref.mask_rows(mask[b], T), lens[b] + d, lens[b] + d,
                                     lens[b], G)
                ref.check(out[b], r, e, f"step {step} layer {l} request {b}")
                take = torch.from_numpy(paths[b]).cuda()
                hist[l][b] = [torch.cat([hist[l][b][i], (K, V)[i][b][:, take]], 1) for i in (0, 1)]
            cache.append_selected(l, K, V, index, n_new)
        lens = [L + n for L, n in zip(lens, n_new)]
    for l in range(NL):
        assert list(cache.seq_lens(l)) == lens
        Ko, Vo = cache.read(l, 0, max(lens))
        o = cache.decode_attn(l, rnd(B, Hq, D), out_fp32=True)
        assert torch.isfinite(o).all()
        for b in range(B):
            Kh, Vh = ref.cached_values(*hist[l][b], lens[b], *bits[l], kmode)
            assert torch.equal(Ko[b, :, :lens[b]].cpu(), as_bf16(Kh)) and torch.equal(Vo[b, :, :lens[b]].cpu(), as_bf16(Vh))
    assert kvq.kvq_device_status(cache.h) == 0
