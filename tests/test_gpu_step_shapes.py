"""The step operators' attention element by element against 64 bits, with bounds derived key by key
(exact_attention), where the instances of the kernels differ: every bit pair and key mode in each
form of the tree kernel, cap, bias, window and scale in each, scored decode at fp32-level accuracy
for every group size, pools and ragged batches of any size."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import kvq

import exact_attention as exact
import step_reference as ref
from test_gpu_softcap import check, f64
from test_gpu_tree import Case

pytestmark = pytest.mark.gpu

# rows per kv head at four query heads each: four, two, one copies of the rows, two row tiles
TOKENS = [6, 13, 30, 40]


def tree(c, what, n_draft=None, mask=None, depth=None, splits=(0,), **o):
    want = []
    for b, L in enumerate(c.lens):
        t = c.T if n_draft is None else n_draft[b]
        Kh, Vh = ref.cached_values(c.K[b], c.V[b], L, *c.bits, c.kmode)
        K, V = (np.concatenate([a, f64(x[b, :, :t])], 1) for a, x in ((Kh, c.Kd), (Vh, c.Vd)))
        d = np.arange(t) if depth is None else f64(depth[b, :t])
        drafted = np.tril(np.ones((t, t), bool)) if mask is None else ref.mask_rows(mask[b], c.T)[:t, :t]
        see = np.concatenate([np.ones((t, L), bool), drafted], 1)
        oo = {**o, "alibi": None if o.get("alibi") is None else f64(o["alibi"])}
        want.append(exact.attention(f64(c.q[b, :t]), K, V, see, L + d, np.concatenate([np.arange(float(L)), L + d]), c.G,
                                    vstep=2.0 ** -25, **oo))
    opts = kvq.ScoreOpts(o.get("cap", 0.0), o.get("alibi"), o.get("window", 0), o.get("scale", 0.0))
    for S in splits:
        kvq.kvq_set_num_splits(c.cache.h, S)
        for fp32 in (True, False):
            out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, n_draft, mask, depth, opts, out_fp32=fp32)
            for b, (r, e) in enumerate(want):
                check(out[b, :len(r)], r, e, f"{what} splits {S} fp32 {fp32} request {b} L={c.lens[b]}")
    kvq.kvq_set_num_splits(c.cache.h, 0)
    assert kvq.kvq_device_status(c.cache.h) == 0


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("D,kmode", [(64, 0), (64, 1), (128, 0), (128, 1)])
def test_bit_pairs(D, kmode, T):
    for bk in (2, 4, 8):
        for bv in (2, 4, 8):
            tree(Case([203], T, Hkv=1, D=D, bits=(bk, bv), kmode=kmode, seed=10 * bk + bv), f"K{bk}V{bv}")


@pytest.mark.parametrize("T", TOKENS)
@pytest.mark.parametrize("D,kmode", [(64, 0), (128, 0), (128, 1)])
def test_score_shapes(D, kmode, T):
    c = Case([333, 40, 0], T, Hkv=1, D=D, kmode=kmode, bits=(8, 4), seed=D + kmode + T)
    mask, depth = ref.random_tree(3, T, T)
    slopes = torch.tensor([0.5, 0.25, -0.03, 0.0], device="cuda")
    nd = [T, max(T - 4, 1), T // 2]
    for kw in (dict(cap=5.0), dict(window=7), dict(window=130, cap=20.0), dict(alibi=slopes),
               dict(alibi=slopes, cap=30.0, window=50), dict(scale=0.2), dict(scale=-0.1, cap=3.0), dict(scale=-0.15)):
        tree(c, str(sorted(kw)), nd, mask, depth, (0, 3), **kw)
    tree(c, "chunk", cap=8.0, window=5)


@pytest.mark.parametrize("G", [1, 3, 5, 6, 7, 8])
def test_head_groups(G):
    """Row tiles that end inside a token's heads, in each form of the kernel."""
    for T in (4, 9, 17, 37):
        c = Case([100, 41], T, Hkv=2, G=G, D=64, bits=(4, 8), seed=G + T)
        mask, depth = ref.random_tree(2, T, G)
        slopes = torch.tensor([2.0 ** -(i % 8 + 1) for i in range(2 * G)], device="cuda")
        tree(c, f"G={G} T={T}", [T, T // 2], mask, depth, (0, 2), alibi=slopes)


def decode(c, lens, what, splits=(0, 3), requests=None, **o):
    kwn = {**o, "alibi": None if o.get("alibi") is None else f64(o["alibi"])}
    want = {}
    for b in range(len(lens)) if requests is None else requests:
        L = lens[b]
        Kh, Vh = ref.cached_values(c.K[b], c.V[b], L, *c.bits, c.kmode)
        kmax = np.abs(Kh).max(1) if c.kmode == 0 else np.broadcast_to(np.abs(Kh).max((1, 2))[:, None], (c.Hkv, c.D))
        vmax = np.broadcast_to(np.abs(Vh).max((1, 2))[:, None], (c.Hkv, c.D))
        want[b] = exact.attention(f64(c.q[b, :1]), Kh, Vh, np.ones((1, L), bool), np.array([L - 1.0]), np.arange(float(L)),
                                  c.G, operands="fp32", kmax=kmax, vmax=vmax, **kwn)
    opts = kvq.ScoreOpts(o.get("cap", 0.0), o.get("alibi"), o.get("window", 0), o.get("scale", 0.0))
    for S in splits:
        kvq.kvq_set_num_splits(c.cache.h, S)
        for fp32 in (True, False):
            out = c.cache.decode_attn_scored(0, c.q[:, 0].contiguous(), opts, out_fp32=fp32)
            for b, (r, e) in want.items():
                check(out[b:b + 1], r, e, f"{what} splits {S} fp32 {fp32} request {b} L={lens[b]}")
    kvq.kvq_set_num_splits(c.cache.h, 0)
    assert kvq.kvq_device_status(c.cache.h) == 0


SHAPES = [dict(), dict(cap=6.0), dict(cap=50.0, window=40), dict(window=1), dict(window=130), dict(scale=-0.1),
          dict(scale=0.3, cap=4.0)]


@pytest.mark.parametrize("kmode,G", [(0, g) for g in range(1, 9)] + [(1, 1), (1, 2), (1, 4)])
def test_scored_decode_heads(kmode, G):
    for D, lens in ((128, [300, 45, 1]), (64, [33, 129, 640])):
        c = Case(lens, 1, G=G, D=D, kmode=kmode, bits=(8, 4), seed=sum(lens) + G)
        slopes = torch.tensor([(-1) ** i * 2.0 ** -(i % 8 + 1) for i in range(c.Hkv * G)], device="cuda")
        for kw in SHAPES + [dict(alibi=slopes), dict(alibi=slopes, cap=9.0, window=77)]:
            decode(c, lens, f"G={G} {sorted(kw)}", **kw)


@pytest.mark.parametrize("D,kmode,G", [(64, 0, 4), (128, 0, 4), (128, 0, 7), (64, 1, 4), (128, 1, 2)])
def test_scored_decode_bit_pairs(D, kmode, G):
    slopes = torch.tensor([2.0 ** -(i % 8 + 1) for i in range(G)], device="cuda")
    for bk in (2, 4, 8):
        for bv in (2, 4, 8):
            c = Case([203, 64], 1, Hkv=1, G=G, D=D, bits=(bk, bv), kmode=kmode, seed=10 * bk + bv)
            decode(c, [203, 64], f"K{bk}V{bv}", alibi=slopes, cap=12.0, window=150)


def test_scored_decode_pools_and_many_requests():
    rng = np.random.default_rng(4)
    lens = [int(x) for x in rng.integers(1, 200, 70)]
    slopes = torch.tensor([0.5, 0.1], device="cuda")
    for pool in (0, 500):
        c = Case(lens, 1, Hkv=1, G=2, D=64, pool=pool, seed=70)
        decode(c, lens, f"pool {pool}", requests=range(0, 70, 9), alibi=slopes, window=90)


def test_decode_without_options_is_decode_attn():
    """No cap, bias or window: both calls are within fp32-level accuracy of the same values."""
    for D, G, kmode in ((128, 4, 0), (64, 7, 0), (128, 2, 1)):
        lens = [500, 33]
        c = Case(lens, 1, G=G, D=D, kmode=kmode, bits=(4, 4), seed=G)
        a = c.cache.decode_attn_scored(0, c.q[:, 0].contiguous(), None, out_fp32=True)
        d = c.cache.decode_attn(0, c.q[:, 0].contiguous(), out_fp32=True)
        assert (a - d).norm() <= 4e-6 * d.norm()


@pytest.mark.parametrize("seed", range(24))
def test_random_cases(seed):
    """Shapes, lengths, formats and options drawn together."""
    rng = np.random.default_rng(seed)
    pick = lambda *x: x[int(rng.integers(len(x)))]
    kmode = pick(0, 0, 1)
    G, D, Hkv = pick(1, 2, 4) if kmode else int(rng.integers(1, 9)), pick(64, 128), pick(1, 2, 3)
    B, T = int(rng.integers(1, 5)), int(np.exp(rng.uniform(0, np.log(150))))
    lens = [int(np.exp(rng.uniform(0, np.log(1500)))) - 1 for _ in range(B)]
    blocks = sum((L + 31) // 32 for L in lens) + B
    c = Case(lens, T, Hkv=Hkv, G=G, D=D, bits=(pick(2, 4, 8), pick(2, 4, 8)), kmode=kmode, pool=pick(0, 0, blocks), seed=seed)
    slopes = torch.from_numpy(rng.uniform(-0.05, 0.6, Hkv * G).astype(np.float32)).cuda()
    o = {}
    if rng.random() < 0.4:
        o["cap"] = pick(3.0, 30.0, 50.0, 100.0)
    if rng.random() < 0.4:
        o["window"] = int(np.exp(rng.uniform(0, np.log(1000))))
    if rng.random() < 0.3:
        o["alibi"] = slopes
    if rng.random() < 0.2:
        o["scale"] = float(np.float32(rng.uniform(-0.2, 0.2)))
    nd = [int(rng.integers(0, T + 1)) for _ in range(B)] if rng.random() < 0.6 else None
    mask, depth = ref.random_tree(B, T, seed) if rng.random() < 0.6 else (None, None)
    what = f"seed {seed}: {lens} T={T} G={G} D={D} K{c.bits[0]}V{c.bits[1]} kmode {kmode} {sorted(o)}"
    tree(c, what, nd, mask, depth, (0, int(rng.integers(1, 9))), **o)
    if min(lens) > 0:
        decode(c, lens, what, (0, int(rng.integers(1, 9))), **o)
