"""kvq_tree_attn and kvq_decode_attn_scored against a plain 64-bit attention over the
oracle's cache values: trees and causal chunks, one token to hundreds, every bit pair and
key mode, score shapes, ragged and empty requests, splits, block pools, masked rows and
non-finite values in masked places, captured graphs, other streams."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import inputs, kvq

import step_reference as ref
from test_gpu_parity import workload

pytestmark = pytest.mark.gpu


class Case:
    def __init__(self, lens, T, Hkv=2, G=4, D=128, bits=(4, 2), kmode=0, pool=0, seed=1, name="tree"):
        self.B, self.T, self.Hkv, self.G, self.D, self.bits, self.kmode = len(lens), T, Hkv, G, D, bits, kmode
        self.lens = list(lens)
        B, Hq = self.B, Hkv * G
        wl = workload(B, Hkv, G, D, name=f"{name}{seed}")
        n = max(max(lens), 1)
        self.K, self.V = inputs.layer_kv(wl, 0, n, "cuda")
        self.cache = kvq.Cache(1, B, Hkv, Hq, D, n + T, [bits], kmodes=[kmode], pool_blocks=pool)
        if max(lens):
            self.cache.append_ragged(0, self.K, self.V, lens)
        self.Kd, self.Vd = inputs.layer_kv(wl, 0, T, "cuda", tag="draft")
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.q = torch.randn((B, T, Hq, D), generator=g, device="cuda").to(torch.bfloat16)

    def reference(self, n_draft=None, mask=None, depth=None, **opts):
        outs, bounds = [], []
        for b, L in enumerate(self.lens):
            t = self.T if n_draft is None else n_draft[b]
            Kh, Vh = ref.cached_values(self.K[b], self.V[b], L, *self.bits, self.kmode)
            see = np.tril(np.ones((t, t), bool)) if mask is None else ref.mask_rows(mask[b], self.T)[:t, :t]
            d = np.arange(t, dtype=np.float64) if depth is None else depth[b, :t].double().cpu().numpy()
            f = lambda x: x.double().cpu().numpy()
            o, e = ref.attention(f(self.q[b, :t]), Kh, Vh, f(self.Kd[b, :, :t]), f(self.Vd[b, :, :t]), see, L + d, L + d, L,
                                 self.G, **opts)
            outs.append(o)
            bounds.append(e)
        return outs, bounds

    def check(self, n_draft=None, mask=None, depth=None, splits=(0,), what="", **opts):
        refs, bounds = self.reference(n_draft, mask, depth, **{**opts, "alibi": None if opts.get("alibi") is None else
                                                               opts["alibi"].double().cpu().numpy()})
        o = kvq.ScoreOpts(opts.get("cap", 0.0), opts.get("alibi"), opts.get("window", 0), opts.get("scale", 0.0))
        for S in splits:
            kvq.kvq_set_num_splits(self.cache.h, S)
            for fp32 in (True, False):
                out = torch.full((self.B, self.T, self.Hkv * self.G, self.D), 7.0, device="cuda",
                                 dtype=torch.float32 if fp32 else torch.bfloat16)
                self.cache.tree_attn(0, self.q, self.Kd, self.Vd, n_draft, mask, depth, o, out=out, out_fp32=fp32)
                torch.cuda.synchronize()
                for b in range(self.B):
                    t = self.T if n_draft is None else n_draft[b]
                    ref.check(out[b, :t], refs[b], bounds[b], f"{what} S={S} fp32={fp32} request {b} L={self.lens[b]}")
                    assert (out[b, t:] == 7.0).all(), (what, "rows behind the last drafted token were written")
        kvq.kvq_set_num_splits(self.cache.h, 0)
        assert kvq.kvq_device_status(self.cache.h) == 0


@pytest.mark.parametrize("kmode", [0, 1])
@pytest.mark.parametrize("L", [0, 1, 15, 31, 32, 33, 127, 128, 129, 160, 300])
def test_lengths(L, kmode):
    c = Case([L, L], 5, kmode=kmode, seed=L + 1)
    c.check(what="chunk")
    mask, depth = ref.random_tree(2, 5, L)
    c.check(mask=mask, depth=depth, splits=(0, 2), what="tree")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kmode", [0, 1])
@pytest.mark.parametrize("bk", [2, 4, 8])
@pytest.mark.parametrize("bv", [2, 4, 8])
def test_bit_pairs(D, kmode, bk, bv):
    Case([203], 6, D=D, bits=(bk, bv), kmode=kmode, seed=bk * 10 + bv).check(what=f"K{bk}V{bv}")


@pytest.mark.parametrize("T", [1, 2, 7, 31, 32, 33, 63, 64, 65, 97, 130, 256, 300])
def test_draft_counts(T):
    """Row tiles end inside a token's heads, drafts cross mask words and key tiles."""
    c = Case([70], T, Hkv=1, seed=T)
    c.check(what="chunk")
    mask, depth = ref.random_tree(1, T, T)
    c.check(mask=mask, depth=depth, what="tree")


@pytest.mark.parametrize("G,kmode", [(1, 0), (2, 1), (3, 0), (5, 0), (7, 0), (8, 0), (1, 1)])
def test_head_groups(G, kmode):
    c = Case([100, 41], 19, G=G, kmode=kmode, seed=G)
    mask, depth = ref.random_tree(2, 19, G)
    c.check(n_draft=[19, 4], mask=mask, depth=depth, what=f"G={G}")


@pytest.mark.parametrize("D,kmode", [(128, 0), (64, 0), (128, 1), (64, 1)])
def test_score_shapes(D, kmode):
    c = Case([333, 40, 0], 9, D=D, kmode=kmode, bits=(8, 4), seed=D + kmode)
    mask, depth = ref.random_tree(3, 9, 3)
    slopes = torch.tensor([2.0 ** -(i + 1) for i in range(8)], device="cuda")
    for kw in (dict(cap=5.0), dict(window=1), dict(window=64), dict(window=130, cap=20.0), dict(alibi=slopes),
               dict(alibi=slopes, cap=30.0, window=50), dict(scale=0.2)):
        c.check(n_draft=[9, 6, 3], mask=mask, depth=depth, splits=(0, 3), what=str(sorted(kw)), **kw)
    c.check(cap=8.0, window=5, what="chunk")


def test_ragged_and_empty_requests():
    lens = [0, 1, 500, 31, 96, 0, 257]
    nd = [5, 0, 11, 1, 0, 3, 8]
    for kmode in (0, 1):
        c = Case(lens, 11, kmode=kmode, seed=40 + kmode)
        mask, depth = ref.random_tree(7, 11, 5)
        c.check(n_draft=nd, mask=mask, depth=depth, splits=(0, 1, 4), what="ragged")
    out = torch.full_like(c.q, 3.0)
    c.cache.tree_attn(0, c.q, c.Kd, c.Vd, [0] * 7, out=out)   # no drafted token at all: nothing happens
    assert (out == 3.0).all()


def test_batch_above_the_parameter_tables():
    rng = np.random.default_rng(9)
    lens = [int(x) for x in rng.integers(0, 150, 70)]
    c = Case(lens, 4, Hkv=1, G=2, D=64, seed=70)
    c.check(n_draft=[int(x) for x in rng.integers(0, 5, 70)], what="b70")


@pytest.mark.parametrize("splits", [1, 2, 3, 5, 16, 64])
def test_splits(splits):
    c = Case([1030, 700], 13, Hkv=1, seed=splits)
    mask, depth = ref.random_tree(2, 13, splits)
    c.check(n_draft=[13, 12], mask=mask, depth=depth, splits=(splits,), what="splits")


def test_block_pools():
    for kmode in (0, 1):
        c = Case([130, 65, 300], 6, pool=40, kmode=kmode, seed=60 + kmode)
        c.check(what="pools", splits=(0, 2))


def test_rows_that_see_nothing():
    """Empty mask rows over an empty cache give zeros; over a cached prefix, the prefix."""
    B, T = 2, 40
    vis = np.tril(np.ones((B, T, T), bool))
    vis[:, 3] = False
    vis[:, 17] = False
    vis[:, :, 20:25] = False
    mask = ref.pack_mask(vis)
    Case([0, 0], T, seed=5).check(mask=mask, what="empty cache")
    c = Case([45, 0], T, seed=6)
    c.check(mask=mask, splits=(0, 2), what="prefix")
    # a window that a row's own position leaves: depth far behind the keys it may see
    depth = torch.full((B, T), 1000, dtype=torch.int32, device="cuda")
    depth[:, ::2] = 0
    c.check(mask=mask, depth=depth, window=100, what="window")


@pytest.mark.parametrize("val", [float("nan"), float("inf"), -float("inf")])
def test_non_finite_values_in_masked_places(val):
    """NaN and infinities behind n_draft and in tokens a row does not see have no influence;
    a row that sees a value gets it in that channel only."""
    c = Case([50, 7], 20, seed=8)
    vis = np.tril(np.ones((2, 20, 20), bool))
    vis[:, :, 6] = False
    vis[:, 6, 6] = True
    nd = [20, 9]
    mask = ref.pack_mask(vis)
    refs, bounds = c.reference(nd, mask)
    c.Kd[:, :, 6] = val
    c.Kd[1, :, 9:] = val
    c.Vd[1, :, 9:] = val
    c.q[1, 9:] = val
    out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, nd, mask, out_fp32=True)
    for b in range(2):
        rows = [t for t in range(nd[b]) if t != 6]
        ref.check(out[b, rows], refs[b][rows], bounds[b][rows], f"keys {val} request {b}")
    c = Case([50, 7], 20, seed=8)
    c.Vd[:, :, 6, 5] = val
    out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, nd, mask, out_fp32=True)
    for b in range(2):
        rows = [t for t in range(nd[b]) if t != 6]
        ref.check(out[b, rows], refs[b][rows], bounds[b][rows], f"values {val} request {b}")
        ch = [d for d in range(128) if d != 5]
        ref.check(out[b, 6][:, ch], refs[b][6][:, ch], bounds[b][6][:, ch], f"values {val} the row that sees it")
        got = out[b, 6, :, 5]
        assert (torch.isnan(got) if val != val else got == val).all()


@pytest.mark.parametrize("kind", ["const", "zero_k", "zero_v", "zero_kv", "tiny", "large", "q_big", "q_huge", "q_small"])
def test_value_ranges(kind):
    """Caches with constant or zero groups, fp16-subnormal scales, large values, and queries
    far from one (scores stay of order one)."""
    B, Hkv, G, D, L, T = 1, 2, 4, 128, 77, 3
    c = Case([L], T, seed=11)
    wl = workload(B, Hkv, G, D, name="range")
    K, V = inputs.edge_kv(kind, wl, 0, L + T, "cuda", (4, 2))
    c.K, c.V = K[:, :, :L].contiguous(), V[:, :, :L].contiguous()
    c.Kd, c.Vd = K[:, :, L:].contiguous(), V[:, :, L:].contiguous()
    c.q = torch.stack([inputs.edge_q(kind, wl, 0, s, "cuda", (4, 2)) for s in range(T)], 1).contiguous()
    kvq.kvq_reset_sequences(c.cache.h, [0])
    c.cache.append(0, c.K, c.V)
    c.check(what=kind, splits=(0, 2))


def test_scored_decode():
    for D, kmode, lens in ((128, 0, [300, 45, 1]), (64, 1, [33, 129, 64]), (128, 1, [1500, 31, 700]), (64, 0, [97, 2, 640])):
        c = Case(lens, 1, D=D, kmode=kmode, bits=(8, 4), seed=sum(lens))
        Hq = c.Hkv * c.G
        slopes = torch.tensor([2.0 ** -(i + 1) for i in range(Hq)], device="cuda")
        for kw in (dict(), dict(cap=6.0), dict(window=1), dict(window=50), dict(alibi=slopes),
                   dict(cap=9.0, window=40, alibi=slopes)):
            o = kvq.ScoreOpts(kw.get("cap", 0.0), kw.get("alibi"), kw.get("window", 0))
            for S in (0, 3):
                kvq.kvq_set_num_splits(c.cache.h, S)
                for fp32 in (True, False):
                    out = c.cache.decode_attn_scored(0, c.q[:, 0], o, out_fp32=fp32)
                    for b, L in enumerate(lens):
                        Kh, Vh = ref.cached_values(c.K[b], c.V[b], L, *c.bits, kmode)
                        kwn = {**kw, "alibi": slopes.double().cpu().numpy()} if "alibi" in kw else kw
                        r, e = ref.attention(c.q[b].double().cpu().numpy(), Kh, Vh, None, None, None,
                                             np.array([L - 1.0]), None, L, c.G, **kwn)
                        ref.check(out[b:b + 1], r, e, f"{kw} S={S} request {b}")
        # no opts at all: the attention of decode_attn (both within their bounds of each other)
        a, d = c.cache.decode_attn_scored(0, c.q[:, 0], None, out_fp32=True), c.cache.decode_attn(0, c.q[:, 0], out_fp32=True)
        assert (a - d).abs().max() <= 1e-2 and (a - d).norm() <= 2e-3 * d.norm()


def test_same_result_again_and_on_another_stream():
    """Bit-equal on repetition, on a side stream, and replayed from graphs that hold two
    calls with a workspace each."""
    c = Case([700, 300], 8, seed=21)
    mask, depth = ref.random_tree(2, 8, 1)
    args = (0, c.q, c.Kd, c.Vd, [8, 5], mask, depth)
    out = torch.zeros_like(c.q)
    c.cache.tree_attn(*args, out=out)
    first = out.clone()
    side = torch.cuda.Stream()
    ws = [c.cache.tree_workspace(8) for _ in range(2)]
    outs = [torch.zeros_like(c.q) for _ in range(2)]
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.cache.tree_attn(*args, out=outs[0], workspace=ws[0])
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first)
    graphs = []
    for i in range(2):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            c.cache.tree_attn(*args, out=outs[i], workspace=ws[i])
        graphs.append(gr)
    for o in outs:
        o.zero_()
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], first) and torch.equal(outs[1], first)


def test_long_context():
    """A context of 20000 tokens, 24 drafted tokens, automatic splits; positions of a window
    that starts inside a tile."""
    c = Case([20000], 24, Hkv=1, G=2, bits=(2, 2), seed=31)
    mask, depth = ref.random_tree(1, 24, 31)
    c.check(mask=mask, depth=depth, what="long")
    c.check(mask=mask, depth=depth, window=7001, what="long window")


def test_first_call_is_not_captured():
    """The first launch after a bind clears the workspace's words: refused inside a capture
    (a replay would clear them again), fine once something ran."""
    c = Case([0, 0], 4, seed=50)
    ws = c.cache.tree_workspace(4)
    out = torch.zeros_like(c.q)
    index = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    for call in (lambda: c.cache.tree_attn(0, c.q, c.Kd, c.Vd, out=out, workspace=ws),
                 lambda: c.cache.append_selected(0, c.Kd, c.Vd, index)):
        with pytest.raises(kvq.KvqError) as e:
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                call()
        assert e.value.code == kvq.KVQ_EINVAL and "captured" in str(e.value)
    c.check(what="after the refusals")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        c.cache.tree_attn(0, c.q, c.Kd, c.Vd, out=out, workspace=ws)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, c.cache.tree_attn(0, c.q, c.Kd, c.Vd))


def test_largest_draft():
    """4096 tokens of a causal chunk over a short prefix: rows picked over the chunk."""
    c = Case([75], 4096, Hkv=1, G=8, D=64, bits=(8, 8), seed=51)
    out = c.cache.tree_attn(0, c.q, c.Kd, c.Vd, out_fp32=True)
    Kh, Vh = ref.cached_values(c.K[0], c.V[0], 75, 8, 8, 0)
    f = lambda x: x.double().cpu().numpy()
    pos = 75 + np.arange(4096.0)
    rows = [0, 1, 15, 16, 31, 32, 127, 2047, 2048, 4080, 4095]
    see = np.tril(np.ones((4096, 4096), bool))[rows]
    r, e = ref.attention(f(c.q[0])[rows], Kh, Vh, f(c.Kd[0]), f(c.Vd[0]), see, pos[rows], pos, 75, 8)
    ref.check(out[0, rows], r, e, "T=4096")
    assert torch.isfinite(out).all() and kvq.kvq_device_status(c.cache.h) == 0


@pytest.mark.slow
def test_cache_beyond_four_gigabytes():
    """Records whose offsets pass 32 bits (32 units of 960,000 tokens, K8V8: 4.4 GB): tree
    attention, scored decode and read-back of the last unit."""
    B, Hkv, D, L, step = 4, 8, 64, 960000, 60000
    cache = kvq.Cache(1, B, Hkv, Hkv, D, L, [(8, 8)])
    last = []
    for i in range(L // step):
        g = torch.Generator(device="cuda").manual_seed(i)
        K, V = (torch.randn((B, Hkv, step, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        cache.append(0, K, V)
        last.append((K[-1, -1:].cpu(), V[-1, -1:].cpu()))
    assert cache.nbytes > 1 << 32
    K, V = (torch.cat([x[k] for x in last], 1) for k in (0, 1))
    Kh, Vh = ref.cached_values(K, V, L, 8, 8, 0)
    T = 3
    g = torch.Generator(device="cuda").manual_seed(99)
    q, Kd, Vd = (torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)
                 for s in ((B, T, Hkv, D), (B, Hkv, T, D), (B, Hkv, T, D)))
    out = cache.tree_attn(0, q, Kd, Vd, out_fp32=True)
    f = lambda x: x.double().cpu().numpy()
    pos = L + np.arange(float(T))
    r, e = ref.attention(f(q[-1, :, -1:]), Kh, Vh, f(Kd[-1, -1:]), f(Vd[-1, -1:]), np.tril(np.ones((T, T), bool)), pos, pos, L, 1)
    ref.check(out[-1, :, -1:], r, e, "tree")
    o = cache.decode_attn_scored(0, q[:, 0].contiguous(), kvq.ScoreOpts(20.0), out_fp32=True)
    r, e = ref.attention(f(q[-1, :1, -1:]), Kh, Vh, None, None, None, np.array([L - 1.0]), None, L, 1, cap=20.0)
    ref.check(o[-1:, -1:], r, e, "scored")
    Ko, Vo = cache.read(0, L - 500, 500)
    as_bf16 = lambda x: torch.from_numpy(x).float().to(torch.bfloat16)
    assert torch.equal(Ko[-1, -1].cpu(), as_bf16(Kh[0, -500:])) and torch.equal(Vo[-1, -1].cpu(), as_bf16(Vh[0, -500:]))
