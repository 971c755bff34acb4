"""Which keys a row of kvq_tree_attn or kvq_decode_attn_scored sees, counted exactly.  All keys are
zero, so all weights are equal, and each value names its token (exact_attention.counting_values):
output times the number of seen keys is the number of them per channel.  A key too many or too few
at the edge of a window, tile, block, split, open group or mask word changes a count by one; the
arithmetic is exact up to the division (weights 2^7, sums below 2^24), so 0.01 is ample."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import kvq

import exact_attention as exact
import step_reference as ref

pytestmark = pytest.mark.gpu

LENS = [0, 1, 31, 32, 33, 127, 128, 129, 160, 257, 300, 500]
WINDOWS = [0, 1, 2, 5, 31, 32, 33, 64, 100, 127, 128, 129, 200, 400]
# query rows per kv head: four, two and one copies of the rows, two row tiles, two row groups
INSTANCES = [(5, 4), (13, 4), (25, 4), (40, 4), (70, 4), (1, 1), (64, 1)]


class Counted:
    def __init__(self, lens, T, G, D=64, Hkv=1, bits=(2, 2), kmode=0, pool=0):
        B = len(lens)
        self.B, self.T, self.G, self.D, self.Hkv, self.lens, self.bits = B, T, G, D, Hkv, lens, bits
        n = max(max(lens), 1)
        self.cache = kvq.Cache(1, B, Hkv, Hkv * G, D, n + T, [bits], kmodes=[kmode], pool_blocks=pool)
        names = torch.from_numpy(exact.counting_values(n + T, D, bits[1])).to(torch.bfloat16).cuda()
        zero = torch.zeros((B, Hkv, n, D), dtype=torch.bfloat16, device="cuda")
        if max(lens):
            self.cache.append_ragged(0, zero, names[:n].expand(B, Hkv, -1, -1).contiguous(), lens)
        self.Kd = torch.zeros((B, Hkv, T, D), dtype=torch.bfloat16, device="cuda")
        self.Vd = torch.stack([names[L:L + T] for L in lens])[:, None].expand(-1, Hkv, -1, -1).contiguous()
        self.q = torch.randn((B, T, Hkv * G, D), device="cuda").to(torch.bfloat16)
        self.levels = 2 ** bits[1] - 1

    def compare(self, out, see, what):
        """out [.., Hq, D] of rows whose seen tokens are the columns of bool see [.., L + T]."""
        n = see.shape[-1]
        onehot = np.zeros((n, self.D))
        onehot[np.arange(n), np.arange(n) % self.D] = 1
        want = (see @ onehot)[..., None, :]
        got = out.double().cpu().numpy() * see.sum(-1)[..., None, None] / self.levels
        assert np.isfinite(got).all(), what
        bad = np.abs(got - want) > 0.01
        assert not bad.any(), (what, np.argwhere(bad)[:4].tolist(), got[bad][:4].tolist(),
                               np.broadcast_to(want, got.shape)[bad][:4].tolist())

    def tree(self, n_draft=None, mask=None, depth=None, window=0, what=""):
        out = torch.full((self.B, self.T, self.Hkv * self.G, self.D), -1.0, device="cuda")
        self.cache.tree_attn(0, self.q, self.Kd, self.Vd, n_draft, mask, depth, kvq.ScoreOpts(window=window), out=out,
                             out_fp32=True)
        torch.cuda.synchronize()
        for b, L in enumerate(self.lens):
            t = self.T if n_draft is None else n_draft[b]
            assert (out[b, t:] == -1.0).all(), what
            d = np.arange(t) if depth is None else depth[b, :t].cpu().numpy()
            drafted = np.tril(np.ones((t, t), bool)) if mask is None else ref.mask_rows(mask[b], self.T)[:t, :t]
            see = np.concatenate([np.ones((t, L), bool), drafted], 1)
            if window:
                see &= (L + d)[:, None] - np.concatenate([np.arange(L), L + d])[None] < window
            self.compare(out[b, :t], see, f"{what} request {b} L={L}")


@pytest.mark.parametrize("kmode", [0, 1])
@pytest.mark.parametrize("T,G", INSTANCES)
def test_windows(T, G, kmode):
    """Causal chunks and trees (depths repeat, run ahead of the mask's order) at every window."""
    c = Counted(LENS, T, G, kmode=kmode, D=128 if T % 2 else 64)
    nd = [max(0, T - 3 * (b % 4)) for b in range(c.B)]
    mask, depth = ref.random_tree(c.B, T, T)
    for window in WINDOWS:
        for S in ((0, 3) if window else (0, 1, 2, 3, 7)):
            kvq.kvq_set_num_splits(c.cache.h, S)
            c.tree(window=window, what=f"chunk window {window} splits {S}")
            c.tree(nd, mask, depth, window, f"tree window {window} splits {S}")
    assert kvq.kvq_device_status(c.cache.h) == 0


@pytest.mark.parametrize("T,G", INSTANCES)
def test_any_mask(T, G):
    """Masks without structure: empty rows, full rows, single bits, tokens that see later ones."""
    rng = np.random.default_rng(T)
    c = Counted(LENS, T, G, bits=(8, 8))
    vis = rng.random((c.B, T, T)) < rng.random((c.B, T, 1)) ** 2
    vis[:, 0] = False
    vis[0, -1] = True
    vis[1] = np.eye(T, dtype=bool)
    mask = ref.pack_mask(vis)
    depth = torch.from_numpy(rng.integers(0, 3 * T, (c.B, T)).astype(np.int32)).cuda()
    for window in (0, 1, T, 2 * T, 64, 300):
        for S in (0, 4):
            kvq.kvq_set_num_splits(c.cache.h, S)
            c.tree(None, mask, depth, window, f"window {window} splits {S}")


@pytest.mark.parametrize("T,G,D,bits,kmode,L", [(16, 4, 128, (4, 2), 0, 20000), (50, 4, 64, (4, 4), 0, 19999),
                                                (600, 1, 64, (8, 8), 1, 5003), (300, 4, 128, (8, 2), 0, 2090)])
def test_long(T, G, D, bits, kmode, L):
    c = Counted([L, L - 1000], T, G, D=D, bits=bits, kmode=kmode)
    mask, depth = ref.random_tree(2, T, 1) if T < 100 else (None, None)
    for window in (0, 1000, 4097, L + 7):
        c.tree(None, mask, depth, window, f"window {window}")


def test_pools_and_many_requests():
    rng = np.random.default_rng(3)
    for pool, B in ((150, 12), (0, 70), (800, 70)):
        lens = [int(x) for x in rng.integers(0, 330, B)]
        c = Counted(lens, 6, 4, pool=pool)
        nd = [int(x) for x in rng.integers(0, 7, B)]
        mask, depth = ref.random_tree(B, 6, B)
        for window in (0, 33, 200):
            c.tree(nd, mask, depth, window, f"pool {pool} batch {B} window {window}")


@pytest.mark.parametrize("kmode,G", [(0, g) for g in range(1, 9)] + [(1, 1), (1, 2), (1, 4)])
def test_scored_decode(kmode, G):
    rng = np.random.default_rng(G)
    for lens, pool in (([x for x in LENS if x], 0), ([int(x) for x in rng.integers(1, 600, 70)], 0),
                       ([int(x) for x in rng.integers(1, 600, 20)], 400)):
        c = Counted(lens, 1, G, D=128 if G % 2 else 64, bits=(2, 4), kmode=kmode, pool=pool)
        for window in WINDOWS + [1000]:
            for S in (0, 2, 5):
                kvq.kvq_set_num_splits(c.cache.h, S)
                out = c.cache.decode_attn_scored(0, c.q[:, 0].contiguous(), kvq.ScoreOpts(window=window), out_fp32=True)
                torch.cuda.synchronize()
                for b, L in enumerate(lens):
                    see = np.arange(L) >= (L - window if window else 0)
                    c.compare(out[b], see, f"window {window} splits {S} request {b} L={L}")
        assert kvq.kvq_device_status(c.cache.h) == 0
