"""Plain 64-bit references of the multi-token step operators, shared by their tests: the
cache's values from the oracle, attention with score shapes and masks, norm + rotation.
Each attention reference comes with an element-wise error bound (see `attention`)."""
import numpy as np
import torch

import oracle

from test_gpu_parity import bits16


def cached_values(K, V, L, bk, bv, kmode):
    """K, V bf16 [Hkv, n, D] of one request -> float64 [Hkv, L, D] values of its first L tokens."""
    H, _, D = K.shape
    Kh, Vh = np.zeros((H, L, D)), np.zeros((H, L, D))
    for h in range(H):
        if L:
            _, Kh[h], Vh[h] = oracle.unit(bits16(K[h, :L]), bits16(V[h, :L]), D, bk, bv, kmode)
    return Kh, Vh


def mask_rows(mask, T):
    """int32 [T, W] bit rows -> bool [T, T]."""
    w = mask.cpu().numpy().view(np.uint32)
    return ((w[:, :, None] >> np.arange(32, dtype=np.uint32)) & 1).reshape(T, -1)[:, :T].astype(bool)


def attention(q, Kh, Vh, Kd, Vd, see_draft, pos_q, pos_d, L, G, cap=0.0, alibi=None, window=0, scale=0.0):
    """One request.  q float64 [t, Hq, D]; Kh, Vh [Hkv, L, D]; Kd, Vd [Hkv, t, D] or None;
    see_draft bool [t, t]; returns (out [t, Hq, D], bound [t, Hq, D]).

    The bound: keys, values and weights enter the products as fp16, each off by at most
    e = 2^-11 of itself (half a step); queries and bf16 keys are scaled by a power of two per
    row and are exact down to 2^-38 of the row's largest.  A score is then off by at most
    ds = scale * sum_d (e |q_d k_d| + 2^-38 (max|q| |k_d| + |q_d| max|k|)) plus 2^-18 of its own
    size and the cap's (fp32 sums of 128 terms, the cap's and the exponent's approximations),
    so a weight by the factor exp(+-ds) (1 +- e), and sum w v / sum w by at most
    (2 (exp(ds) (1 + e) - 1) + e) * sum w |v| / sum w, plus 2^-20 absolute (fp16 values
    below the normal range)."""
    t, Hq, D = q.shape
    scale = scale or D ** -0.5
    out, bound = np.zeros((t, Hq, D)), np.zeros((t, Hq, D))
    pk = np.arange(L, dtype=np.float64)
    see = np.ones((t, L), bool)
    if Kd is not None:
        pk = np.concatenate([pk, pos_d])
        see = np.concatenate([see, see_draft], 1)
    dist = pos_q[:, None] - pk[None]
    if window:
        see = see & (dist < window)
    e = 2.0 ** -11
    for h in range(Hq):
        k, v = Kh[h // G], Vh[h // G]
        if Kd is not None:
            k, v = np.concatenate([k, Kd[h // G]]), np.concatenate([v, Vd[h // G]])
        for r in range(t):
            s_ = see[r]
            if not s_.any():
                continue
            kk, vv = k[s_], v[s_]
            s = (kk @ q[r, h]) * scale
            aq, ak = np.abs(q[r, h]), np.abs(kk)
            ds = scale * (e * (ak @ aq) + 2.0 ** -38 * (aq.max() * ak.sum(1) + aq.sum() * ak.max(1)))
            ds = ds + 2.0 ** -18 * (np.abs(s) + cap)
            if cap:
                s = cap * np.tanh(s / cap)
            if alibi is not None:
                bias = alibi[h] * dist[r][s_]
                s = s - bias
                ds = ds + 2.0 ** -21 * np.abs(bias)
            w = np.exp(s - s.max())
            out[r, h] = (w @ vv) / w.sum()
            f = 2 * (np.exp(ds.max()) * (1 + e) - 1) + e
            bound[r, h] = f * (w @ np.abs(vv)) / w.sum() + 2.0 ** -20
    return out, bound


def check(out, ref, bound, what=""):
    """Output tensor (fp32 or bf16) against the reference within the bound plus its rounding."""
    o = out.double().cpu().numpy()
    half = torch.finfo(out.dtype).eps / 2
    tol = bound * (1 + half) + half * np.abs(ref) + 2.0 ** -133
    bad = ~(np.abs(o - ref) <= tol)
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:3].tolist(), float(np.nanmax(np.abs(o - ref))),
                           float(np.nanmax(np.abs(o - ref) / np.maximum(tol, 1e-30))))


def norm_rope(x, w, pos, inv_freq, rot, inter, eps):
    """x float64 [..., D] (one head per row), pos broadcastable to x[..., 0]."""
    D = x.shape[-1]
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * w if w is not None else x.copy()
    if rot == 0:
        return y
    ang = np.asarray(pos, np.float64)[..., None] * inv_freq[:rot // 2]
    c, s = np.cos(ang), np.sin(ang)
    a, b = (y[..., 0:rot:2], y[..., 1:rot:2]) if inter else (y[..., :rot // 2], y[..., rot // 2:rot])
    ra, rb = a * c - b * s, b * c + a * s
    z = y.copy()
    if inter:
        z[..., 0:rot:2], z[..., 1:rot:2] = ra, rb
    else:
        z[..., :rot // 2], z[..., rot // 2:rot] = ra, rb
    return z


def random_tree(B, T, seed):
    """(mask int32 [B, T, W], depth int32 [B, T]) of random drafted trees on the GPU."""
    rng = np.random.default_rng(seed)
    vis = np.zeros((B, T, T), bool)
    depth = np.zeros((B, T), np.int32)
    for b in range(B):
        for t in range(T):
            if t and rng.random() < 0.95:
                par = int(rng.integers(max(0, t - 6), t))
                vis[b, t] = vis[b, par]
                depth[b, t] = depth[b, par] + 1
            vis[b, t, t] = True
    return pack_mask(vis), torch.from_numpy(depth).cuda()


def pack_mask(vis):
    B, T, _ = vis.shape
    W = (T + 31) // 32
    v = np.zeros((B, T, W * 32), np.uint64)
    v[:, :, :T] = vis
    words = (v.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return torch.from_numpy(words.view(np.int32)).cuda()
