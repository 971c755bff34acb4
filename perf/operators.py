"""What the operators around a decode step cost: cases, inputs, plain forms, exact values.

Four groups of calls that a speculative or long-prompt step makes beside append and decode:

  rope    kvq_norm_rope: RMS norm of every query and key head, rotation by position, and
          the split of the projection's rows into q (by token) and K, V (by kv head)
  tree    kvq_tree_attn: drafted tokens (a tree, or a causal chunk) attend over the packed
          cache and over one another; capped scores, distance bias, sliding window
  scored  kvq_decode_attn_scored: one query token per sequence over the packed cache with
          capped scores, distance bias or a sliding window
  commit  kvq_append_selected + kvq_read: the accepted drafted tokens are quantised into the
          cache and read back as the values the cache now stands for
  read    kvq_read: a token range of the cache as bf16

A case is a dict of plain values; `run` computes it with elementary torch operations in 32
bits (`own` false) or with this repository's calls (`own` true).  `exact` has the values in
64 bits, written apart from the plain forms.

Definition of the cache's values (groups of 32; every quantiser step one rounded binary32
operation): s = fp16((max - min) / (2^b - 1)), z = fp16(min), code = clamp(rint((x - z) / s)),
value = code * s + z.  Values per token over 32 channels; keys per channel over 32 tokens
(the last L mod 32 tokens stay bf16) or per token over 32 channels.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one decode step of a 64-sequence batch, Llama-shaped attention (32 q / 8 kv heads)
        {"name": "rope_step", "op": "rope", "B": 64, "n": 1, "Hkv": 8, "G": 4, "D": 128, "L": 4000, "rot": 128,
         "inter": False, "norm": True, "offset": False, "far": 0, "pad": 0},
        # a tree of 17 drafted tokens, Qwen-shaped attention (28 q / 4 kv heads), half the
        # channels rotated in adjacent pairs, no norm, rows padded in the projection's output
        {"name": "rope_tree", "op": "rope", "B": 32, "n": 17, "Hkv": 4, "G": 7, "D": 128, "L": 8191, "rot": 64,
         "inter": True, "norm": False, "offset": True, "far": 0, "pad": 64},
        # a prompt of 4096 tokens for four sequences
        {"name": "rope_prompt", "op": "rope", "B": 4, "n": 4096, "Hkv": 8, "G": 4, "D": 128, "L": 0, "rot": 128,
         "inter": False, "norm": True, "offset": False, "far": 0, "pad": 0},
        # one user, short context, 8 drafted tokens: latency
        {"name": "tree_single", "op": "tree", "B": 1, "T": 8, "Hkv": 8, "G": 4, "D": 128, "L": 133, "bk": 8, "bv": 4,
         "kmode": 0, "tree": True, "ragged": False, "cap": 0.0, "window": 0, "alibi": False},
        # batch 64 at context 4096, K4V2, 16 drafted tokens (the 3.25-bit map's common layer)
        {"name": "tree_b64_4k", "op": "tree", "B": 64, "T": 16, "Hkv": 8, "G": 4, "D": 128, "L": 4096, "bk": 4,
         "bv": 2, "kmode": 0, "tree": True, "ragged": False, "cap": 0.0, "window": 0, "alibi": False},
        # Qwen shape, batch 32, contexts of different lengths up to 8192, K8V2, 33 drafted tokens
        {"name": "tree_qwen_8k", "op": "tree", "B": 32, "T": 33, "Hkv": 4, "G": 7, "D": 128, "L": 8192, "bk": 8,
         "bv": 2, "kmode": 0, "tree": True, "ragged": True, "cap": 0.0, "window": 0, "alibi": False},
        # batch 16 at context 32768, 64 drafted tokens, K4V4
        {"name": "tree_b16_32k", "op": "tree", "B": 16, "T": 64, "Hkv": 8, "G": 4, "D": 128, "L": 32768, "bk": 4,
         "bv": 4, "kmode": 0, "tree": True, "ragged": False, "cap": 0.0, "window": 0, "alibi": False},
        # a prompt's next chunk of 500 tokens (causal) over a cached prefix, capped scores, per-token keys
        {"name": "tree_chunk", "op": "tree", "B": 8, "T": 500, "Hkv": 4, "G": 4, "D": 64, "L": 1000, "bk": 8, "bv": 8,
         "kmode": 1, "tree": False, "ragged": True, "cap": 30.0, "window": 0, "alibi": False},
        # one decode token, capped scores and a sliding window of 1024 tokens
        {"name": "scored_window", "op": "scored", "B": 64, "Hkv": 8, "G": 4, "D": 128, "L": 4111, "bk": 8, "bv": 4,
         "kmode": 0, "ragged": True, "cap": 50.0, "window": 1024, "alibi": False},
        # one decode token, distance bias, Qwen shape at context 8192
        {"name": "scored_bias", "op": "scored", "B": 32, "Hkv": 4, "G": 7, "D": 128, "L": 8192, "bk": 4, "bv": 2,
         "kmode": 0, "ragged": False, "cap": 0.0, "window": 0, "alibi": True},
        # up to 6 of 16 drafted tokens accepted for each of 64 sequences, then read back
        {"name": "commit_step", "op": "commit", "B": 64, "T": 16, "n": 6, "Hkv": 8, "G": 4, "D": 128, "L": 4096,
         "bk": 8, "bv": 4, "kmode": 0},
        # a cached range of 8000 tokens back as bf16 (a prefix moved to another layout)
        {"name": "read_8k", "op": "read", "B": 8, "n": 8000, "t0": 33, "Hkv": 8, "G": 4, "D": 128, "L": 8050,
         "bk": 4, "bv": 2, "kmode": 0},
    ]


def _logint(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope", "tree", "tree", "tree", "tree", "scored", "scored", "commit", "read"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8])
    kmode = rng.choice([0, 0, 1])
    G = rng.choice([1, 2, 4]) if kmode else rng.choice([1, 2, 3, 4, 5, 6, 7, 8])
    c = {"op": op, "Hkv": Hkv, "G": G, "D": D}
    if op == "rope":
        c["n"] = rng.choice([1, rng.randint(2, 64), _logint(rng, 65, 4096)])
        c["B"] = max(1, min(_logint(rng, 1, 64), 16384 * 48 * 128 // (c["n"] * (G + 2) * Hkv * D)))
        c["L"] = _logint(rng, 1, 4096)
        c["rot"] = rng.choice([D, D, D // 2, 32])
        c["inter"] = rng.random() < 0.4
        c["norm"] = rng.random() < 0.6
        c["offset"] = rng.random() < 0.5
        c["far"] = _logint(rng, 1, 1000000) if c["offset"] else 0     # offsets may point far ahead
        c["pad"] = rng.choice([0, 0, 8, 64])
        return c
    c.update(kmode=kmode, bk=rng.choice([2, 4, 8]), bv=rng.choice([2, 4, 8]))
    c["L"] = _logint(rng, 1, 32768)
    c["B"] = _logint(rng, 1, 64)
    if op in ("tree", "scored"):
        c["ragged"] = rng.random() < 0.5
        c["cap"] = rng.choice([0.0, 0.0, 20.0, 50.0])
        c["window"] = rng.choice([0, 0, _logint(rng, 8, 8192)])
        c["alibi"] = rng.random() < 0.3
        if op == "tree":
            c["T"] = rng.choice([rng.randint(1, 8), rng.randint(9, 64), _logint(rng, 65, 512)])
            c["tree"] = c["T"] <= 128 and rng.random() < 0.7
            lim = 16 * 8 * 64 * 4 * 32768 * 128 // (Hkv * G * c["T"] * (c["L"] + c["T"]) * D)
            c["B"] = max(1, min(c["B"], lim, 16 * 8 * 32768 // (Hkv * c["L"])))
        else:
            c["B"] = max(1, min(c["B"], 32 * 28 * 8192 * 128 // (Hkv * G * c["L"] * D)))
        return c
    c["L"] = max(32, c["L"] // 32 * 32) if op == "commit" else c["L"]
    if op == "commit":
        c["T"] = _logint(rng, 2, 200)
        c["n"] = rng.randint(1, c["T"])
        c["B"] = max(1, min(c["B"], 64 * 8 * 4096 // (Hkv * c["L"]), 64 * 8 * 16 * 128 // (Hkv * c["n"] * D)))
        return c
    c["t0"] = rng.randint(0, c["L"] - 1)
    c["n"] = rng.randint(1, c["L"] - c["t0"])
    c["B"] = max(1, min(c["B"], 8 * 8 * 8050 * 128 // (Hkv * c["L"] * D)))
    return c


def _lens(c):
    """Cached tokens of every sequence before the call."""
    B, L = c["B"], c["L"]
    if not c.get("ragged"):
        return [L] * B
    return [L - (i * 997) % (L // 2 + 1) for i in range(B)]


def _drafts(c):
    """Drafted tokens of every sequence (ragged batches draft different numbers)."""
    if not c.get("ragged"):
        return [c["T"]] * c["B"]
    return [c["T"] - (i * 3) % (c["T"] // 4 + 1) for i in range(c["B"])]


def _accepted(c):
    return [c["n"] - (i * 5) % c["n"] for i in range(c["B"])]


# ------------------------------------------------------------------ inputs
def _gen(seed, device=DEV):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed) & 0x7FFFFFFF)
    return g


def _kv(c, n, g):
    """Keys with a few strong channels per head, normal values (bf16 [B, Hkv, n, D])."""
    B, H, D = c["B"], c["Hkv"], c["D"]
    scale = torch.ones((H, D), device=DEV)
    pick = torch.rand((H, D), generator=g, device=DEV).argsort(1)[:, :8]
    scale.scatter_(1, pick, 10 + 10 * torch.rand((H, 8), generator=g, device=DEV))
    K = torch.randn((B, H, n, D), generator=g, device=DEV)
    K = K.mul_(scale[None, :, None, :]).to(torch.bfloat16)
    V = torch.randn((B, H, n, D), generator=g, device=DEV).to(torch.bfloat16)
    return K, V


def _quant(x, bits, dim):
    """Codes (uint8), scale, zero (fp16) of groups of 32 along dim of float x."""
    mn, mx = x.amin(dim, keepdim=True), x.amax(dim, keepdim=True)
    s = ((mx - mn) / float(2 ** bits - 1)).half()
    z = mn.half()
    q = ((x - z.float()) / torch.where(s == 0, torch.ones_like(s), s).float()).round().clamp(0, 2 ** bits - 1)
    q = torch.where(s == 0, torch.zeros_like(q), q)
    return q.to(torch.uint8), s, z


def _quant_tokens(x, bits):
    B, H, n, D = x.shape
    return _quant(x.float().view(B, H, n, D // 32, 32), bits, 4)


def _quant_channels(x, bits):
    B, H, n, D = x.shape
    return _quant(x.float().view(B, H, n // 32, 32, D), bits, 3)


def _plain_cache(c, K, V, lens):
    """The cache as arrays: codes, scales, zeros; the bf16 keys of the open groups."""
    st = {"v": [], "k": []}
    n = K.shape[2]
    for b0 in range(0, K.shape[0], 4):
        st["v"].append(_quant_tokens(V[b0:b0 + 4], c["bv"]))
        if c["kmode"]:
            st["k"].append(_quant_tokens(K[b0:b0 + 4], c["bk"]))
        else:
            st["k"].append(_quant_channels(K[b0:b0 + 4, :, :n // 32 * 32], c["bk"]))
    st["v"] = [torch.cat(t) for t in zip(*st["v"])]
    st["k"] = [torch.cat(t) for t in zip(*st["k"])]
    if not c["kmode"]:   # every sequence's last, open group
        base = torch.tensor([L // 32 * 32 for L in lens], device=DEV)
        idx = (base[:, None] + torch.arange(32, device=DEV)).clamp(max=n - 1)
        st["tail_base"] = base
        st["tail"] = K.gather(2, idx[:, None, :, None].expand(-1, K.shape[1], -1, K.shape[3])).contiguous()
    return st


def _own_cache(c, K, V, lens, extra=0):
    from layer_wise_mixed_b200 import kvq
    B, H, n, D = K.shape
    cache = kvq.Cache(1, B, H, H * c["G"], D, max(n, max(lens) + extra), [(c.get("bk", 8), c.get("bv", 8))],
                      kmodes=[c.get("kmode", 0)])
    if max(lens) > 0:
        cache.append_ragged(0, K, V, lens)
    return cache


def _tree(c, g):
    """Parents of drafted tokens: token 0 is the root, others hang on one of the 8 before."""
    B, T = c["B"], c["T"]
    r = torch.rand((B, T), generator=g, device=DEV).cpu().numpy()
    vis = np.zeros((B, T, T), bool)
    depth = np.zeros((B, T), np.int32)
    rows = np.arange(B)
    for t in range(T):
        if t:
            lo = max(0, t - 8)
            par = lo + (r[:, t] * (t - lo)).astype(np.int64)
            vis[:, t] = vis[rows, par]
            depth[:, t] = depth[rows, par] + 1
        vis[:, t, t] = True
    return vis, depth


def _pack_mask(vis):
    """Bit j of word j / 32 of row t: token t sees token j (int32 [B, T, ceil(T / 32)])."""
    B, T, _ = vis.shape
    W = (T + 31) // 32
    v = np.zeros((B, T, W * 32), np.uint64)
    v[:, :, :T] = vis
    words = (v.reshape(B, T, W, 32) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)
    return torch.from_numpy(words.view(np.int32)).to(DEV)


def _slopes(Hq):
    return torch.tensor([2.0 ** (-8.0 * (i + 1) / Hq) for i in range(Hq)], device=DEV, dtype=torch.float32)


def prepare(case, seed):
    c = case
    g = _gen(seed)
    op, B, H, G, D = c["op"], c["B"], c["Hkv"], c["G"], c["D"]
    Hq = H * G
    st = {"c": c}
    if op == "rope":
        n, W = c["n"], (Hq + 2 * H) * D
        qkv = torch.randn((B, n, W + c["pad"]), generator=g, device=DEV).to(torch.bfloat16)
        st["qkv"] = qkv[:, :, :W]
        st["inv_freq"] = (1e6 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])).float()
        st["wq"] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)) if c["norm"] else None
        st["wk"] = (1 + 0.2 * torch.randn(D, generator=g, device=DEV)) if c["norm"] else None
        st["offset"] = None
        if c["offset"]:
            st["offset"] = torch.from_numpy(_tree({"B": B, "T": n}, g)[1] + np.int32(c["far"])).to(DEV)
        if own:
            from layer_wise_mixed_b200 import kvq
            # the positions follow the cached lengths: a small cache stands for the user's
            cache = kvq.Cache(1, B, H, Hq, D, max(c["L"], 1), [(2, 2)])
            if c["L"]:
                z = torch.zeros((B, H, c["L"], D), dtype=torch.bfloat16, device=DEV)
                cache.append(0, z, z)
            st["cache"] = cache
            st["rope"] = kvq.Rope(c["rot"], st["inv_freq"], st["wq"], st["wk"], 1e-6, c["inter"])
        return st
    if op in ("tree", "scored"):
        lens = _lens(c)
        n = (max(lens) + 31) // 32 * 32
        K, V = _kv(c, n, g)
        T = c.get("T", 1)
        st["q"] = torch.randn((B, T, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
        st["alibi"] = _slopes(Hq) if c["alibi"] else None
        if op == "tree":
            st["Kd"], st["Vd"] = _kv(c, T, g)
            st["drafts"] = _drafts(c)
            st["depth"] = st["mask"] = None
            if c["tree"]:
                vis, depth = _tree(c, g)
                st["depth"] = torch.from_numpy(depth).to(DEV)
                st["mask"] = _pack_mask(vis)
            # rows behind a sequence's last drafted token are left as they were: zeros here
            st["out"] = torch.zeros((B, T, Hq, D), dtype=torch.bfloat16, device=DEV)
        if own:
            from layer_wise_mixed_b200 import kvq
            st["cache"] = _own_cache(c, K, V, lens)
            st["opts"] = kvq.ScoreOpts(c["cap"], st["alibi"], c["window"])
            if op == "tree":
                st["ws"] = st["cache"].tree_workspace(T)
        else:
            st["cache"] = _plain_cache(c, K, V, lens)
            st["lens"] = torch.tensor(lens, device=DEV)
            if op == "tree":
                st["nd"] = torch.tensor(st["drafts"], device=DEV)
        return st
    lens = _lens(c)
    n = (max(lens) + 31) // 32 * 32
    K, V = _kv(c, n, g)
    if op == "commit":
        st["Kd"], st["Vd"] = _kv(c, c["T"], g)
        order = torch.rand((B, c["T"]), generator=g, device=DEV).argsort(1)[:, :c["n"]]
        st["index"] = order.sort(1).values.to(torch.int32).contiguous()
        st["n_new"] = _accepted(c)
        if own:
            st["cache"] = _own_cache(c, K, V, lens, c["n"])
            st["Ko"] = torch.zeros((B, H, c["n"], D), dtype=torch.bfloat16, device=DEV)
            st["Vo"] = torch.zeros_like(st["Ko"])
        else:
            st["acc"] = torch.tensor(st["n_new"], device=DEV)
        return st
    if own:
        st["cache"] = _own_cache(c, K, V, lens)
    else:
        st["cache"] = _plain_cache(c, K, V, lens)
    return st


# ------------------------------------------------------------------ one pass
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(st):
    c = st["c"]
    op, cache = c["op"], st["cache"]
    if op == "rope":
        return cache.norm_rope(0, st["qkv"], st["rope"], st["offset"])
    if op == "tree":
        return cache.tree_attn(0, st["q"], st["Kd"], st["Vd"], st["drafts"], st["mask"], st["depth"], st["opts"],
                               out=st["out"], workspace=st["ws"])
    if op == "scored":
        return cache.decode_attn_scored(0, st["q"][:, 0], st["opts"])
    if op == "commit":
        cache.append_selected(0, st["Kd"], st["Vd"], st["index"], st["n_new"])
        out = cache.read(0, c["L"], c["n"], st["Ko"], st["Vo"])
        cache.truncate(0, c["L"])
        return out
    return cache.read(0, c["t0"], c["n"])


def _dequant(codes, s, z, shape):
    return (codes.float() * s.float() + z.float()).reshape(shape)


def _plain_kv(st):
    """Keys and values the cache stands for, 32 bits [B, Hkv, n, D]."""
    c, ca = st["c"], st["cache"]
    B, H, D = c["B"], c["Hkv"], c["D"]
    n = ca["v"][0].shape[2]
    V = _dequant(*ca["v"], (B, H, n, D))
    K = _dequant(*ca["k"], (B, H, n, D))
    if not c["kmode"]:
        pos = ca["tail_base"][:, None] + torch.arange(32, device=DEV)
        ok = pos < n
        bi, j = ok.nonzero(as_tuple=True)
        K[bi, :, pos[bi, j]] = ca["tail"][bi, :, j].float()
    return K, V


def _run_plain(st):
    c = st["c"]
    return {"rope": _plain_rope, "tree": _plain_attn, "scored": _plain_attn, "commit": _plain_commit,
            "read": _plain_read}[c["op"]](st)


def _plain_rope(st):
    c = st["c"]
    B, n, H, G, D, R = c["B"], c["n"], c["Hkv"], c["G"], c["D"], c["rot"]
    Hq = H * G
    x = st["qkv"].float()
    q = x[..., :Hq * D].reshape(B, n, Hq, D)
    k = x[..., Hq * D:(Hq + H) * D].reshape(B, n, H, D)
    v = st["qkv"][..., (Hq + H) * D:].reshape(B, n, H, D)
    off = torch.arange(n, device=DEV)[None].expand(B, n) if st["offset"] is None else st["offset"]
    ang = (c["L"] + off).double()[..., None] * st["inv_freq"].double()      # far positions need 64 bits
    cos, sin = ang.cos().float()[:, :, None], ang.sin().float()[:, :, None]

    def one(t, w):
        if w is not None:
            t = t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * w
        a, b = (t[..., 0:R:2], t[..., 1:R:2]) if c["inter"] else (t[..., :R // 2], t[..., R // 2:R])
        y = t.clone()
        ya, yb = a * cos - b * sin, b * cos + a * sin
        if c["inter"]:
            y[..., 0:R:2], y[..., 1:R:2] = ya, yb
        else:
            y[..., :R // 2], y[..., R // 2:R] = ya, yb
        return y.to(torch.bfloat16)

    return (one(q, st["wq"]), one(k, st["wk"]).transpose(1, 2).contiguous(), v.transpose(1, 2).contiguous())


def _plain_attn(st):
    c = st["c"]
    B, H, G, D = c["B"], c["Hkv"], c["G"], c["D"]
    K, V = _plain_kv(st)
    n, T = K.shape[2], st["q"].shape[1]
    lens = st["lens"]
    pos_k = torch.arange(n, device=DEV)[None].expand(B, n)
    ok = (pos_k < lens[:, None])[:, None].expand(B, T, n)
    if c["op"] == "tree":
        depth = torch.arange(T, device=DEV)[None].expand(B, T) if st["depth"] is None else st["depth"]
        pos_q = lens[:, None] + depth
        if st["mask"] is None:
            vis = torch.ones((T, T), dtype=torch.bool, device=DEV).tril()[None].expand(B, T, T)
        else:
            vis = ((st["mask"][..., None] >> torch.arange(32, device=DEV, dtype=torch.int32)) & 1).reshape(B, T, -1)
            vis = vis[..., :T].bool()
        vis = vis & (torch.arange(T, device=DEV) < st["nd"][:, None])[:, None]
        K, V = torch.cat([K, st["Kd"].float()], 2), torch.cat([V, st["Vd"].float()], 2)
        ok, pos_k = torch.cat([ok, vis], 2), torch.cat([pos_k, pos_q], 1)
    else:
        pos_q = lens[:, None] - 1
    q = st["q"].float().reshape(B, T, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * T, D)
    s = torch.matmul(q, K.transpose(2, 3)).mul_(D ** -0.5).view(B, H, G, T, -1)
    if c["cap"]:
        s = torch.tanh(s.div_(c["cap"])).mul_(c["cap"])
    dist = pos_q[:, :, None] - pos_k[:, None]
    if st["alibi"] is not None:
        s -= st["alibi"].view(H, G, 1, 1) * dist.float()[:, None, None]
    if c["window"]:
        ok = ok & (dist < c["window"])
    s.masked_fill_(~ok[:, None, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    m = torch.where(m == float("-inf"), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(B, H, G * T, -1), V).view(B, H, G, T, D) / torch.where(l == 0, torch.ones_like(l), l)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, H * G, D)
    if c["op"] == "scored":
        return o[:, 0].to(torch.bfloat16)
    o = torch.where((torch.arange(T, device=DEV) < st["nd"][:, None])[:, :, None, None], o, torch.zeros_like(o))
    return o.to(torch.bfloat16)


def _plain_commit(st):
    c = st["c"]
    B, H, D, n = c["B"], c["Hkv"], c["D"], c["n"]
    idx = st["index"].long()[:, None, :, None].expand(B, H, n, D)
    K, V = st["Kd"].gather(2, idx), st["Vd"].gather(2, idx)
    Vo = _dequant(*_quant_tokens(V, c["bv"]), (B, H, n, D)).to(torch.bfloat16)
    if c["kmode"]:
        Ko = _dequant(*_quant_tokens(K, c["bk"]), (B, H, n, D)).to(torch.bfloat16)
    else:   # whole groups are quantised, the rest stays bf16
        Ko, full = K.clone(), n // 32 * 32
        if full:
            Kg = _dequant(*_quant_channels(K[:, :, :full], c["bk"]), (B, H, full, D)).to(torch.bfloat16)
            done = torch.arange(full, device=DEV) < (st["acc"] // 32 * 32)[:, None]
            Ko[:, :, :full] = torch.where(done[:, None, :, None], Kg, K[:, :, :full])
    keep = (torch.arange(n, device=DEV) < st["acc"][:, None])[:, None, :, None]
    zero = torch.zeros((), dtype=torch.bfloat16, device=DEV)
    return torch.where(keep, Ko, zero), torch.where(keep, Vo, zero)


def _plain_read(st):
    c = st["c"]
    K, V = _plain_kv(st)
    sl = slice(c["t0"], c["t0"] + c["n"])
    return K[:, :, sl].to(torch.bfloat16), V[:, :, sl].to(torch.bfloat16)


# ------------------------------------------------------------------ what a pass cannot do without
def _cache_bytes(c, L):
    """Packed bytes of L tokens of one (sequence, kv head)."""
    D = c["D"]
    r = 0 if c["kmode"] else L % 32
    kb = (L - r) * D * c["bk"] / 8 + (L * D / 32 * 4 if c["kmode"] else L // 32 * D * 4) + r * D * 2
    return kb + L * D * c["bv"] / 8 + L * D / 32 * 4


def work(case):
    c = case
    op, B, H, G, D = c["op"], c["B"], c["Hkv"], c["G"], c["D"]
    Hq = H * G
    if op == "rope":
        rows = B * c["n"]
        by = rows * (Hq + 2 * H) * D * 2 * 2 + (rows * 4 if c["offset"] else 0) + c["rot"] * 2
        return {"bytes": by, "flops": rows * (Hq + H) * (4 * D * c["norm"] + 3 * c["rot"])}
    if op in ("tree", "scored"):
        by = fl = 0
        T = c.get("T", 1)
        nd = _drafts(c) if op == "tree" else [1] * B
        for L, t in zip(_lens(c), nd):
            seen = min(L, c["window"] + t) if c["window"] else L
            own_keys = (t if c["tree"] else (t + 1) / 2) if op == "tree" else 0
            by += H * _cache_bytes(c, seen) + 2 * t * Hq * D * 2
            if op == "tree":
                by += 2 * t * H * D * 2 + (t * (T + 31) // 32 * 4 + 4 * t if c["tree"] else 0)
            fl += 4 * D * Hq * t * (min(L, c["window"]) if c["window"] else L) + 4 * D * Hq * t * own_keys
        return {"bytes": by, "flops": fl}
    if op == "commit":
        n = sum(_accepted(c))
        pk = sum(_cache_bytes(c, a) for a in _accepted(c)) * H
        return {"bytes": 2 * n * H * D * 2 * 2 + 2 * pk, "flops": n * H * D * 2 * 6}
    by = B * H * (_cache_bytes(c, c["n"]) + 2 * c["n"] * D * 2)
    return {"bytes": by, "flops": B * H * c["n"] * D * 2 * 2}


# ------------------------------------------------------------------ exact values
def _x_group(x, bits, axis):
    """Values a group quantiser stands for, 64 bits; its rounded steps as defined."""
    lo, hi = torch.aminmax(x, dim=axis, keepdim=True)
    levels = 2 ** bits - 1
    scale = torch.div(hi - lo, torch.full_like(hi, levels)).to(torch.float16).float()
    zero = lo.to(torch.float16).float()
    code = torch.div(x - zero, scale)
    code = torch.clamp(torch.round(torch.nan_to_num(code, nan=0.0, posinf=0.0, neginf=0.0)), min=0, max=levels)
    code[(scale == 0).expand_as(code)] = 0
    return code.double() * scale.double() + zero.double()


def _x_values(c, K, V, L):
    """One sequence's cache values [Hkv, L, D] in 64 bits from its bf16 keys and values."""
    H, D = K.shape[0], K.shape[2]
    V = _x_group(V[:, :L].float().reshape(H, L, D // 32, 32), c["bv"], 3).reshape(H, L, D)
    K = K[:, :L]
    if c["kmode"]:
        return _x_group(K.float().reshape(H, L, D // 32, 32), c["bk"], 3).reshape(H, L, D), V
    whole = L - L % 32
    parts = []
    if whole:
        parts.append(_x_group(K[:, :whole].float().reshape(H, whole // 32, 32, D), c["bk"], 2).reshape(H, whole, D))
    parts.append(K[:, whole:].double())
    return torch.cat(parts, 1), V


def exact(case, seed):
    c = case
    if work(c)["flops"] > 2e12:
        return None
    return {"rope": _x_rope, "tree": _x_attn, "scored": _x_attn, "commit": _x_commit, "read": _x_read}[c["op"]](c, seed)


def _inputs(c, seed):
    """The inputs of prepare, without the framework's cache."""
    global own
    keep, own = own, False
    try:
        return prepare(c, seed)
    finally:
        own = keep


def _x_rope(c, seed):
    st = _inputs(c, seed)
    B, n, H, G, D, R = c["B"], c["n"], c["Hkv"], c["G"], c["D"], c["rot"]
    x = st["qkv"].double().reshape(B, n, H * G + 2 * H, D)
    out = x.clone()
    p = torch.full((B, n), float(c["L"]), dtype=torch.float64, device=DEV)
    p += torch.arange(n, device=DEV).double() if st["offset"] is None else st["offset"].double()
    for h in range(H * G + H):
        w = st["wq"] if h < H * G else st["wk"]
        y = x[:, :, h]
        if w is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / D + 1e-6) * w.double()
        out[:, :, h] = y
        for i in range(R // 2):
            i0, i1 = (2 * i, 2 * i + 1) if c["inter"] else (i, i + R // 2)
            th = p * st["inv_freq"][i].double()
            co, si = torch.cos(th), torch.sin(th)
            out[:, :, h, i0] = y[:, :, i0] * co - y[:, :, i1] * si
            out[:, :, h, i1] = y[:, :, i0] * si + y[:, :, i1] * co
    k = out[:, :, H * G:H * G + H].permute(0, 2, 1, 3)
    return out[:, :, :H * G], k, out[:, :, H * G + H:].permute(0, 2, 1, 3)


def _cached_inputs(c, seed):
    """The bf16 keys and values that prepare puts into the cache, redrawn, then the rest."""
    g = _gen(seed)
    K, V = _kv(c, (max(_lens(c)) + 31) // 32 * 32, g)
    return K, V, g


def _x_attn(c, seed):
    K, V, g = _cached_inputs(c, seed)
    B, H, G, D, T = c["B"], c["Hkv"], c["G"], c["D"], c.get("T", 1)
    Hq = H * G
    q = torch.randn((B, T, Hq, D), generator=g, device=DEV).to(torch.bfloat16)
    tree = c["op"] == "tree"
    if tree:
        Kd, Vd = _kv(c, T, g)
        nd = _drafts(c)
        vis, depth = _tree(c, g) if c["tree"] else (np.tril(np.ones((B, T, T), bool)),
                                                     np.tile(np.arange(T, dtype=np.int32), (B, 1)))
    out = torch.zeros((B, T, Hq, D), dtype=torch.float64, device=DEV)
    slope = [2.0 ** (-8.0 * (i + 1) / Hq) for i in range(Hq)]
    for b, L in enumerate(_lens(c)):
        Kb, Vb = _x_values(c, K[b], V[b], L)
        kp = torch.arange(L, device=DEV).double()
        if tree:
            t = nd[b]
            d = torch.from_numpy(depth[b, :t]).to(DEV).double()
            qp, kp = L + d, torch.cat([kp, L + d])
            Kb, Vb = torch.cat([Kb, Kd[b, :, :t].double()], 1), torch.cat([Vb, Vd[b, :, :t].double()], 1)
            see = torch.ones((t, L + t), dtype=torch.bool, device=DEV)
            see[:, L:] = torch.from_numpy(vis[b, :t, :t]).to(DEV)
        else:
            t, qp = 1, torch.full((1,), L - 1.0, dtype=torch.float64, device=DEV)
            see = torch.ones((1, L), dtype=torch.bool, device=DEV)
        dist = qp[:, None] - kp[None]
        if c["window"]:
            see &= dist < c["window"]
        for h in range(Hq):
            s = q[b, :t, h].double() @ Kb[h // G].T / math.sqrt(D)
            if c["cap"]:
                s = c["cap"] * torch.tanh(s / c["cap"])
            if c["alibi"]:
                s = s - float(np.float32(slope[h])) * dist
            s = torch.where(see, s, torch.full_like(s, -math.inf))
            top = s.max(1, keepdim=True).values
            e = torch.where(see, torch.exp(s - torch.where(torch.isinf(top), 0.0, top)), 0.0)
            den = e.sum(1, keepdim=True)
            out[b, :t, h] = torch.where(den > 0, (e @ Vb[h // G]) / den, 0.0)
    return out if tree else out[:, 0]


def _x_commit(c, seed):
    _, _, g = _cached_inputs(c, seed)
    Kd, Vd = _kv(c, c["T"], g)
    B, H, D, n = c["B"], c["Hkv"], c["D"], c["n"]
    pick = torch.rand((B, c["T"]), generator=g, device=DEV).argsort(1)[:, :n].sort(1).values
    Ko = torch.zeros((B, H, n, D), dtype=torch.float64, device=DEV)
    Vo = torch.zeros_like(Ko)
    for b, a in enumerate(_accepted(c)):
        rows = pick[b, :a]
        Ko[b, :, :a], Vo[b, :, :a] = _x_values(c, Kd[b][:, rows], Vd[b][:, rows], a)
    return Ko, Vo


def _x_read(c, seed):
    K, V, _ = _cached_inputs(c, seed)
    outs = [_x_values(c, K[b], V[b], L) for b, L in enumerate(_lens(c))]
    sl = slice(c["t0"], c["t0"] + c["n"])
    return (torch.stack([o[0][:, sl] for o in outs]), torch.stack([o[1][:, sl] for o in outs]))
