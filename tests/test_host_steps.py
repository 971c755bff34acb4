"""Host-side refusals of the multi-token step entry points (no GPU: every call below fails
before any launch, or does nothing) and of their Python wrappers."""
import ctypes

import pytest
import torch

from layer_wise_mixed_b200 import build as kbuild
from layer_wise_mixed_b200 import kvq

FAKE = 1 << 40   # never dereferenced


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kvq.load()


@pytest.fixture()
def plan(lib):
    h = kvq.kvq_plan(kvq.make_desc(1, 2, 2, 8, 64, 100, [(4, 2)]))
    kvq.kvq_bind(h, FAKE, kvq.kvq_workspace_bytes(h))
    yield h
    kvq.kvq_destroy(h)


def rope(**kw):
    d = dict(rot_dim=64, interleaved=0, inv_freq=FAKE, q_weight=None, k_weight=None, eps=1e-6)
    d.update(kw)
    return ctypes.byref(kvq.kvq_rope_desc(*d.values()))


def opts(cap=0.0, alibi=None, window=0, scale=0.0):
    return ctypes.byref(kvq.kvq_score_opts(cap, alibi, window, scale))


def test_norm_rope(lib, plan):
    W = (8 + 4) * 64
    ok = dict(layer=0, qkv=FAKE, bs=W, ts=W, n=1, off=None, rope=rope(), q=FAKE, K=FAKE, V=FAKE)

    def call(**kw):
        a = {**ok, **kw}
        return lib.kvq_norm_rope(plan, *a.values(), None)
    assert call(layer=1) == kvq.KVQ_EINVAL
    for name in ("qkv", "rope", "q", "K", "V"):
        assert call(**{name: None}) == kvq.KVQ_EINVAL, name
    for name in ("qkv", "q", "K", "V"):
        assert call(**{name: FAKE + 8}) == kvq.KVQ_EALIGN, name
    assert call(off=FAKE + 2) == kvq.KVQ_EALIGN
    assert call(n=0) == kvq.KVQ_EINVAL
    assert call(ts=W - 8) == kvq.KVQ_EINVAL
    assert call(ts=W + 4) == kvq.KVQ_EINVAL
    assert call(bs=-8) == kvq.KVQ_EINVAL
    assert call(bs=4) == kvq.KVQ_EINVAL
    assert call(rope=rope(rot_dim=-16)) == kvq.KVQ_EINVAL
    assert call(rope=rope(rot_dim=80)) == kvq.KVQ_EINVAL
    assert call(rope=rope(rot_dim=24)) == kvq.KVQ_EUNSUPPORTED
    assert call(rope=rope(inv_freq=None)) == kvq.KVQ_EINVAL
    assert call(rope=rope(q_weight=FAKE + 1)) == kvq.KVQ_EALIGN
    assert call(rope=rope(eps=-1.0)) == kvq.KVQ_EINVAL
    assert call(rope=rope(eps=float("nan"))) == kvq.KVQ_EINVAL
    assert call(n=1 << 30) == kvq.KVQ_EUNSUPPORTED


def test_tree_attn(lib, plan):
    n = ctypes.c_size_t()
    assert lib.kvq_tree_attn_workspace_bytes(plan, 0, ctypes.byref(n)) == kvq.KVQ_EINVAL
    assert lib.kvq_tree_attn_workspace_bytes(plan, 4097, ctypes.byref(n)) == kvq.KVQ_EUNSUPPORTED
    assert lib.kvq_tree_attn_workspace_bytes(plan, 4, None) == kvq.KVQ_EINVAL
    assert lib.kvq_tree_attn_workspace_bytes(None, 4, ctypes.byref(n)) == kvq.KVQ_EINVAL
    need = kvq.kvq_tree_attn_workspace_bytes(plan, 4)
    nd = (ctypes.c_int32 * 2)(4, 4)
    ok = dict(layer=0, q=FAKE, K=FAKE, V=FAKE, T=4, nd=None, mask=None, depth=None, opts=None, out=FAKE, fp32=0, ws=FAKE,
              wb=need)

    def call(**kw):
        a = {**ok, **kw}
        return lib.kvq_tree_attn(plan, *a.values(), None)
    assert call(layer=-1) == kvq.KVQ_EINVAL
    for name in ("q", "K", "V", "out"):
        assert call(**{name: None}) == kvq.KVQ_EINVAL, name
        assert call(**{name: FAKE + 4}) == kvq.KVQ_EALIGN, name
    assert call(mask=FAKE + 2) == kvq.KVQ_EALIGN
    assert call(depth=FAKE + 1) == kvq.KVQ_EALIGN
    assert call(T=0) == kvq.KVQ_EINVAL
    assert call(T=5000) == kvq.KVQ_EUNSUPPORTED
    for bad in ((5, 4), (4, -1)):
        assert call(nd=(ctypes.c_int32 * 2)(*bad)) == kvq.KVQ_EINVAL
    assert call(ws=None) == kvq.KVQ_EUNBOUND
    assert call(wb=need - 1) == kvq.KVQ_EUNBOUND
    assert call(ws=FAKE + 128) == kvq.KVQ_EALIGN
    assert call(opts=opts(cap=-1.0)) == kvq.KVQ_EINVAL
    assert call(opts=opts(cap=float("inf"))) == kvq.KVQ_EINVAL
    assert call(opts=opts(cap=float("nan"))) == kvq.KVQ_EINVAL
    assert call(opts=opts(window=-1)) == kvq.KVQ_EINVAL
    assert call(opts=opts(scale=float("nan"))) == kvq.KVQ_EINVAL
    assert call(opts=opts(alibi=FAKE + 2)) == kvq.KVQ_EALIGN
    assert call(nd=(ctypes.c_int32 * 2)(0, 0)) == kvq.KVQ_OK     # no drafted token: nothing to do


def test_scored_decode(lib, plan):
    call = lambda **kw: lib.kvq_decode_attn_scored(plan, *{**dict(layer=0, q=FAKE, o=None, out=FAKE, fp32=0), **kw}.values(),
                                                   None)
    assert call() == kvq.KVQ_EINVAL and "empty" in kvq.kvq_last_error()
    assert call(q=None) == kvq.KVQ_EINVAL
    assert call(out=FAKE + 8) == kvq.KVQ_EALIGN
    assert call(o=opts(window=-3)) == kvq.KVQ_EINVAL
    assert call(layer=7) == kvq.KVQ_EINVAL


def test_append_selected_and_read(lib, plan):
    ok = dict(layer=0, K=FAKE, V=FAKE, n_src=4, index=FAKE, n_new=None, n_max=2)
    call = lambda **kw: lib.kvq_append_selected(plan, *{**ok, **kw}.values(), None)
    assert call(K=None) == kvq.KVQ_EINVAL
    assert call(index=None) == kvq.KVQ_EINVAL
    assert call(index=FAKE + 2) == kvq.KVQ_EALIGN
    assert call(V=FAKE + 8) == kvq.KVQ_EALIGN
    assert call(n_src=0) == kvq.KVQ_EINVAL
    assert call(n_max=0) == kvq.KVQ_EINVAL
    assert call(n_max=101) == kvq.KVQ_ECAPACITY
    assert call(n_new=(ctypes.c_int32 * 2)(1, 3)) == kvq.KVQ_EINVAL
    assert call(n_new=(ctypes.c_int32 * 2)(0, 0)) == kvq.KVQ_OK   # nothing appended
    read = lambda t0, n, K=FAKE, V=FAKE: lib.kvq_read(plan, 0, t0, n, K, V, None)
    assert read(0, 1) == kvq.KVQ_EINVAL        # empty layer
    assert read(-1, 1) == kvq.KVQ_EINVAL
    assert read(0, 0) == kvq.KVQ_EINVAL
    assert read(0, 1, None, None) == kvq.KVQ_EINVAL
    assert read(0, 1, FAKE + 8) == kvq.KVQ_EALIGN
    assert read(2 ** 31 - 1, 2 ** 31 - 1) == kvq.KVQ_EINVAL


def test_unbound_and_paged_plans(lib):
    h = kvq.kvq_plan(kvq.make_desc(1, 2, 2, 8, 64, 100, [(4, 2)]))
    p = kvq.kvq_plan(kvq.make_paged_desc(1, 2, 2, 8, 128, 100, 3.0))
    try:
        for hh, code in ((h, kvq.KVQ_EUNBOUND), (p, kvq.KVQ_EUNSUPPORTED)):
            assert lib.kvq_norm_rope(hh, 0, FAKE, 2048, 2048, 1, None, rope(), FAKE, FAKE, FAKE, None) == code
            assert lib.kvq_tree_attn(hh, 0, FAKE, FAKE, FAKE, 1, None, None, None, None, FAKE, 0, FAKE, 1 << 30, None) == code
            assert lib.kvq_decode_attn_scored(hh, 0, FAKE, None, FAKE, 0, None) == code
            assert lib.kvq_append_selected(hh, 0, FAKE, FAKE, 1, FAKE, None, 1, None) == code
            assert lib.kvq_read(hh, 0, 0, 1, FAKE, FAKE, None) == code
    finally:
        kvq.kvq_destroy(h)
        kvq.kvq_destroy(p)


def test_python_wrappers_refuse_wrong_tensors(lib):
    cache = kvq.Cache(1, 2, 2, 8, 64, 100, [(4, 2)], device="cpu")   # host memory: nothing is launched below
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)
    q, K, i32 = bf(2, 4, 8, 64), bf(2, 2, 4, 64), torch.zeros((2, 4), dtype=torch.int32)
    bad = [lambda: cache.tree_attn(0, q[:, :, :7], K, K),
           lambda: cache.tree_attn(0, q.float(), K, K),
           lambda: cache.tree_attn(0, q, K[:, :, :3], K),
           lambda: cache.tree_attn(0, q, K, K.transpose(2, 3).contiguous().transpose(2, 3)),
           lambda: cache.tree_attn(0, q, K, K, n_draft=[1]),
           lambda: cache.tree_attn(0, q, K, K, mask=torch.zeros((2, 4, 2), dtype=torch.int32)),
           lambda: cache.tree_attn(0, q, K, K, mask=torch.zeros((2, 4, 1), dtype=torch.int64)),
           lambda: cache.tree_attn(0, q, K, K, depth=i32[:, :3]),
           lambda: cache.tree_attn(0, q, K, K, opts=kvq.ScoreOpts(alibi=torch.zeros(7))),
           lambda: cache.decode_attn_scored(0, q),
           lambda: cache.append_selected(0, K, K, i32[:1]),
           lambda: cache.append_selected(0, K, K, i32.long()),
           lambda: cache.append_selected(0, K, K, i32, n_new=[1, 1, 1]),
           lambda: cache.norm_rope(0, bf(2, 3, 100), kvq.Rope(0)),
           lambda: cache.norm_rope(0, torch.zeros((2, 3, 768)), kvq.Rope(0)),
           lambda: cache.norm_rope(0, bf(2, 3, 768), kvq.Rope(0, None, torch.ones(63))),
           lambda: cache.norm_rope(0, bf(2, 3, 768), kvq.Rope(0), offset=i32),
           lambda: kvq.Rope(64, torch.zeros(31)),
           lambda: kvq.Rope(64, torch.zeros(32, dtype=torch.float64)),
           lambda: kvq.ScoreOpts(alibi=torch.zeros(8, dtype=torch.float16))]
    for i, f in enumerate(bad):
        with pytest.raises(ValueError):
            f()
