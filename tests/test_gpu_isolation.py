"""An infinite or NaN value appended to one request leaves the attention of the others, bit for bit."""
import pytest
import torch

from layer_wise_mixed_b200 import kvq

from test_gpu_tree import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("val", [float("inf"), -float("inf"), float("nan"), 3e38, -7e4])
@pytest.mark.parametrize("kmode", [0, 1])
def test_other_requests_keep_their_bits(kmode, val):
    L, T = 70, 6
    c = Case([L, L, L], T, kmode=kmode, bits=(8, 8), seed=4)
    c.V[1].mul_(2.0 ** -6)   # (small scales: a scaling of the layer would cost them bits)
    kvq.kvq_reset_sequences(c.cache.h, [0, 1, 2])
    c.cache.append(0, c.K, c.V)
    tree = c.cache.tree_attn(0, c.q, c.Kd, c.Vd)
    Kn, Vn = c.K[:, :, :1].contiguous(), c.V[:, :, :1].contiguous()
    Vn[0, 0, 0, 5] = val
    Kn[0, 1, 0, 7] = val
    c.cache.append_ragged(0, Kn, Vn, [1, 0, 0])
    assert torch.equal(c.cache.tree_attn(0, c.q, c.Kd, c.Vd)[1:], tree[1:])
    assert kvq.kvq_device_status(c.cache.h) == 0


def outputs(c, q):
    opts = kvq.ScoreOpts(30.0, window=50)
    return [c.decode_attn(0, q, out_fp32=True), c.decode_attn_scored(0, q, opts, out_fp32=True)]


@pytest.mark.parametrize("val", [float("inf"), -float("inf"), float("nan"), 3e38])
@pytest.mark.parametrize("kmode", [0, 1])
@pytest.mark.parametrize("how", ["append", "fused"])
def test_decode_of_other_requests(how, kmode, val):
    """The decode kernels scale their operands by the layer's largest scale: beside a request that
    was given an infinity, the others come out as beside one that was given a finite value.  The
    append completes a key group (two launches in the fused call)."""
    L, D = 63 if how == "append" else 70, 128
    outs = []
    for v in (0.5, val):
        c = Case([L, L, L], 1, kmode=kmode, bits=(8, 4), seed=6)
        c.V[2].mul_(4.0)   # the largest scales are in another request, with either value
        c.K[2].mul_(4.0)
        kvq.kvq_reset_sequences(c.cache.h, [0, 1, 2])
        c.cache.append(0, c.K, c.V)
        Kn, Vn = (torch.randn((3, c.Hkv, 1, D), generator=torch.Generator(device="cuda").manual_seed(i), device="cuda")
                  .to(torch.bfloat16) for i in (1, 2))
        Kn[0, 1, 0, 7] = v
        Vn[0, 0, 0, 5] = v
        q = c.q[:, 0].contiguous()
        if how == "append":
            c.cache.append(0, Kn, Vn)
            first = []
        else:
            first = [c.cache.append_decode(0, Kn, Vn, q, out_fp32=True)]
        outs.append(first + outputs(c.cache, q))
        assert kvq.kvq_device_status(c.cache.h) == 0
    for a, b in zip(*outs):
        assert torch.isfinite(a).all() and torch.equal(a[1:], b[1:])


@pytest.mark.parametrize("val", [float("inf"), float("nan"), 3e38])
def test_paged_decode_of_other_requests(val):
    B, Hkv, G, D, L = 3, 2, 4, 128, 96
    outs = []
    for v in (0.5, val):
        g = torch.Generator(device="cuda").manual_seed(3)
        K, V = (torch.randn((B, Hkv, L, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        q = torch.randn((B, Hkv * G, D), generator=g, device="cuda").to(torch.bfloat16)
        K[2].mul_(4.0)
        V[2].mul_(4.0)
        K[0, 1, 40, 7] = V[0, 0, 41, 5] = v
        cache = kvq.Cache(1, B, Hkv, Hkv * G, D, L, avg_bits=3.0)
        tags = torch.where(torch.arange(L, device="cuda") % 2 == 0, 2, 4).to(torch.uint8).expand(B, -1).contiguous()
        cache.append_tagged(0, K, V, tags)
        outs.append(cache.decode_attn(0, q, out_fp32=True))
    assert torch.isfinite(outs[0]).all() and torch.equal(outs[0][1:], outs[1][1:])
