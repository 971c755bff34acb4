"""Cache calls refuse memory of another device before anything is launched: every tensor, the
ones inside a Rope and a ScoreOpts and the workspace among them.  No GPU: the "meta" device is
the cache's here and host tensors are the foreign ones, then a host cache is refused itself."""
import pytest
import torch

from layer_wise_mixed_b200 import build as kbuild
from layer_wise_mixed_b200 import kvq

B, HKV, HQ, D, T = 2, 2, 8, 64, 4


@pytest.fixture()
def launches(monkeypatch):
    """The C entry points of the step calls, replaced by a record of their names."""
    kbuild.build()
    names = []
    for f in ("kvq_norm_rope", "kvq_tree_attn", "kvq_decode_attn_scored", "kvq_append_selected", "kvq_read"):
        monkeypatch.setattr(kvq, f, lambda *a, _f=f: names.append(_f))
    return names


def cache_on(device):
    c = kvq.Cache(1, B, HKV, HQ, D, 100, [(4, 2)], device="cpu")
    c._dev = torch.device(device)
    return c


def bf(*s, device="meta"):
    return torch.zeros(s, dtype=torch.bfloat16, device=device)


def refused(call, word):
    with pytest.raises(ValueError, match=word):
        call()


def test_host_tensors_inside_options_are_refused(launches):
    c = cache_on("meta")
    qkv = bf(B, 3, (HQ + 2 * HKV) * D)
    f32 = lambda n: torch.zeros(n)
    for rope in (kvq.Rope(64, f32(32)), kvq.Rope(0, None, f32(64)), kvq.Rope(0, None, None, f32(64))):
        refused(lambda: c.norm_rope(0, qkv, rope), "inv_freq and weights are on cpu")
    refused(lambda: kvq.Rope(64, f32(32), torch.zeros(64, device="meta")), "different devices")
    q, K = bf(B, T, HQ, D), bf(B, HKV, T, D)
    opts = kvq.ScoreOpts(alibi=f32(HQ))
    refused(lambda: c.tree_attn(0, q, K, K, opts=opts), "alibi is on cpu")
    refused(lambda: c.decode_attn_scored(0, bf(B, HQ, D), opts), "alibi is on cpu")
    assert launches == []


def test_workspaces_are_checked(launches):
    c = cache_on("meta")
    q, K = bf(B, T, HQ, D), bf(B, HKV, T, D)
    n = kvq.kvq_tree_attn_workspace_bytes(c.h, T)
    refused(lambda: c.tree_attn(0, q, K, K, workspace=torch.zeros(n, dtype=torch.uint8)), "workspace")
    # an expanded tensor counts more elements than it has memory
    one = torch.zeros(1, dtype=torch.uint8, device="meta").expand(n)
    refused(lambda: c.tree_attn(0, q, K, K, workspace=one), "workspace")
    assert launches == []


def test_a_host_cache_launches_nothing(launches):
    c = cache_on("cpu")
    q, K = bf(B, T, HQ, D, device="cpu"), bf(B, HKV, T, D, device="cpu")
    index = torch.zeros((B, 2), dtype=torch.int32)
    for stream in (None, 0, 1 << 40):
        for call in (lambda: c.norm_rope(0, bf(B, 3, (HQ + 2 * HKV) * D, device="cpu"), kvq.Rope(0), stream=stream),
                     lambda: c.tree_attn(0, q, K, K, stream=stream),
                     lambda: c.decode_attn_scored(0, bf(B, HQ, D, device="cpu"), stream=stream),
                     lambda: c.append_selected(0, K, K, index, stream=stream),
                     lambda: c.read(0, 0, 1, stream=stream)):
            refused(call, "kernels need a CUDA device")
    assert launches == []
