"""Calls on a stream that is not the current one, given as a torch stream or as a raw handle:
what the call allocates must be memory of that stream.  Memory of the current stream would be
handed out again there while the call's kernels still wait on the other stream."""
import numpy as np
import pytest
import torch

from layer_wise_mixed_b200 import inputs, kvq

from test_gpu_parity import workload

pytestmark = pytest.mark.gpu

HANDLE = pytest.mark.parametrize("handle", [False, True], ids=["stream", "handle"])


def setup():
    B, Hkv, G, D, T = 2, 2, 4, 128, 8
    wl = workload(B, Hkv, G, D, name="streams")
    K, V = inputs.layer_kv(wl, 0, 700, "cuda")
    cache = kvq.Cache(1, B, Hkv, Hkv * G, D, 720, [(4, 2)])
    cache.append_ragged(0, K, V, [700, 300])
    Kd, Vd = inputs.layer_kv(wl, 0, T, "cuda", tag="draft")
    q = torch.randn((B, T, Hkv * G, D), generator=torch.Generator(device="cuda").manual_seed(3), device="cuda")
    qkv = torch.randn((B, T, (Hkv * G + 2 * Hkv) * D), device="cuda").to(torch.bfloat16)
    return cache, q.to(torch.bfloat16), Kd, Vd, qkv


def tensors(x):
    return [x] if torch.is_tensor(x) else list(x)


@HANDLE
def test_workspace_of_the_call_is_not_handed_out_again(handle, monkeypatch):
    """tree_attn without a workspace, split, on a stream that is busy: a tensor that the current
    stream allocates right after the call, of the workspace's size, is other memory."""
    cache, q, Kd, Vd, _ = setup()
    kvq.kvq_set_num_splits(cache.h, 4)
    want = cache.tree_attn(0, q, Kd, Vd)
    out = torch.zeros_like(want)
    taken = []
    make = kvq.Cache.tree_workspace

    def tree_workspace(self, T):
        ws = make(self, T)
        taken.append((ws.data_ptr(), ws.numel()))
        return ws
    monkeypatch.setattr(kvq.Cache, "tree_workspace", tree_workspace)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)   # about 10 ms
    cache.tree_attn(0, q, Kd, Vd, out=out, stream=side.cuda_stream if handle else side)
    (ptr, n), = taken
    others = [torch.zeros(n, dtype=torch.uint8, device="cuda") for _ in range(4)]
    assert all(o.data_ptr() + n <= ptr or ptr + n <= o.data_ptr() for o in others)
    torch.cuda.synchronize()
    assert torch.equal(out, want) and not any(o.any() for o in others)
    assert kvq.kvq_device_status(cache.h) == 0


@HANDLE
def test_fresh_outputs_are_memory_of_the_call_s_stream(handle):
    """The current stream's freed blocks, which its queued work may still use, are not what a
    call on another stream writes its outputs to; the results are those of the current stream."""
    cache, q, Kd, Vd, qkv = setup()
    rope = kvq.Rope(128, torch.rand(64, device="cuda"))
    calls = {
        "norm_rope": lambda s: cache.norm_rope(0, qkv, rope, stream=s),
        "tree_attn": lambda s: cache.tree_attn(0, q, Kd, Vd, stream=s),
        "decode_attn_scored": lambda s: cache.decode_attn_scored(0, q[:, 0].contiguous(), kvq.ScoreOpts(30.0), stream=s),
        "decode_attn": lambda s: cache.decode_attn(0, q[:, 0].contiguous(), stream=s),
        "read": lambda s: cache.read(0, 5, 290, stream=s),
    }
    for name, call in calls.items():
        want = tensors(call(None))
        keep = [w.clone() for w in want]
        freed = {w.data_ptr() for w in want}
        sizes = [(w.shape, w.dtype) for w in want]
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        del want                       # back to the current stream's pool
        got = tensors(call(side.cuda_stream if handle else side))
        assert not freed & {g.data_ptr() for g in got}, name
        torch.cuda.synchronize()
        assert [(g.shape, g.dtype) for g in got] == sizes, name
        assert all(torch.equal(g, k) for g, k in zip(got, keep)), name


def test_append_on_another_stream():
    cache, q, Kd, Vd, _ = setup()
    other = setup()[0]
    index = torch.tensor([[0, 3, 5], [1, 1, 7]], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    cache.append_selected(0, Kd, Vd, index, [3, 2], stream=side.cuda_stream)
    torch.cuda.current_stream().wait_stream(side)
    other.append_selected(0, Kd, Vd, index, [3, 2])
    assert np.array_equal(cache.export_layer(0), other.export_layer(0))


def test_a_stream_object_of_another_library():
    """Any object that holds the handle as cuda_stream names a stream, as in the older calls."""
    class Other:
        cuda_stream = torch.cuda.Stream().cuda_stream
    cache, q, Kd, Vd, _ = setup()
    want = cache.tree_attn(0, q, Kd, Vd)
    torch.cuda.synchronize()
    got = cache.tree_attn(0, q, Kd, Vd, stream=Other())
    torch.cuda.synchronize()
    assert torch.equal(got, want)
