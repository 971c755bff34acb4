"""Python binding of the C ABI in include/kvq.h (ctypes; argument marshalling only).

Every function keeps the C name and forwards to libkvq.so; all computation runs in
the library's CUDA kernels.  There is no fallback: if libkvq.so is missing this module
raises on first use.  PyTorch appears only to pass device pointers and the current
CUDA stream, and (in ``Cache``) to allocate the caller-owned workspace.
"""
from __future__ import annotations

import array
import contextlib
import ctypes
import os
import re
from typing import List, Optional, Sequence, Tuple

import numpy as np

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libkvq.so")
HEADER = os.path.join(os.path.dirname(_HERE), "include", "kvq.h")

KVQ_OK = 0
KVQ_EINVAL = -1
KVQ_EUNSUPPORTED = -2
KVQ_ECAPACITY = -3
KVQ_EUNBOUND = -4
KVQ_EALIGN = -5
KVQ_ECUDA = -6
KVQ_EDEVICE = -7
KVQ_PER_CHANNEL = 0
KVQ_PER_TOKEN = 1
KVQ_DECODE_MMA_SYNC = 0
KVQ_DECODE_TCGEN05 = 1

_NAMES = {0: "KVQ_OK", -1: "KVQ_EINVAL", -2: "KVQ_EUNSUPPORTED", -3: "KVQ_ECAPACITY",
          -4: "KVQ_EUNBOUND", -5: "KVQ_EALIGN", -6: "KVQ_ECUDA", -7: "KVQ_EDEVICE"}


class KvqError(RuntimeError):
    def __init__(self, code: int, msg: str):
        super().__init__(f"{_NAMES.get(code, code)}: {msg}")
        self.code = code


class kvq_layer_cfg(ctypes.Structure):
    _fields_ = [("bk", ctypes.c_int), ("bv", ctypes.c_int), ("kmode", ctypes.c_int), ("vmode", ctypes.c_int)]


class kvq_plan_desc(ctypes.Structure):
    _fields_ = [("num_layers", ctypes.c_int), ("batch", ctypes.c_int), ("n_kv_heads", ctypes.c_int),
                ("n_q_heads", ctypes.c_int), ("head_dim", ctypes.c_int), ("group", ctypes.c_int),
                ("max_ctx", ctypes.c_int), ("layers", ctypes.POINTER(kvq_layer_cfg)),
                ("paged", ctypes.c_int), ("page_tokens", ctypes.c_int), ("avg_bits", ctypes.c_float),
                ("pool_blocks", ctypes.c_int)]


class kvq_rope_desc(ctypes.Structure):
    _fields_ = [("rot_dim", ctypes.c_int), ("interleaved", ctypes.c_int), ("inv_freq", ctypes.c_void_p),
                ("q_weight", ctypes.c_void_p), ("k_weight", ctypes.c_void_p), ("eps", ctypes.c_float)]


class kvq_score_opts(ctypes.Structure):
    _fields_ = [("softcap", ctypes.c_float), ("alibi", ctypes.c_void_p), ("window", ctypes.c_int),
                ("scale", ctypes.c_float)]


_lib = None


def load() -> ctypes.CDLL:
    """Load libkvq.so (raises FileNotFoundError if it was not built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise FileNotFoundError(f"{LIB_PATH} is missing: build it with `python -m layer_wise_mixed_b200.build`")
    L = ctypes.CDLL(LIB_PATH)
    P, I, SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
    sig = {
        "kvq_plan": (I, [ctypes.POINTER(kvq_plan_desc), ctypes.POINTER(P)]),
        "kvq_workspace_bytes": (I, [P, ctypes.POINTER(SZ)]),
        "kvq_bind": (I, [P, P, SZ]),
        "kvq_append": (I, [P, I, P, P, I, P]),
        "kvq_append_tagged": (I, [P, I, P, P, I, P, P, P]),
        "kvq_append_ragged": (I, [P, I, P, P, P, I, P]),
        "kvq_seq_lens": (I, [P, I, P]),
        "kvq_decode_attn": (I, [P, I, P, P, I, P]),
        "kvq_append_decode": (I, [P, I, P, P, P, P, I, P]),
        "kvq_decode_attn_noalloc": (I, [P, I, P, P, I, P]),
        "kvq_set_num_splits": (I, [P, I]),
        "kvq_set_decode_path": (I, [P, I]),
        "kvq_get_num_splits": (I, [P, I, ctypes.POINTER(I)]),
        "kvq_export_layer": (I, [P, I, P, SZ, ctypes.POINTER(SZ)]),
        "kvq_seq_len": (I, [P, I, ctypes.POINTER(I)]),
        "kvq_truncate": (I, [P, I, I]),
        "kvq_reset_sequences": (I, [P, P, I]),
        "kvq_device_status": (I, [P, P, ctypes.POINTER(ctypes.c_uint)]),
        "kvq_tag_distortion": (I, [I, I, I, I, I, I, P, P, P, P, I, P, P, P]),
        "kvq_tag_allocate": (I, [I, P, P, P, ctypes.c_double, P, P]),
        "kvq_tag_distortion_workspace_bytes": (I, [I, I, I, I, I, I, I, ctypes.POINTER(SZ)]),
        "kvq_tag_distortion_device": (I, [I, I, I, I, I, I, P, P, P, P, I, P, SZ, P, P, P, P]),
        "kvq_norm_rope": (I, [P, I, P, ctypes.c_int64, ctypes.c_int64, I, P, ctypes.POINTER(kvq_rope_desc), P, P, P,
                              P]),
        "kvq_tree_attn_workspace_bytes": (I, [P, I, ctypes.POINTER(SZ)]),
        "kvq_tree_attn": (I, [P, I, P, P, P, I, P, P, P, ctypes.POINTER(kvq_score_opts), P, I, P, SZ, P]),
        "kvq_decode_attn_scored": (I, [P, I, P, ctypes.POINTER(kvq_score_opts), P, I, P]),
        "kvq_append_selected": (I, [P, I, P, P, I, P, P, I, P]),
        "kvq_read": (I, [P, I, I, I, P, P, P]),
        "kvq_destroy": (None, [P]),
        "kvq_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        f = getattr(L, name)
        f.restype = res
        f.argtypes = args
    _lib = L
    return L


def header_functions() -> List[str]:
    """Names of the functions declared in include/kvq.h."""
    text = open(HEADER).read()
    return sorted(set(re.findall(r"^\s*KVQ_API\s+(?:int|void|const char)\s*\*?\s*(kvq_\w+)\s*\(", text, re.M)))


def _check(rc: int):
    if rc != KVQ_OK:
        raise KvqError(rc, load().kvq_last_error().decode())
    return rc


_raw_stream = None   # torch's raw-handle form of current_stream (no Stream object per call)


def _stream(stream) -> Optional[int]:
    if stream is None:
        global _raw_stream
        if _raw_stream is None:
            import torch
            get, dev = getattr(torch._C, "_cuda_getCurrentRawStream", None), torch.cuda.current_device
            _raw_stream = (lambda: get(dev())) if get else (lambda: torch.cuda.current_stream().cuda_stream)
        return _raw_stream()
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def _torch_stream(stream, device):
    """The torch stream of a stream object or of a raw handle on `device`."""
    import torch
    if isinstance(stream, torch.cuda.Stream):
        return stream
    if not isinstance(stream, int):
        stream = stream.cuda_stream   # (another library's stream object)
    if stream in (0, 1):   # the legacy default stream's two handles
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(stream, device=device)


def _ptr(x) -> int:
    return x if isinstance(x, int) else x.data_ptr()


# ------------------------------------------------------------------ C names
def kvq_plan(desc: kvq_plan_desc) -> int:
    h = ctypes.c_void_p()
    _check(load().kvq_plan(ctypes.byref(desc), ctypes.byref(h)))
    return h.value


def kvq_workspace_bytes(h: int) -> int:
    n = ctypes.c_size_t()
    _check(load().kvq_workspace_bytes(h, ctypes.byref(n)))
    return n.value


def kvq_bind(h: int, dev_ptr: int, nbytes: int):
    _check(load().kvq_bind(h, dev_ptr, nbytes))


def kvq_append(h: int, layer: int, K, V, n_new: int, stream=None):
    _check(load().kvq_append(h, layer, _ptr(K), _ptr(V), n_new, _stream(stream)))


def kvq_append_tagged(h: int, layer: int, K, V, n_new: int, host_tags, dev_tags, stream=None):
    """host_tags: contiguous uint8 numpy array [B, n_new]; dev_tags: the same bytes on the device."""
    host_tags = np.ascontiguousarray(host_tags, np.uint8)
    _check(load().kvq_append_tagged(h, layer, _ptr(K), _ptr(V), n_new, host_tags.ctypes.data_as(ctypes.c_void_p),
                                    _ptr(dev_tags), _stream(stream)))


def kvq_append_ragged(h: int, layer: int, K, V, n_new, stream=None):
    """K, V [B, Hkv, n_max, D]; request b appends its first n_new[b] tokens."""
    import numpy as np
    n = np.ascontiguousarray(n_new, np.int32)
    _check(load().kvq_append_ragged(h, layer, _ptr(K), _ptr(V), n.ctypes.data_as(ctypes.c_void_p), K.shape[2],
                                    _stream(stream)))


def kvq_seq_lens(h: int, layer: int, batch: int):
    import numpy as np
    out = np.zeros(batch, np.int32)
    _check(load().kvq_seq_lens(h, layer, out.ctypes.data_as(ctypes.c_void_p)))
    return out


def kvq_decode_attn(h: int, layer: int, q, out, out_fp32: bool, stream=None):
    _check(load().kvq_decode_attn(h, layer, _ptr(q), _ptr(out), int(bool(out_fp32)), _stream(stream)))


def kvq_append_decode(h: int, layer: int, K, V, q, out, out_fp32: bool, stream=None):
    _check(load().kvq_append_decode(h, layer, _ptr(K), _ptr(V), _ptr(q), _ptr(out), int(bool(out_fp32)),
                                    _stream(stream)))


def kvq_decode_attn_noalloc(h: int, layer: int, q, out, out_fp32: bool, stream=None):
    _check(load().kvq_decode_attn_noalloc(h, layer, _ptr(q), _ptr(out), int(bool(out_fp32)), _stream(stream)))


def kvq_set_num_splits(h: int, n: int):
    _check(load().kvq_set_num_splits(h, n))


def kvq_set_decode_path(h: int, path: int):
    _check(load().kvq_set_decode_path(h, path))


def kvq_get_num_splits(h: int, layer: int) -> int:
    n = ctypes.c_int()
    _check(load().kvq_get_num_splits(h, layer, ctypes.byref(n)))
    return n.value


def kvq_export_layer(h: int, layer: int) -> np.ndarray:
    need = ctypes.c_size_t()
    _check(load().kvq_export_layer(h, layer, None, 0, ctypes.byref(need)))
    buf = np.empty(need.value, np.uint8)
    _check(load().kvq_export_layer(h, layer, buf.ctypes.data_as(ctypes.c_void_p), buf.nbytes,
                                   ctypes.byref(need)))
    return buf


def kvq_seq_len(h: int, layer: int) -> int:
    n = ctypes.c_int()
    _check(load().kvq_seq_len(h, layer, ctypes.byref(n)))
    return n.value


def kvq_truncate(h: int, layer: int, L: int):
    _check(load().kvq_truncate(h, layer, L))


def kvq_reset_sequences(h: int, seqs):
    n = np.ascontiguousarray(seqs, np.int32)
    _check(load().kvq_reset_sequences(h, n.ctypes.data_as(ctypes.c_void_p), n.size))


def kvq_device_status(h: int, stream=None) -> int:
    f = ctypes.c_uint()
    rc = load().kvq_device_status(h, _stream(stream), ctypes.byref(f))
    _check(rc)
    return f.value


def kvq_destroy(h: int):
    load().kvq_destroy(h)


def kvq_last_error() -> str:
    return load().kvq_last_error().decode()


def kvq_tag_distortion(Q, K, V, tags, num_tags: int):
    """Per-tag distortion from calibration prefills (host numpy arrays): Q uint16 (bf16
    bits) [NL, R, Hq, T, D], K/V [NL, R, Hkv, T, D], tags int32 [R, T].
    Returns (D2, D4, counts)."""
    import numpy as np
    Q = np.ascontiguousarray(Q, np.uint16)
    K = np.ascontiguousarray(K, np.uint16)
    V = np.ascontiguousarray(V, np.uint16)
    tags = np.ascontiguousarray(tags, np.int32)
    NL, R, Hq, T, D = Q.shape
    Hkv = K.shape[2]
    if K.shape != (NL, R, Hkv, T, D) or V.shape != K.shape or tags.shape != (R, T):
        raise ValueError("shape mismatch")
    D2 = np.zeros(num_tags, np.float64)
    D4 = np.zeros(num_tags, np.float64)
    counts = np.zeros(num_tags, np.int64)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(load().kvq_tag_distortion(NL, R, Hq, Hkv, D, T, p(Q), p(K), p(V), p(tags), num_tags, p(D2), p(D4),
                                     p(counts)))
    return D2, D4, counts


def kvq_tag_distortion_workspace_bytes(NL: int, R: int, Hq: int, Hkv: int, D: int, T: int, num_tags: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().kvq_tag_distortion_workspace_bytes(NL, R, Hq, Hkv, D, T, num_tags, ctypes.byref(n)))
    return n.value


def kvq_tag_distortion_device(Q, K, V, tags, num_tags: int, workspace=None, stream=None):
    """kvq_tag_distortion on the GPU: Q, K, V CUDA tensors (bf16 or int16/uint16 holding bf16
    bits) [NL, R, Hq, T, D] / [NL, R, Hkv, T, D]; tags host int32 [R, T].  The workspace
    (a CUDA uint8 tensor) is allocated here when not given.  Returns (D2, D4, counts)."""
    import numpy as np
    import torch
    for a in (Q, K, V):
        if not (a.is_cuda and a.is_contiguous() and a.element_size() == 2):
            raise ValueError("Q, K, V must be contiguous 2-byte CUDA tensors")
    tags = np.ascontiguousarray(tags, np.int32)
    NL, R, Hq, T, D = Q.shape
    Hkv = K.shape[2]
    if tuple(K.shape) != (NL, R, Hkv, T, D) or tuple(V.shape) != tuple(K.shape) or tags.shape != (R, T):
        raise ValueError("shape mismatch")
    need = kvq_tag_distortion_workspace_bytes(NL, R, Hq, Hkv, D, T, num_tags)
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=Q.device)
    D2 = np.zeros(num_tags, np.float64)
    D4 = np.zeros(num_tags, np.float64)
    counts = np.zeros(num_tags, np.int64)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    st = _stream(stream)
    _check(load().kvq_tag_distortion_device(NL, R, Hq, Hkv, D, T, Q.data_ptr(), K.data_ptr(), V.data_ptr(), p(tags),
                                            num_tags, workspace.data_ptr(), workspace.numel(), p(D2), p(D4),
                                            p(counts), st))
    return D2, D4, counts


def kvq_tag_allocate(D2, D4, counts, avg_bits: float):
    """INT2/INT4 per tag under the average-bit budget: (bits int32 [K], total distortion)."""
    import numpy as np
    D2 = np.ascontiguousarray(D2, np.float64)
    D4 = np.ascontiguousarray(D4, np.float64)
    counts = np.ascontiguousarray(counts, np.int64)
    bits = np.zeros(len(counts), np.int32)
    total = ctypes.c_double(0.0)
    p = lambda a: a.ctypes.data_as(ctypes.c_void_p)
    _check(load().kvq_tag_allocate(len(counts), p(D2), p(D4), p(counts), float(avg_bits), p(bits),
                                   ctypes.byref(total)))
    return bits, total.value


def _opt_ptr(x):
    return None if x is None else _ptr(x)


def _host_i32(x):
    """(address, array kept alive) of an optional host int32 array."""
    if x is None:
        return None, None
    if isinstance(x, (list, tuple)):
        a = array.array("i", x)   # (raises for fractions and for what int32 does not hold)
        return a.buffer_info()[0], a
    x = np.asarray(x)
    a = np.ascontiguousarray(x, np.int32)
    if x.dtype.kind not in "iu" or (a != x).any():
        raise ValueError("counts must be integers that int32 holds")
    return a.ctypes.data, a


def _ref(s):
    """byref of an optional structure (Rope and ScoreOpts hold theirs)."""
    if s is None:
        return None
    return getattr(s, "ref", None) or ctypes.byref(s)


_NO_CONTEXT = contextlib.nullcontext()


def kvq_norm_rope(h: int, layer: int, qkv, batch_stride: int, token_stride: int, n: int, offset, rope: kvq_rope_desc,
                  q, K, V, stream=None):
    _check(load().kvq_norm_rope(h, layer, _ptr(qkv), batch_stride, token_stride, n, _opt_ptr(offset),
                                _ref(rope), _ptr(q), _ptr(K), _ptr(V), _stream(stream)))


def kvq_tree_attn_workspace_bytes(h: int, T: int) -> int:
    n = ctypes.c_size_t(0)
    _check(load().kvq_tree_attn_workspace_bytes(h, T, ctypes.byref(n)))
    return n.value


def kvq_tree_attn(h: int, layer: int, q, K, V, T: int, n_draft, mask, depth, opts: Optional[kvq_score_opts], out,
                  out_fp32: bool, workspace, workspace_bytes: int, stream=None):
    nd, keep = _host_i32(n_draft)
    _check(load().kvq_tree_attn(h, layer, _ptr(q), _ptr(K), _ptr(V), T, nd, _opt_ptr(mask), _opt_ptr(depth),
                                _ref(opts), _ptr(out), int(bool(out_fp32)), _ptr(workspace), workspace_bytes, _stream(stream)))


def kvq_decode_attn_scored(h: int, layer: int, q, opts: Optional[kvq_score_opts], out, out_fp32: bool, stream=None):
    _check(load().kvq_decode_attn_scored(h, layer, _ptr(q), _ref(opts), _ptr(out),
                                         int(bool(out_fp32)), _stream(stream)))


def kvq_append_selected(h: int, layer: int, K, V, n_src: int, index, n_new, n_max: int, stream=None):
    nn, keep = _host_i32(n_new)
    _check(load().kvq_append_selected(h, layer, _ptr(K), _ptr(V), n_src, _ptr(index), nn, n_max, _stream(stream)))


def kvq_read(h: int, layer: int, t0: int, n: int, K, V, stream=None):
    _check(load().kvq_read(h, layer, t0, n, _opt_ptr(K), _opt_ptr(V), _stream(stream)))


class Rope(kvq_rope_desc):
    """kvq_rope_desc from tensors: inv_freq fp32 [rot_dim / 2], weights fp32 [head_dim] or None
    (CUDA, kept alive here)."""

    def __init__(self, rot_dim, inv_freq=None, q_weight=None, k_weight=None, eps=1e-6, interleaved=False):
        for t in (inv_freq, q_weight, k_weight):
            if t is not None and (str(t.dtype) != "torch.float32" or not t.is_contiguous()):
                raise ValueError("inv_freq and weights must be contiguous float32")
        if inv_freq is not None and inv_freq.numel() < rot_dim // 2:
            raise ValueError("inv_freq has fewer than rot_dim / 2 entries")
        super().__init__(rot_dim, int(bool(interleaved)), _opt_ptr(inv_freq), _opt_ptr(q_weight), _opt_ptr(k_weight),
                         eps)
        self.tensors = (inv_freq, q_weight, k_weight)
        devices = {t.device for t in self.tensors if t is not None}
        if len(devices) > 1:
            raise ValueError("inv_freq and weights are on different devices")
        self.device = devices.pop() if devices else None   # (norm_rope compares it with the cache's)
        sizes = {t.numel() for t in (q_weight, k_weight) if t is not None}
        if len(sizes) > 1:
            raise ValueError("q_weight and k_weight differ in length")
        self.head_dim = sizes.pop() if sizes else None
        self.ref = ctypes.byref(self)


class ScoreOpts(kvq_score_opts):
    """kvq_score_opts; alibi: fp32 CUDA tensor [n_q_heads] or None (kept alive here)."""

    def __init__(self, softcap=0.0, alibi=None, window=0, scale=0.0):
        if alibi is not None and (str(alibi.dtype) != "torch.float32" or not alibi.is_contiguous()):
            raise ValueError("alibi must be contiguous float32")
        super().__init__(softcap, _opt_ptr(alibi), window, scale)
        self.alibi_tensor = alibi
        self.ref = ctypes.byref(self)


# ------------------------------------------------------------------ convenience owner
def make_paged_desc(num_layers: int, batch: int, n_kv_heads: int, n_q_heads: int, head_dim: int, max_ctx: int,
                    avg_bits: float):
    return kvq_plan_desc(num_layers, batch, n_kv_heads, n_q_heads, head_dim, 32, max_ctx, None, 1, 16, avg_bits, 0)


def make_desc(num_layers: int, batch: int, n_kv_heads: int, n_q_heads: int, head_dim: int, max_ctx: int,
              layer_bits: Sequence[Tuple[int, int]], kmodes: Optional[Sequence[int]] = None, pool_blocks: int = 0):
    cfgs = (kvq_layer_cfg * num_layers)()
    for i, (bk, bv) in enumerate(layer_bits):
        cfgs[i] = kvq_layer_cfg(bk, bv, KVQ_PER_CHANNEL if kmodes is None else kmodes[i], KVQ_PER_TOKEN)
    d = kvq_plan_desc(num_layers, batch, n_kv_heads, n_q_heads, head_dim, 32, max_ctx, cfgs, 0, 16, 0.0, pool_blocks)
    d._cfgs = cfgs   # keep the array alive with the descriptor
    return d


class Cache:
    """A plan plus a torch-allocated workspace on the current CUDA device.  Pass
    avg_bits (and no layer_bits) for a paged INT2/INT4 plan."""

    def __init__(self, num_layers, batch, n_kv_heads, n_q_heads, head_dim, max_ctx, layer_bits=None,
                 kmodes=None, device="cuda", avg_bits=None, pool_blocks=0):
        import torch
        if avg_bits is not None:
            self.desc = make_paged_desc(num_layers, batch, n_kv_heads, n_q_heads, head_dim, max_ctx, avg_bits)
        else:
            self.desc = make_desc(num_layers, batch, n_kv_heads, n_q_heads, head_dim, max_ctx, layer_bits, kmodes,
                                  pool_blocks)
        self.h = kvq_plan(self.desc)
        self._destroy = load().kvq_destroy   # held so that teardown at interpreter exit still works
        self.nbytes = kvq_workspace_bytes(self.h)
        self.ws = torch.empty(self.nbytes + 256, dtype=torch.uint8, device=device)
        base = self.ws.data_ptr()
        self.ws_ptr = (base + 255) // 256 * 256
        kvq_bind(self.h, self.ws_ptr, self.nbytes)
        self.B, self.Hkv, self.Hq, self.D = batch, n_kv_heads, n_q_heads, head_dim
        self._dev, self._bf16, self._f32, self._i32 = self.ws.device, torch.bfloat16, torch.float32, torch.int32

    def append(self, layer, K, V, stream=None):
        assert K.is_contiguous() and V.is_contiguous() and K.shape == V.shape
        kvq_append(self.h, layer, K, V, K.shape[2], stream)

    def append_tagged(self, layer, K, V, tags, stream=None):
        """tags: uint8 torch tensor [B, n] (2 or 4) on the device."""
        assert K.is_contiguous() and V.is_contiguous() and K.shape == V.shape
        kvq_append_tagged(self.h, layer, K, V, K.shape[2], tags.cpu().numpy(), tags, stream)

    def decode_attn(self, layer, q, out=None, out_fp32=False, stream=None):
        if out is None:
            out = self._decode_out(q, out_fp32, stream)
        kvq_decode_attn(self.h, layer, q, out, out_fp32, stream)
        return out

    def _decode_out(self, q, out_fp32, stream):
        """A fresh output of a decode step that runs on `stream`."""
        dtype = self._f32 if out_fp32 else self._bf16
        if stream is None:
            return q.new_empty((self.B, self.Hq, self.D), dtype=dtype)
        with self._on(stream):
            out = q.new_empty((self.B, self.Hq, self.D), dtype=dtype)
        self._hand_over(stream, out)
        return out

    def append_decode(self, layer, K, V, q, out=None, out_fp32=False, stream=None):
        """One decode step: append the token K, V [B, Hkv, 1, D] and attend with q."""
        assert K.is_contiguous() and V.is_contiguous() and K.shape == V.shape and K.shape[2] == 1
        if out is None:
            out = self._decode_out(q, out_fp32, stream)
        kvq_append_decode(self.h, layer, K, V, q, out, out_fp32, stream)
        return out

    def append_ragged(self, layer, K, V, n_new, stream=None):
        """K, V [B, Hkv, n_max, D] (contiguous); request b appends its first n_new[b] tokens."""
        assert K.is_contiguous() and V.is_contiguous() and K.shape == V.shape
        kvq_append_ragged(self.h, layer, K, V, n_new, stream)

    def seq_lens(self, layer):
        return kvq_seq_lens(self.h, layer, self.B)

    # -------- steps of several tokens, score shapes, reading back
    # (these calls are a few microseconds of kernel time at small sizes: the checks below keep to
    # plain attribute comparisons)
    def _tensor(self, t, name, shape, dtype):
        """Check one tensor argument: shape, type, device, contiguity."""
        if t.shape != shape or t.dtype != dtype:
            raise ValueError(f"{name}: expected {dtype} {tuple(shape)}, got {t.dtype} {tuple(t.shape)}")
        if t.device != self._dev:
            raise ValueError(f"{name} is on {t.device}, the cache on {self._dev}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")

    def _on(self, stream):
        """Context of a call: the cache's device and `stream` (None: the current one) are current
        in it, so that what a call allocates belongs to the stream that the call runs on."""
        import torch
        if stream is not None and self._dev.type == "cuda":
            s = _torch_stream(stream, self._dev)
            if s.device != self._dev:
                raise ValueError(f"stream is on {s.device}, the cache on {self._dev}")
            return torch.cuda.stream(s)
        if self._dev.type != "cuda":
            raise ValueError(f"the cache is on {self._dev}: kernels need a CUDA device")
        if torch.cuda.current_device() == self._dev.index:
            return _NO_CONTEXT
        return torch.cuda.device(self._dev)

    def _hand_over(self, stream, *fresh):
        """Tensors that a call on `stream` allocated go to a caller whose current stream may be
        another: their memory is not reused before that stream's work at the time they are freed
        has run, either."""
        if stream is not None:
            import torch
            cur = torch.cuda.current_stream(self._dev)
            for t in fresh:
                t.record_stream(cur)

    def norm_rope(self, layer, qkv, rope, offset=None, q=None, K=None, V=None, stream=None):
        """qkv bf16 [B, n, (Hq + 2 Hkv) * D] (rows may be padded); rope a Rope; offset int32
        [B, n] positions behind the cached tokens, None: 0 .. n - 1.  Returns (q [B, n, Hq, D],
        K, V [B, Hkv, n, D])."""
        B, D, row = self.B, self.D, (self.Hq + 2 * self.Hkv) * self.D
        shape = qkv.shape
        if len(shape) != 3 or shape[0] != B or shape[2] != row:
            raise ValueError(f"qkv: expected [{B}, n, {row}], got {tuple(shape)}")
        bs, ts, cs = qkv.stride()
        if qkv.dtype != self._bf16 or cs != 1 or qkv.device != self._dev:
            raise ValueError("qkv must be bfloat16 on the cache's device with adjacent channels")
        n = shape[1]
        if offset is not None:
            self._tensor(offset, "offset", (B, n), self._i32)
        if rope.head_dim not in (None, D):
            raise ValueError(f"norm weights must have head_dim = {D} entries")
        if rope.device not in (None, self._dev):
            raise ValueError(f"inv_freq and weights are on {rope.device}, the cache on {self._dev}")
        sq, sk = (B, n, self.Hq, D), (B, self.Hkv, n, D)
        # a dimension of size 1 may carry any stride: give the packed one
        ts = ts if n > 1 else row
        bs = bs if B > 1 else 0
        with self._on(stream):
            if q is None:
                q = qkv.new_empty(sq)
            else:
                self._tensor(q, "q", sq, self._bf16)
            if K is None:
                K = qkv.new_empty(sk)
            else:
                self._tensor(K, "K", sk, self._bf16)
            if V is None:
                V = qkv.new_empty(sk)
            else:
                self._tensor(V, "V", sk, self._bf16)
            kvq_norm_rope(self.h, layer, qkv, bs, ts, n, offset, rope, q, K, V)
        self._hand_over(stream, q, K, V)
        return q, K, V

    def tree_workspace(self, T):
        """Workspace for tree_attn with T drafted tokens (uint8, 256-byte aligned)."""
        import torch
        return torch.empty(kvq_tree_attn_workspace_bytes(self.h, T), dtype=torch.uint8, device=self._dev)

    def _attn_out(self, out, like, shape, out_fp32):
        if out is None:
            return like.new_empty(shape, dtype=self._f32) if out_fp32 else like.new_empty(shape)
        self._tensor(out, "out", shape, self._f32 if out_fp32 else self._bf16)
        return out

    def _slopes(self, opts):
        if opts is not None and opts.alibi_tensor is not None:
            if opts.alibi_tensor.numel() != self.Hq:
                raise ValueError(f"alibi must have one slope per query head ({self.Hq})")
            if opts.alibi_tensor.device != self._dev:
                raise ValueError(f"alibi is on {opts.alibi_tensor.device}, the cache on {self._dev}")

    def tree_attn(self, layer, q, K, V, n_draft=None, mask=None, depth=None, opts=None, out=None, out_fp32=False,
                  workspace=None, stream=None):
        """T drafted tokens over the cache and one another: q [B, T, Hq, D], K, V [B, Hkv, T, D];
        n_draft host ints [B]; mask int32 [B, T, ceil(T / 32)] bits; depth int32 [B, T]; opts a
        ScoreOpts.  workspace: one that tree_workspace(T) gave; calls that may overlap (other
        streams, captured graphs) need one each.  Rows of a fresh `out` behind n_draft[b] are
        unset."""
        B, T = self.B, q.shape[1]
        sq, sk = (B, T, self.Hq, self.D), (B, self.Hkv, T, self.D)
        self._tensor(q, "q", sq, self._bf16)
        self._tensor(K, "K", sk, self._bf16)
        self._tensor(V, "V", sk, self._bf16)
        if n_draft is not None and len(n_draft) != B:
            raise ValueError(f"n_draft must have {B} entries")
        if mask is not None:
            self._tensor(mask, "mask", (B, T, (T + 31) // 32), self._i32)
        if depth is not None:
            self._tensor(depth, "depth", (B, T), self._i32)
        self._slopes(opts)
        if workspace is not None and (workspace.device != self._dev or not workspace.is_contiguous()):
            raise ValueError(f"workspace must be contiguous memory of {self._dev}")
        with self._on(stream):
            out = self._attn_out(out, q, sq, out_fp32)
            # (a workspace of the call's own is memory of the call's stream: reused in its order)
            ws = self.tree_workspace(T) if workspace is None else workspace
            kvq_tree_attn(self.h, layer, q, K, V, T, n_draft, mask, depth, opts, out, out_fp32, ws,
                          ws.numel() * ws.element_size())
        self._hand_over(stream, out)
        return out

    def decode_attn_scored(self, layer, q, opts=None, out=None, out_fp32=False, stream=None):
        """decode_attn with capped scores, distance bias or a sliding window (a ScoreOpts)."""
        shape = (self.B, self.Hq, self.D)
        self._tensor(q, "q", shape, self._bf16)
        self._slopes(opts)
        with self._on(stream):
            out = self._attn_out(out, q, shape, out_fp32)
            kvq_decode_attn_scored(self.h, layer, q, opts, out, out_fp32)
        self._hand_over(stream, out)
        return out

    def append_selected(self, layer, K, V, index, n_new=None, stream=None):
        """Append slots index[b, :n_new[b]] (int32 [B, n_max]) of K, V [B, Hkv, n_src, D]."""
        n_src, n_max = K.shape[2], index.shape[-1]
        sk = (self.B, self.Hkv, n_src, self.D)
        self._tensor(K, "K", sk, self._bf16)
        self._tensor(V, "V", sk, self._bf16)
        self._tensor(index, "index", (self.B, n_max), self._i32)
        if n_new is not None and len(n_new) != self.B:
            raise ValueError(f"n_new must have {self.B} entries")
        with self._on(stream):
            kvq_append_selected(self.h, layer, K, V, n_src, index, n_new, n_max)

    def read(self, layer, t0, n, K=None, V=None, stream=None):
        """Tokens [t0, t0 + n) as bf16 (K, V [B, Hkv, n, D]); rows behind a shorter sequence's
        last token are left as they were."""
        import torch
        sk = (self.B, self.Hkv, n, self.D)
        with self._on(stream):
            if K is None:
                K = torch.empty(sk, dtype=self._bf16, device=self._dev)
            else:
                self._tensor(K, "K", sk, self._bf16)
            if V is None:
                V = torch.empty(sk, dtype=self._bf16, device=self._dev)
            else:
                self._tensor(V, "V", sk, self._bf16)
            kvq_read(self.h, layer, t0, n, K, V)
        self._hand_over(stream, K, V)
        return K, V

    def truncate(self, layer, L):
        kvq_truncate(self.h, layer, L)

    def export_layer(self, layer):
        return kvq_export_layer(self.h, layer)

    def seq_len(self, layer):
        return kvq_seq_len(self.h, layer)

    def __del__(self):
        h = getattr(self, "h", None)
        destroy = getattr(self, "_destroy", None)
        if h and destroy is not None:
            destroy(h)
            self.h = None
