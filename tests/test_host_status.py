"""kvq_device_status before anything was launched: the workspace holds whatever the caller's memory
held, and the status word in it is not read (the pointer below is never dereferenced)."""
import ctypes

from layer_wise_mixed_b200 import build as kbuild
from layer_wise_mixed_b200 import kvq


def test_status_before_the_first_launch():
    kbuild.build()
    L = kvq.load()
    h = kvq.kvq_plan(kvq.make_desc(1, 2, 2, 8, 64, 100, [(4, 2)]))
    try:
        fake = 1 << 40
        kvq.kvq_bind(h, fake, kvq.kvq_workspace_bytes(h))
        for call in (lambda: kvq.KVQ_OK,
                     # calls that do nothing do not launch either
                     lambda: L.kvq_append_selected(h, 0, fake, fake, 1, fake, (ctypes.c_int32 * 2)(0, 0), 1, None),
                     lambda: L.kvq_tree_attn(h, 0, fake, fake, fake, 1, (ctypes.c_int32 * 2)(0, 0), None, None, None, fake, 0,
                                             fake, kvq.kvq_tree_attn_workspace_bytes(h, 1), None)):
            assert call() == kvq.KVQ_OK
            flags = ctypes.c_uint(7)
            assert L.kvq_device_status(h, None, ctypes.byref(flags)) == kvq.KVQ_OK
            assert flags.value == 0
    finally:
        kvq.kvq_destroy(h)
