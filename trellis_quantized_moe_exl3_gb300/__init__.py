"""GB300-native (sm_103a) EXL3 trellis-quantized routed-expert MoE layer.

The compute path is the CUDA library built from ``csrc/`` (C ABI in
``include/exl3.h``); this package only binds it.  ``synth`` holds the seeded
synthetic workloads.
"""
from . import synth  # noqa: F401


def _api():
    from . import api
    return api


_ATTENTION = ("PagedKVCache", "PagedBatch", "qk_norm_rope", "kv_append", "paged_attention")
_SPECULATE = ("PagePool", "PagedStep", "verify_drafts")


def __getattr__(name):
    if name == "DecoderBlock":
        from .block import DecoderBlock
        return DecoderBlock
    if name in _ATTENTION:
        from . import attention
        value = globals()[name] = getattr(attention, name)  # found directly from now on
        return value
    if name in _SPECULATE:
        from . import speculate
        value = globals()[name] = getattr(speculate, name)
        return value
    if name in ("Layer", "route", "rmsnorm", "device_status"):
        return getattr(_api(), name)
    raise AttributeError(name)
