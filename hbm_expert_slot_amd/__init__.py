"""hbm_expert_slot_amd: the expert-slot MoE decode step for MI355X (gfx950).

libslotcache.so (HIP, built in-tree by hbm_expert_slot_amd.build) does all of
the work; `binding` is its ctypes binding, `SlotCache` binds torch device
buffers to a handle, and `ops` has the operators on 4-bit weights (quantising,
products and the whole mixture-of-experts layer, `ops.MoELayer`) and attention:
over prompts (`ops.prompt_attention`) and over a key/value cache in 4 bits, with
its writing and eviction (`ops.KV4Cache`).
"""
from . import binding
from .binding import SlotCacheError

__all__ = ["binding", "ops", "SlotCacheError", "SlotCache"]


def __getattr__(name):
    if name == "SlotCache":
        from .cache import SlotCache
        return SlotCache
    if name == "ops":
        import importlib
        return importlib.import_module(".ops", __name__)
    raise AttributeError(name)
