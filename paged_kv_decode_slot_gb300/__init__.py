"""paged_kv_decode_slot_gb300 -- libpagedkv: decode-step attention over a paged KV cache on GB300.

The compute path is the C-ABI library ``libpagedkv.so`` (hand-written sm_103a CUDA, declared
in ``include/pkv.h``); ``binding`` exposes its entry points under the same names with torch
tensors as arguments (PyTorch supplies device memory and streams only).  ``inputs`` draws
seeded synthetic workloads; ``step`` runs a whole decode step.

The binding is loaded on first use of one of its names, so that ``build`` can be imported
before the library exists; using any entry point without the built library raises
ImportError (there is no fallback path).
"""


import types

_OTHERS = ("BLOCK_SIZE", "CacheDesc", "PkvError", "cache_desc", "check", "library", "max_partitions_for",
           "tapered_partitions_for", "IN_KERNEL_MERGE_WEIGHTS", "split_attention_launches", "multi_attention_launches")


class _Binding(types.ModuleType):
    """The binding, once it is loaded: a name that is replaced in it is replaced here too."""

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        if name in globals() and _of_the_binding(name):
            globals()[name] = value


def _of_the_binding(name):
    return name.startswith(("pkv_", "PKV_")) or name in _OTHERS


def __getattr__(name):
    if _of_the_binding(name):
        from . import binding
        binding.__class__ = _Binding
        globals()[name] = value = getattr(binding, name)  # found without this function from now on
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
