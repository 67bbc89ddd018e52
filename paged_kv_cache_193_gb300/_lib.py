"""ctypes declarations of the C ABI in ``include/pa.h``.

Loading fails loudly (``ImportError``) when ``libpa.so`` has not been built:
there is no fallback implementation.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_build", "libpa.so")

PA_OK = 0
PA_ERR_INVALID_ARG = 1
PA_ERR_UNSUPPORTED = 2
PA_ERR_WORKSPACE = 3
PA_ERR_CUDA = 4

PA_KV_BF16 = 0
PA_KV_FP8_E4M3 = 1

PA_STATIC_WORKSPACE_BYTES = 32 << 20

PA_DEVERR_BAD_BLOCK = 0x1
PA_DEVERR_BAD_CONTEXT = 0x2
PA_DEVERR_TIMEOUT = 0x4
PA_DEVERR_BAD_SLOT = 0x8
PA_DEVERR_OUT_OF_BLOCKS = 0x10
PA_DEVERR_BAD_AXIS = 0x20

# name -> (restype, argtypes); the order matches include/pa.h
_P, _I, _F, _SZ = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
_L = ctypes.c_int64
SIGNATURES = {
    "pa_slot_mapping": (_I, [_P, _I, _P, _I, _I, _P, _P]),
    "pa_cache_append": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _F, _P]),
    "pa_decode_max_partitions": (_I, [_I, _I, _I]),
    "pa_decode_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I]),
    "pa_decode_partitions": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I,
                                  _P, _SZ, _P]),
    "pa_decode_reduce": (_I, [_P, _SZ, _P, _I, _I, _I, _I, _I, _I, _P, _P]),
    "pa_decode": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F, _F, _I, _P, _SZ,
                       _P, _P]),
    "pa_decode_step": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F, _F,
                            _I, _P, _SZ, _P, _P, _P]),
    "pa_cache_append_scaled": (_I, [_P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _P, _P, _P]),
    "pa_decode_step_scaled": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P,
                                   _P, _F, _I, _P, _SZ, _P, _P, _P]),
    "pa_decode_step_fp8_qk": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _P,
                                   _P, _F, _F, _I, _P, _SZ, _P, _P, _P]),
    "pa_block_alloc": (_I, [_P, _I, _P, _I, _I, _I, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P, _P]),
    "pa_block_alloc_chunk": (_I, [_P, _I, _P, _P, _I, _I, _P, _P, _P, _I, _P, _P, _I, _I, _I, _P, _P]),
    "pa_chunk_slot_mapping": (_I, [_P, _I, _P, _P, _I, _I, _P, _P]),
    "pa_prefill": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F, _P,
                        _P]),
    "pa_prefill_scaled": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _F, _P,
                               _P]),
    "pa_prefill_mma": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _F,
                            _P, _P]),
    "pa_rope_append": (_I, [_P, _L, _P, _L, _P, _L, _P, _I, _P, _P, _I, _I, _F, _P, _I, _I, _P, _P, _P, _I,
                            _I, _I, _I, _I, _F, _P, _P, _P]),
    "pa_block_summary": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "pa_sparse_select": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P]),
    "pa_sparse_decode": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _F, _P, _P,
                              _I, _I, _P, _P]),
    "pa_sparse_attend": (_I, [_P, _P, _P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _F,
                              _I, _I, _I, _P, _P, _P, _P]),
    "pa_norm_rope_append": (_I, [_P, _L, _P, _L, _P, _L, _P, _L, _P, _L, _F, _F, _P, _I, _P, _P, _I, _I, _F, _P, _I,
                                 _I, _P, _P, _P, _I, _I, _I, _I, _I, _F, _P, _P, _P]),
    "pa_shared_prefix_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "pa_shared_prefix_launches": (_I, [_I, _I, _I, _I, _I, _I, _I, _I, _I]),
    "pa_shared_prefix_decode": (_I, [_P, _P, _P, _P, _I, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P,
                                     _P, _F, _P, _SZ, _P, _P]),
    "pa_cross_workspace_size": (_SZ, [_I, _I, _I, _I, _I, _I, _I, _I]),
    "pa_cross_attention": (_I, [_P, _P, _P, _P, _I, _P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _F, _P, _P, _F,
                                _P, _SZ, _P, _P]),
    "pa_decode_static_workspace": (_I, [_P, _P, _P, _P, _I, _P, _I, _I, _I, _I, _I, _I, _I, _F,
                                        _F, _I, _P, _P]),
    "pa_test_set_share": (_I, [_L, _I]),
    "pa_test_set_wait": (_I, [ctypes.c_uint64, _I]),
    "pa_device_errors": (_I, [ctypes.POINTER(ctypes.c_uint), _I]),
    "pa_status_string": (ctypes.c_char_p, [_I]),
    "pa_last_error": (ctypes.c_char_p, []),
}

BINDING_PATH = os.path.join(HERE, "_build", "_pa_binding.so")
# the calls of the CPython binding, in the order its bind() takes their addresses
BINDING_CALLS = ("pa_rope_append", "pa_block_summary", "pa_sparse_select", "pa_sparse_decode", "pa_sparse_attend",
                 "pa_norm_rope_append", "pa_shared_prefix_decode", "pa_cross_attention")

_lib = None
_binding = None


def binding():
    """The CPython binding, calling into the library that load() gives.  Like
    load(), raises ImportError when it has not been built, or was built for
    another torch or Python than this one's."""
    global _binding
    if _binding is None:
        if not os.path.exists(BINDING_PATH):
            raise ImportError(
                f"{BINDING_PATH} not found: build the CUDA library first "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        import torch  # the module links against its libraries

        from .build import binding_for, built_for
        has, needs = built_for(BINDING_PATH), binding_for(torch)
        if has != needs:
            raise ImportError(
                f"{BINDING_PATH} was built for {has}, this is {needs}: build it again "
                "(python -c 'import __graft_entry__ as g; g.build()')")
        loader = importlib.machinery.ExtensionFileLoader("_pa_binding", BINDING_PATH)
        spec = importlib.util.spec_from_file_location("_pa_binding", BINDING_PATH, loader=loader)
        module = importlib.util.module_from_spec(spec)
        loader.exec_module(module)
        lib = load()
        module.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in BINDING_CALLS))
        _binding = module
    return _binding


def load(path: str | None = None) -> ctypes.CDLL:
    """Load libpa.so (``PA_LIBRARY`` in the environment selects another build
    of the same library, e.g. a launch-shape variant)."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or os.environ.get("PA_LIBRARY") or LIB_PATH
    if not os.path.exists(p):
        raise ImportError(
            f"{p} not found: build the CUDA library first "
            "(python -c 'import __graft_entry__ as g; g.build()')")
    lib = ctypes.CDLL(p)
    for name, (res, args) in SIGNATURES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    if path is None:
        _lib = lib
    return lib
