"""ctypes view of libspecverify.so: one Python prototype per C entry point."""
from __future__ import annotations

import ctypes
import os

LIB = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libspecverify.so")

_P = ctypes.c_void_p
_I = ctypes.c_int
_SZ = ctypes.c_size_t
_F = ctypes.c_float
_S = ctypes.c_int64   # strides

# name -> (restype, argtypes), mirroring include/spec_verify.h
PROTOTYPES = {
    "spec_strerror": (ctypes.c_char_p, [_I]),
    "spec_set_wait_bound": (_I, [_I]),
    "spec_verify_greedy_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "spec_verify_greedy": (_I, [_P, _I, _I, _I, _I, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P,
                                _P, _SZ, _P]),
    "spec_verify_greedy_noalloc": (_I, [_P, _I, _I, _I, _I, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P, _P]),
    "spec_verify_sample_workspace_bytes": (_SZ, [_I, _I, _I]),
    "spec_verify_sample": (_I, [_P, _P, _P, _P, _I, _I, _I, ctypes.c_int32, _P, _P, _P, _P, _P,
                                _P, _P, _P, _SZ, _P]),
    "spec_process_workspace_bytes": (_SZ, [_I, _I]),
    "spec_process_logits": (_I, [_P, _I, _I, _I, _F, _I, _F, _P, _P, _P, _P, _P, _SZ, _P]),
    "spec_verify_sample_logits_workspace_bytes": (_SZ, [_I, _I, _I]),
    "spec_verify_sample_logits": (_I, [_P, _P, _I, _I, _I, _I, _F, _I, _F, _P, _P, ctypes.c_int32,
                                       _P, _P, _P, _P, _P, _P, _P, _P, _SZ, _P]),
    "spec_commit_realign_kv": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                    _P, _P, _P]),
    "spec_repad_kv": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "spec_unpad_kv": (_I, [_P, _P, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "spec_resync_draft_kv": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P,
                                  _P, _P, _P]),
    "spec_commit_paged": (_I, [_I, _I, _I, _I, _P, _P, _P, _P, _P, _P, _P, _P, _P]),
    "spec_verify_tree_workspace_bytes": (_SZ, [_I, _I, _I, _I]),
    "spec_verify_tree": (_I, [_P, _I, _I, _I, _I, _P, _P, _P, ctypes.c_int32, _P, _P, _P, _P, _P, _P,
                              _P, _P, _SZ, _P]),
    "spec_compact_tree_kv": (_I, [_P, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P, _P]),
    "spec_verify_tree_sample_workspace_bytes": (_SZ, [_I, _I, _I]),
    "spec_verify_tree_sample": (_I, [_P, _P, _P, _P, _P, _P, _I, _I, _I, ctypes.c_int32, _P, _P, _P, _P,
                                     _P, _P, _P, _P, _P, _SZ, _P]),
    "spec_tree_mask": (_I, [_I, _I, _P, _P, _P, _P, _P, _P, _P]),
    "spec_norm_rope_kv": (_I, [_P, _S, _P, _S, _P, _S, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _P,
                               _P, _P, _F, _P, _I, _I, _P, _P, _P]),
    "spec_norm_rope_kv_paged": (_I, [_P, _S, _P, _S, _P, _S, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I,
                                     _P, _P, _P, _P, _P, _F, _P, _I, _I, _P, _P, _P]),
    "spec_prompt_attention": (_I, [_P, _S, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _F, _P, _P, _P, _P]),
    "spec_prompt_attention_paged": (_I, [_P, _S, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I, _P, _P, _F, _P,
                                         _P, _P, _P]),
    "spec_tree_attention_workspace_bytes": (_SZ, [_I, _I, _I, _I, _I, _I, _I]),
    "spec_tree_attention": (_I, [_P, _S, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _P, _P, _F, _P, _P, _P, _P, _SZ,
                                 _P]),
    "spec_tree_attention_paged": (_I, [_P, _S, _P, _I, _I, _I, _I, _I, _I, _I, _I, _I, _I, _P, _I, _P, _P, _F, _P,
                                       _P, _P, _P, _SZ, _P]),
    "spec_group_same_length": (_I, [_P, _I, _I, _I, _P, _P, _P, _P, _P, _P]),
}

_lib = None


def load() -> ctypes.CDLL:
    """Load the built HIP library; raise if it is missing (there is no fallback).

    torch is imported first: the library must bind to the same HIP runtime as
    the framework whose device memory and streams it is handed.  torch ships
    its own libamdhip64 (same SONAME as the system one); loading ours first
    would map the system runtime and leave torch on a second one.
    """
    global _lib
    if _lib is not None:
        return _lib
    import torch  # noqa: F401  (maps torch's HIP runtime before ours resolves against it)
    if not os.path.exists(LIB):
        raise RuntimeError(
            f"{LIB} is not built; run `python -m speculative_decoding_verification_04_amd.build` "
            "(the verify-and-commit step has no non-HIP implementation)")
    lib = ctypes.CDLL(LIB)
    for name, (res, args) in PROTOTYPES.items():
        fn = getattr(lib, name)
        fn.restype = res
        fn.argtypes = args
    _lib = lib
    return lib
