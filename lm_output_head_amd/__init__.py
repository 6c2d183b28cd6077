"""FlashHead inference for MI355X (gfx950): hand-written HIP kernels behind a
C ABI (include/flashhead.h), with this thin torch/ctypes binding on top."""

import importlib

from ._abi import (FH_BF16, FH_F32, FH_PROBE_SAMPLE, FH_PROBE_TOPK,  # noqa: F401
                   FH_QUANT_INT4_G32, FH_QUANT_INT8_G32, FH_QUANT_NONE, FH_TOKEN_ARGMAX,
                   FH_TOKEN_SAMPLE,
                   FlashHeadError)
from ._abi import load as load_library  # noqa: F401

_NAMES = {
    "flashhead": ("FlashHead", "fh_create", "fh_destroy", "fh_forward", "fh_forward_adaptive", "fh_forward_noalloc",
                  "fh_probs_fp8", "fh_score", "fh_dense_forward", "fh_get_int4", "fh_get_int8", "fh_spec_verify",
                  "fh_profile_begin", "fh_profile_end", "fh_set_path", "fh_sync_status", "fh_balanced_assign",
                  "fh_cluster", "fh_last_error", "fh_version"),
    "serve": ("LogitRules", "W8A8Head", "rmsnorm", "logits_apply", "fh_rmsnorm", "fh_w8a8_create",
              "fh_w8a8_create_codes", "fh_w8a8_destroy", "fh_w8a8_get", "fh_w8a8_workspace", "fh_w8a8_matmul",
              "fh_w8a8_forward", "fh_logits_workspace", "fh_logits_apply"),
    "fp8": ("FP8Head", "rmsnorm_fp8", "fp8_quant", "fh_rmsnorm_fp8", "fh_fp8_quant", "fh_fp8_create",
            "fh_fp8_create_codes", "fh_fp8_destroy", "fh_fp8_get", "fh_fp8_workspace", "fh_fp8_matmul",
            "fh_fp8_matmul_native", "fh_fp8_forward"),
    "beam": ("beam_select", "beam_reorder", "fh_beam_workspace", "fh_beam_select", "fh_beam_reorder",
             "fh_beam_reorder_check"),
}
_HOME = {name: module for module, names in _NAMES.items() for name in names}


def __getattr__(name):
    # the torch-facing binding is imported lazily so that the ABI module and
    # the build script stay usable without initialising torch; once imported, a
    # module is the package's attribute, and its names are looked up in it at each use
    home = _HOME.get(name)
    if home is None:
        raise AttributeError(name)
    module = globals().get(home)
    return getattr(importlib.import_module("." + home, __name__) if module is None else module, name)
