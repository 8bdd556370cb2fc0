"""Hybrid Muon + AdamW optimizer step for MI355X (gfx950).

The compute runs in libmuonadamw.so (hand-written HIP kernels behind the C ABI of
include/muon_adamw.h); this package is its thin Python binding plus the MuonAdamW
parameter-group wrapper and the training operators around the AdamW parameters (ops).
PyTorch supplies device memory and streams only.
"""
import importlib.util

from ._lib import (LIB_PATH, MFMA_PROBE_OPERAND_VALUES, MFMA_PROBE_THREADS, MuonAdamWError, Route, abi_version, adamw_step, adamw_step_multi, load,
                   mfma_probe, mfma_probe_flops, muon_check_plan, muon_ns_time, muon_phases, muon_route_of, muon_step,
                   muon_static_init, muon_step_static, muon_tune, muon_tune_configs,
                   muon_tune_reset,
                   muon_workspace_bytes, newton_schulz, newton_schulz_workspace_bytes,
                   stream_probe)
from .optim import MuonAdamW

__all__ = ["LIB_PATH", "MFMA_PROBE_OPERAND_VALUES", "MFMA_PROBE_THREADS", "MuonAdamWError", "Route", "abi_version", "adamw_step", "adamw_step_multi",
           "load", "mfma_probe", "mfma_probe_flops", "muon_check_plan", "muon_ns_time", "muon_phases", "muon_route_of",
           "muon_static_init", "muon_step", "muon_step_static", "muon_tune", "muon_tune_configs", "muon_tune_reset",
           "muon_workspace_bytes", "newton_schulz", "newton_schulz_workspace_bytes",
           "stream_probe", "MuonAdamW"]

# The training operators are torch.autograd functions, so their module needs torch; it is
# imported with the first of these names that is used.
_OPS = ("ADAMW_BYTE_BLOCK", "adamw_byte_state", "adamw_byte_step_multi", "adamw_byte_values",
        "adamw_step_embedding", "distill_backward", "distill_forward", "distill_loss",
        "distill_loss_grad", "embedding", "embedding_backward", "embedding_forward",
        "embedding_workspace_bytes", "head_loss", "head_loss_backward", "head_loss_forward",
        "head_loss_grad", "head_loss_workspace_bytes", "layer_norm", "layer_norm_backward",
        "layer_norm_forward", "layer_norm_workspace_bytes", "residual_norm",
        "residual_norm_backward", "residual_norm_forward", "residual_norm_workspace_bytes")
if importlib.util.find_spec("torch") is not None:  # else `import *` has the rest
    __all__ += _OPS


def __getattr__(name):
    if name not in _OPS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import ops

    globals().update((n, getattr(ops, n)) for n in _OPS)
    return globals()[name]
