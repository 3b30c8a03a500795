"""Tensor-parallel sharded GEMMs on GB300 (sm_103a).

The compute lives in the CUDA library ``libtps.so`` built from ``csrc/``;
this package only marshals torch tensors into its C ABI (``include/tps.h``).
Importing the package does not load the library; the first call does, and
fails loudly if it is missing.
"""
__all__ = ["plan_shards", "matmul_fwd_bwd", "mlp_fwd_bwd", "vocab_ce_fwd_bwd", "linear_ce_fwd", "linear_ce_bwd",
           "rope_plan", "rope_fwd", "rope_bwd", "grad_norm", "adamw_plan", "adamw_step", "inputs"]


def __getattr__(name):
    if name in ("plan_shards", "matmul_fwd_bwd", "mlp_fwd_bwd", "vocab_ce_fwd_bwd",
                "mlp_workspace_bytes", "ce_workspace_bytes", "last_device_error", "library",
                "profile", "TpsError", "linear_ce_fwd", "linear_ce_bwd", "linear_ce_workspace_bytes", "rope_plan",
                "rope_fwd", "rope_bwd", "grad_norm", "adamw_plan", "adamw_step", "adamw_scalars"):
        from . import api
        return getattr(api, name)
    raise AttributeError(name)
