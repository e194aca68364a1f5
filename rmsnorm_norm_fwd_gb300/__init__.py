"""Fused row-wise RMSNorm / LayerNorm, forward and backward, for GB300 (sm_103a).

The kernels live in libgbnorm.so behind the C ABI of ``include/gbnorm.h``;
``binding`` marshals torch tensors onto it.  The binding is imported on first
use of one of its names, so that ``rmsnorm_norm_fwd_gb300.inputs`` and
``rmsnorm_norm_fwd_gb300.build`` work before the library exists; any use of
the ops without the built library raises ImportError.
"""

_OPS = ("rmsnorm_fwd", "layernorm_fwd", "rmsnorm_bwd", "layernorm_bwd", "norm_bwd_workspace_size",
        "norm_fwd_ex", "norm_bwd_ex", "norm_bwd_ex_workspace_size",
        "variant_name", "force_variant", "variants", "ex_variants", "ex_force_variant", "ex_last_variant",
        "read_fault", "set_grid_limit", "GbnormError", "lib")

# Norms with 8-bit rows: 8-bit output, 8-bit checkpoint, the backward from it,
# reading back.
_Q8_OPS = ("norm_fwd_q8", "norm_fwd_ck8", "norm_bwd_ck8", "norm_bwd_ck8_workspace_size", "read_q8", "read_ck8",
           "Checkpoint8", "checkpoint8_empty", "q8_last_variant")

__all__ = list(_OPS) + list(_Q8_OPS)


def __getattr__(name):
    if name in _OPS:
        from . import binding
        return getattr(binding, name)
    if name in _Q8_OPS:
        from . import q8
        globals()[name] = f = getattr(q8, name)  # later uses find it without this call
        return f
    raise AttributeError(name)
