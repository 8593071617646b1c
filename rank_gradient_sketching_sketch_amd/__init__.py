"""LoGRA sketch-accumulate + RowAdam-apply on MI355X (gfx950).

The compute path is the C-ABI library ``liblogra.so`` (HIP kernels); the
functions here are a thin ctypes binding over it. Importing the package does
not load the library; the first call does, and fails loudly if it is not
built.
"""
from __future__ import annotations

import types

__all__ = [
    "logra_abi_version", "logra_status_string", "logra_sign_words",
    "logra_sketch_workspace_bytes", "logra_sketch_accumulate",
    "logra_sketch_project", "logra_sketch_fold", "LaunchOpts",
    "logra_backward_dx", "logra_backward_dx_sketch",
    "logra_sqnorm_workspace_bytes", "logra_update_sqnorm", "logra_rowadam_apply",
    "logra_sqnorm_prepare", "logra_update_sqnorm_prepared", "logra_update_sqnorm_noalloc",
    "logra_sqnorm_batch_workspace_bytes", "logra_update_sqnorm_batch",
    "logra_kl_budget_at", "logra_kl_step_scale", "KLBudget",
    "GradList", "logra_grad_workspace_bytes", "logra_grad_norm", "logra_grad_clip",
    "logra_expert_sort_workspace_bytes", "logra_expert_sort", "logra_expert_gather",
    "logra_expert_combine", "logra_expert_combine_backward",
    "logra_sketch_experts_workspace_bytes", "logra_sketch_experts",
    "logra_route", "logra_route_backward", "logra_fp8_quantize", "logra_fp8_matmul", "AdamWList", "logra_adamw",
    "LOGRA_SOFTMAX", "LOGRA_SIGMOID",
    "LograError", "MatrixDesc", "library_path", "load_library",
]


_kept = {}                      # names that were looked up, as the binding has them


class _Binding(types.ModuleType):
    """The binding's module: what is replaced in it shows through the package."""

    def __setattr__(self, name, value):
        super().__setattr__(name, value)
        _forget()

    def __delattr__(self, name):
        super().__delattr__(name)
        _forget()


def _forget():
    while _kept:
        name, value = _kept.popitem()
        if globals().get(name) is value:        # not one that a caller has put here
            del globals()[name]


def __getattr__(name):
    if name in __all__:
        from . import binding
        binding.__class__ = _Binding
        globals()[name] = _kept[name] = value = getattr(binding, name)     # later look-ups do not come here
        return value
    raise AttributeError(name)
