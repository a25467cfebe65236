"""MoE token routing, dispatch and combine for one MI355X (gfx950).

The path runs in hand-written HIP kernels behind the C ABI of
``include/moe_route.h`` (libmoeroute.so, built by
``python -m combine_moe_route_amd.build``). This package is its thin ctypes
binding; torch provides device memory and the current stream only.

The binding is imported on first use of any API name, so building the
library never needs an existing one; using the API without the library
raises ImportError.
"""
import types

_API = (
    "DispatchBuffers",
    "MoeRouteError",
    "alloc_dispatch",
    "alloc_dispatch_quantized",
    "moe_combine",
    "moe_combine_recv",
    "moe_combine_send",
    "moe_dispatch",
    "moe_dispatch_max_rows",
    "moe_dispatch_no_alloc",
    "moe_dispatch_quantized",
    "moe_dispatch_workspace_bytes",
    "moe_gated_act_quant_fp8",
    "moe_gated_act_quant_int8",
    "moe_grouped_gemm_bf16",
    "moe_grouped_gemm_fp8",
    "moe_grouped_gemm_int8",
    "moe_grouped_gemm_workspace_bytes",
    "moe_harness_expert_scale",
    "moe_rmsnorm_quant",
    "moe_route_dispatch",
    "moe_route_replicas",
    "moe_route_scored",
    "moe_route_topk",
    "moe_route_topk_shared",
    "status_string",
)

__all__ = list(_API)


def _forget(names, held):
    """Drop the names that still stand here as `held`, the binding's namespace, has them."""
    for name in names:
        if name in _API and name in held and globals().get(name) is held[name]:
            del globals()[name]


class _Binding(types.ModuleType):
    """The binding's class: a name that is replaced there is looked up again here."""

    def __setattr__(self, name, value):
        _forget((name,), vars(self))
        super().__setattr__(name, value)

    def __delattr__(self, name):
        _forget((name,), vars(self))
        super().__delattr__(name)


def __getattr__(name):
    if name in _API:
        from . import binding
        # found directly from now on: coming here costs 0.5 us a call
        value = globals()[name] = getattr(binding, name)
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
