"""Shape-fused Muon optimizer step for AMD MI355X (gfx950), and the layer operators that feed it.

The computation lives in hand-written HIP kernels behind the C ABI of
``include/muon.h`` (``libmuon.so``); this package only loads that library and
marshals arguments.  Importing does not load the library; ``MuonPlan`` and the
``muon_*`` functions do, and fail loudly if it has not been built.  The layer
operators (``linear``, ``expert_linear``, ``route``, ``dispatch``, ``combine``,
``dropout``; ``ops.py``), those around a block's products (``layer_norm``, ``rms_norm``, ``gate``,
``balance_loss``; ``block.py``) and the layers in four bits (``mx_quantize``, ``mx_linear``,
``mx_expert_linear``; ``mx.py``) need torch and are loaded at their first use.
"""

from .binding import (  # noqa: F401
    EXPORTED,
    KERNEL_CLASSES,
    LIB_PATH,
    MUON_BF16,
    MUON_F32,
    MUON_MODE_BF16_MFMA,
    MUON_MODE_FP32,
    MuonError,
    MuonPlan,
    PlanInfo,
    info_dict,
    load_library,
    make_descs,
    make_opts,
    muon_default_opts,
    muon_last_error,
    muon_plan_create,
    muon_plan_describe,
    muon_plan_destroy,
    muon_plan_query,
    muon_plan_status,
    muon_plan_timings,
    muon_step,
    muon_step_noalloc,
    MUON_NOALLOC_SCRATCH_BYTES,
)

_OPS = ("linear", "expert_linear", "linear_forward", "linear_backward", "Routing", "route", "dispatch",
        "dispatch_forward", "dispatch_backward", "combine", "combine_forward", "combine_backward", "dropout",
        "dropout_forward")
_BLOCK = ("layer_norm", "rms_norm", "norm_forward", "norm_backward", "Gating", "gate", "gate_forward", "gate_backward",
          "Balance", "balance_loss", "balance_forward", "balance_backward")
_MX = ("MxWeight", "mx_quantize", "mx_dequantize", "mx_linear", "mx_expert_linear")


def __getattr__(name):
    if name in _OPS:
        from . import ops
        globals().update({n: getattr(ops, n) for n in _OPS})
        return globals()[name]
    if name in _BLOCK:
        from . import block
        globals().update({n: getattr(block, n) for n in _BLOCK})
        return globals()[name]
    if name in _MX:
        from . import mx
        globals().update({n: getattr(mx, n) for n in _MX})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
