"""TIDE layout-aware FSDP2 collectives, single-GPU hot path for GB300 (sm_103a).

``tide_rs_reduce`` and ``tide_ag_place`` run in hand-written CUDA kernels in
``libtide.so`` (C ABI: include/tide.h); this package only binds them.  So do the
training block's operators that run between the two (include/tide_ops.h): RMS
norm, linear layer, 8-bit activation checkpoints.
"""

from .tide import (  # noqa: F401
    LIB_PATH, PointerArray, TideError, TidePlan, pointer_array,
    tide_plan_create, tide_plan_destroy, tide_plan_items, tide_plan_level2_order, tide_plan_param_geometry,
    tide_plan_shard_elems, tide_plan_set_option, tide_plan_check, tide_plan_inbox_elems,
    tide_rs_reduce, tide_rs_reduce_noalloc, tide_rs_staged, tide_rs_reduce_slots, tide_slot_pack,
    tide_ag_place, tide_rd_rounds, tide_rd_send_count, tide_ag_rd_exchange, tide_ag_stage_place,
    tide_ag_stage_init, tide_ag_rd_exchange_rails, stage_shard_pointers,
    tide_debug_bounds_violations, tide_debug_bounds_selftest,
    TIDE_OPT_RS_KERNEL, TIDE_OPT_WAIT_LIMIT_NS, TIDE_OPT_TEST_DROP_TILE, TIDE_OPT_RS_AVERAGE,
    TIDE_OPT_RS_ACCUMULATE, TIDE_OPT_AG_UNPADDED, TIDE_OPT_SUM_ORDER, TIDE_OPT_CHECK_OVERLAP,
    TIDE_OPT_RD_EXCHANGE, TIDE_OPT_AG_TRANSPORT,
    TIDE_SUM_LANDING, TIDE_SUM_RELATIVE, TIDE_AG_SM, TIDE_AG_COPY_ENGINES, TIDE_AG_BULK,
)

# The operators take torch tensors; the collectives do not need torch, so it is
# imported when the first operator is asked for.
_OPS = frozenset((
    "Checkpoint8", "TIDE_CKPT_BLOCK", "tide_checkpoint_store", "tide_checkpoint_load", "tide_rms_norm",
    "tide_rms_norm_backward", "tide_linear", "tide_linear_grad_input", "tide_linear_grad_weight",
    "tide_ops_check", "tide_ops_set_option", "TIDE_OPS_OPT_WAIT_LIMIT_NS", "TIDE_OPS_OPT_TEST_DROP_LOAD",
    "TIDE_ACT_NONE", "TIDE_ACT_RELU", "TIDE_ACT_GELU", "TIDE_ACT_GELU_ERF", "TIDE_ACT_SILU",
))


def __getattr__(name):
    if name not in _OPS:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import ops
    globals().update({n: getattr(ops, n) for n in _OPS})
    return globals()[name]


def __dir__():
    return sorted(set(globals()) | _OPS)
