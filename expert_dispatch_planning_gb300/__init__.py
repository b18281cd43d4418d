"""GB300 (sm_103a) Mixture-of-Experts routing and dispatch planning.

Four steps, each one C-ABI call into ``libmoe_dispatch.so``:
``route_topk`` -> ``plan`` -> ``permute`` -> (experts) -> ``combine``
(``route_plan`` does the first two in one call, one launch where it can).
Around the experts: ``residual_norm`` before the router, ``expert_ffn`` between
permute and combine, and the gradients ``combine_backward``,
``expert_ffn_backward`` and ``residual_norm_backward``.  Between two blocks:
``block_norm`` and ``block_norm_backward``.  For up to 64 tokens ``layer`` does
everything from the router's logits to the weighted sum.
"""
from ._lib import MOE_LAYER_MAX_TOKENS as LAYER_MAX_TOKENS  # noqa: F401
from ._lib import MoeError, load  # noqa: F401
from .api import (BalancedPlan, BlockNormOut, NormOut, Plan, block_norm, block_norm_backward, combine,  # noqa: F401
                  combine_backward, expert_ffn, expert_ffn_backward, layer, residual_norm, residual_norm_backward)
from .api import (get_status, permute, plan, plan_balanced,  # noqa: F401
                  plan_launches, rank_layout, rank_layout_workspace, route_plan, route_plan_launches, route_topk, set_plan_fault, tile_map)

__all__ = ["BalancedPlan", "BlockNormOut", "LAYER_MAX_TOKENS", "MoeError", "NormOut", "Plan", "block_norm", "block_norm_backward", "layer",
           "plan_balanced", "combine", "combine_backward", "expert_ffn",
           "expert_ffn_backward", "residual_norm", "residual_norm_backward", "get_status", "load", "permute", "plan", "plan_launches",
           "rank_layout", "rank_layout_workspace", "route_plan", "route_plan_launches", "route_topk", "set_plan_fault", "tile_map"]
