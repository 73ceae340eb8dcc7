"""Training the routed experts: one forward and one backward pass out of the
C ABI's calls, beside mm_route_logits and its gradient for the router.

    ids, w, counts, sums, loss = mm_route_logits(logits, k, True, token_mask=mask)
    out, saved = moe_experts_train(hidden, ids, w, w_gate_up, w_down, token_mask=mask)
    grads = moe_experts_train_backward(d_out, saved, w_gate_up, w_down)
    d_logits = mm_route_logits_backward(logits, ids, counts, True, grads.d_topk_w, d_loss,
                                        token_mask=mask)

What is kept between the two passes, next to the inputs: the slots' places and
the pre-activations in 8 bits (2 I bytes a slot and 1/32 of that in scales). The
activations are computed again from those, the token rows copied again.
"""
from __future__ import annotations

from typing import NamedTuple, Optional

import torch

from . import _lib


class ExpertsSaved(NamedTuple):
    """What moe_experts_train keeps for its backward pass."""
    hidden: torch.Tensor    # [T, H], the caller's
    places: torch.Tensor    # [T, k] int32
    offsets: torch.Tensor   # [E + 1] int32
    row_w: torch.Tensor     # [T k] fp32, the rows' routing weights
    codes: torch.Tensor     # [T k, 2I] int8
    scales: torch.Tensor    # [T k, 2I / 32] uint8


class ExpertsGrads(NamedTuple):
    d_hidden: torch.Tensor     # [T, H]
    d_topk_w: torch.Tensor     # [T, k] fp32
    d_w_gate_up: torch.Tensor  # [E, 2I, H]
    d_w_down: torch.Tensor     # [E, H, I]


def moe_experts_train(hidden, topk_ids, topk_w, w_gate_up, w_down, token_mask=None, stream=None):
    """out [T, H] = sum_j topk_w[t, j] W_down[e_j] (silu(g) * u), (g, u) = W_gate_up[e_j]
    hidden[t], and what the backward pass needs. hidden [T, H], w_gate_up [E, 2I, H]
    (gate rows first), w_down [E, H, I], all bfloat16 or float16; topk_ids [T, k] int32,
    topk_w [T, k] fp32. Tokens that token_mask [T] drops enter nothing: their out and
    gradients are zeros, whatever their hidden rows hold. Rows, pre-activations and
    expert outputs are rounded to the type; sums are fp32."""
    E = w_down.shape[0]
    places, offsets = _lib.mm_group_slots(topk_ids, E, token_mask=token_mask, stream=stream)
    rows, row_w = _lib.mm_dispatch_rows(hidden, places, w=topk_w, stream=stream)
    z = _lib.mm_grouped_product(rows, w_gate_up, offsets, stream=stream)
    act, codes, scales = _lib.mm_swiglu_pack(z, offsets=offsets, stream=stream)
    y = _lib.mm_grouped_product(act, w_down, offsets, out=rows, stream=stream)
    out = _lib.mm_combine_rows(y, places, w=topk_w, stream=stream)
    return out, ExpertsSaved(hidden, places, offsets, row_w, codes, scales)


def _check_backward(d_out, s: ExpertsSaved, w_gate_up, w_down, d_w_gate_up, d_w_down,
                    accumulate: bool) -> None:
    """Refuses what a later call of the step would, before the first one writes: a gradient
    that one call had added to would be added to twice when the step is tried again."""
    if accumulate and (d_w_gate_up is None or d_w_down is None):
        raise ValueError("accumulate needs d_w_gate_up and d_w_down")
    (T, H), E, I = s.hidden.shape, s.offsets.shape[0] - 1, s.codes.shape[1] // 2
    up, down = (E, 2 * I, H), (E, H, I)
    for t, shape, name in ((d_out, (T, H), "d_out"), (w_gate_up, up, "w_gate_up"),
                           (w_down, down, "w_down"), (d_w_gate_up, up, "d_w_gate_up"),
                           (d_w_down, down, "d_w_down")):
        _lib._shape(t, shape, name)
    for t, name in ((d_out, "d_out"), (w_gate_up, "w_gate_up"), (w_down, "w_down"),
                    (d_w_gate_up, "d_w_gate_up"), (d_w_down, "d_w_down")):
        fp32 = name.startswith("d_w") and t is not None and t.dtype == torch.float32
        at = _lib._ptr(t, torch.float32 if fp32 else s.hidden.dtype, name)
        if at is not None and at % 16 and T > 0:
            raise ValueError(f"{name} must be 16-byte aligned")
    _lib._device("moe_experts_train_backward", s.hidden, d_out, w_gate_up, w_down,
                 d_w_gate_up, d_w_down)


def moe_experts_train_backward(d_out, saved: ExpertsSaved, w_gate_up, w_down,
                               d_w_gate_up: Optional[torch.Tensor] = None,
                               d_w_down: Optional[torch.Tensor] = None, accumulate: bool = False,
                               weight_dtype=None, stream=None) -> ExpertsGrads:
    """The gradients of moe_experts_train for d_out [T, H]. d_w_gate_up and d_w_down:
    results to write into, or to add to with accumulate, which needs both (of the weights'
    type or float32); weight_dtype: the type of new ones. A call that is refused has
    written nothing."""
    s = saved
    _check_backward(d_out, s, w_gate_up, w_down, d_w_gate_up, d_w_down, accumulate)
    d_rows, _ = _lib.mm_dispatch_rows(d_out, s.places, stream=stream)
    da = _lib.mm_grouped_product_dx(d_rows, w_down, s.offsets, stream=stream)
    dz, act, d_row_w = _lib.mm_swiglu_pack_backward(s.codes, s.scales, da, row_w=s.row_w,
                                                    offsets=s.offsets, stream=stream)
    d_w_down = _lib.mm_grouped_product_dw(d_rows, act, s.offsets, out=d_w_down,
                                          out_dtype=weight_dtype if d_w_down is None else None,
                                          accumulate=accumulate, stream=stream)
    rows, _ = _lib.mm_dispatch_rows(s.hidden, s.places, rows=d_rows, stream=stream)
    d_w_gate_up = _lib.mm_grouped_product_dw(dz, rows, s.offsets, out=d_w_gate_up,
                                             out_dtype=weight_dtype if d_w_gate_up is None else None,
                                             accumulate=accumulate, stream=stream)
    dx = _lib.mm_grouped_product_dx(dz, w_gate_up, s.offsets, out=rows, stream=stream)
    d_hidden, d_topk_w = _lib.mm_combine_rows(dx, s.places, row_values=d_row_w, stream=stream)
    return ExpertsGrads(d_hidden, d_topk_w, d_w_gate_up, d_w_down)
