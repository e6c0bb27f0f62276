"""The attention half of a video-DiT block around the sparse attention.

    n = norm(x) (1 + scale) + shift            svgear_block_norm
    q, k, v = n W_qkv^T + b_qkv                svgear_mx_quantize, svgear_mx_product
    Q, K, V = heads of rotated, normed q, k, v svgear_qkv_rope
    O = sparse attention                       svgear_forward
    y = O W_out^T + b_out                      svgear_mx_quantize (heads joined), svgear_mx_product
    r = x + gate y,  h = norm(r) (1 + scale') + shift'   svgear_block_norm

Everything runs on one stream through the C entry points; the weights are
MXFP4 (svgear.mx_quantize of a checkpoint's matrices).  No counterpart in the
paper, which evaluates inside such blocks.
"""
from __future__ import annotations

import dataclasses
from typing import Optional, Sequence, Tuple

from . import svgear as sv

__all__ = ["BlockWeights", "attention_block"]


@dataclasses.dataclass
class BlockWeights:
    """Weights of one block: MXFP4 (codes, scales) of W_qkv [3*H*d, D] and W_out [D, H*d], float32 biases
    and the float32 weights of the q and k norms ([H*d] over the token, [d] per head)."""
    qkv: Tuple
    out: Tuple
    qkv_bias: Optional[object] = None
    out_bias: Optional[object] = None
    q_norm: Optional[object] = None
    k_norm: Optional[object] = None


def attention_block(x, w: BlockWeights, H: int, *, Cq: int, Ck: int, iters: int, rho: float, axes: Sequence[int],
                    grid: Sequence[int], shift=None, scale=None, gate=None, next_shift=None, next_scale=None,
                    offsets=None, init_q=None, init_k=None, ws=None, eps: float = 1e-6):
    """x [N, D] (bfloat16, or float32 with the branch in bfloat16) is the residual stream of one sample;
    shift, scale, gate and next_* are float32 [G, D] modulations over the groups of `offsets` (or N/G rows
    each).  The attention is over all N rows: rows from offsets[G] on belong to no group, enter the projection
    as zeros and are zero in r and h, so a sample's padding is left out of x, not behind the last group.
    ws is a workspace of svgear_workspace_size bytes to keep between calls.  Returns (r, h): the new
    residual stream and the normed, modulated input of the block's other half."""
    import torch
    with torch.cuda.device(x.device):
        return _attention_block(x, w, H, Cq, Ck, iters, rho, axes, grid, shift, scale, gate, next_shift, next_scale,
                                offsets, init_q, init_k, ws, eps)


def _attention_block(x, w, H, Cq, Ck, iters, rho, axes, grid, shift, scale, gate, next_shift, next_scale, offsets,
                     init_q, init_k, ws, eps):
    import torch
    N = x.shape[0]
    _, n = sv.block_norm(x, scale=scale, shift=shift, offsets=offsets, eps=eps, dtype=torch.bfloat16)
    d = w.qkv[0].shape[0] // (3 * H)
    qkv = sv.mx_linear(n, *w.qkv, w.qkv_bias).view(N, 3, H, d)
    cols = None if w.q_norm is None else w.q_norm.shape[0]
    norm = sv.SVGEAR_QKNORM_NONE if cols is None else sv.SVGEAR_QKNORM_HEAD if cols == d else sv.SVGEAR_QKNORM_TOKEN
    Q, K, V = sv.qkv_rope(*qkv.unbind(1), axes=axes, grid=grid, wq=w.q_norm, wk=w.k_norm, norm=norm, eps=eps)
    O = sv.forward(Q, K, V, Cq, Ck, iters, rho, 0.0, init_q, init_k, ws=ws)[0]
    y = sv.mx_product(*sv.mx_quantize(O), *w.out, w.out_bias)
    return sv.block_norm(x, y, gate=gate, scale=next_scale, shift=next_shift, offsets=offsets, eps=eps)
