"""The one-pass attention layer as a sequence of library calls.

forward:  opr_rope(q), opr_rope(k) by the layout's position ids (bf16 in,
          fp16 out) -> opr_attn_fwd
backward: opr_attn_bwd with the position ids, which rotates dq and dk back
          (the gradients w.r.t. the unrotated q and k)
OnePassAttentionLayer puts the layer's projections, the norm of each head of q
and k and any rotary variant around it:
forward:  opr_linear (q, k and v) -> opr_qk_norm_rope -> opr_attn_fwd -> opr_linear
backward: the same calls' gradients in reverse
(One-Pass to Reason: positions from "位置 ID 策略", mask from "分块稀疏注意力掩码").
Every numerical step runs in libopr's CUDA kernels; this module only orders the
calls and keeps buffers.
"""

from __future__ import annotations

import numpy as np
import torch

from ._abi import (Layout, OprError, opr_attn_bwd, opr_attn_fwd, opr_build_layout, opr_linear, opr_linear_bwd,
                   opr_qk_norm_rope, opr_qk_norm_rope_bwd, opr_rope)


def visible_pairs_closed_form(turn_lens, conv_turn_ptr) -> int:
    """Visible (q, k) pairs per head of a one-pass layout, counted per turn.

    With A_i = sum_{j<i}(h_j + r_j) (the history length seen by turn i):
    h rows see A_i + causal h; t rows A_i + h + causal t; r^in rows A_i + h +
    causal r; r^out rows A_i + h + t + causal r.  Used as the useful-work
    count of the throughput metric (the pages' complexity analysis counts the
    same attended pairs).
    """
    tl = np.asarray(turn_lens, dtype=np.int64).reshape(-1, 3)
    cp = np.asarray(conv_turn_ptr, dtype=np.int64)
    total = 0
    for c in range(len(cp) - 1):
        A = 0
        for h, t, r in tl[cp[c]:cp[c + 1]]:
            total += h * A + h * (h + 1) // 2
            total += t * (A + h) + t * (t + 1) // 2
            total += r * (A + h) + r * (r + 1) // 2
            total += r * (A + h + t) + r * (r + 1) // 2
            A += h + r
    return int(total)


def useful_flops(pairs: int, hq: int, d: int, backward: bool) -> float:
    """4 d flops per visible pair and q head forward; 2.5 times that backward."""
    f = 4.0 * d * pairs * hq
    return f * 3.5 if backward else f


def one_pass_forward(q_pre, k_pre, v, lay: Layout, base: float, scale=None, out_dtype=torch.float32):
    """RoPE (bf16 in, fp16 out), an fp16 copy of v (so that P V runs with fp16 P), all three
    written in the layout's attention order, then masked attention.  Returns (o, lse, q_rot,
    k_rot): o and lse in the stream order, q_rot and k_rot in the attention order (the form
    one_pass_backward takes)."""
    q = torch.empty(q_pre.shape, dtype=torch.float16, device=q_pre.device)
    k = torch.empty(k_pre.shape, dtype=torch.float16, device=k_pre.device)
    v16 = torch.empty(v.shape, dtype=torch.float16, device=v.device)
    # rotated q, k and the fp16 v go to the attention order (rows lay.attn_pos)
    opr_rope(q_pre, lay.pos_id, base, out=q, dev_status=lay.dev_status, row_map=lay.attn_pos)
    opr_rope(k_pre, lay.pos_id, base, out=k, dev_status=lay.dev_status, row_map=lay.attn_pos)
    opr_rope(v, None, base, out=v16, dev_status=lay.dev_status, row_map=lay.attn_pos)
    o, lse = opr_attn_fwd(q, k, v16, lay, scale, out_dtype)
    return o, lse, q, k


def one_pass_backward(q_rot, k_rot, v, o, do, lse, lay: Layout, base: float, scale=None):
    """Gradients w.r.t. the unrotated q, k and v (the backward rotates dq and dk back)."""
    return opr_attn_bwd(q_rot, k_rot, v, o, do, lse, lay, scale, rope_base=base)


class OnePassAttention:
    """Layout built once from per-turn lengths, then forward/backward calls.

    >>> att = OnePassAttention(turn_lens, conv_turn_ptr, seq_conv_ptr, base=1e6)
    >>> o, lse, q_rot, k_rot = att.forward(q, k, v)
    >>> dq, dk, dv = att.backward(q_rot, k_rot, v, o, do, lse)
    """

    def __init__(self, turn_lens, conv_turn_ptr, seq_conv_ptr, base: float, device="cuda"):
        self.layout = opr_build_layout(turn_lens, conv_turn_ptr, seq_conv_ptr, device=device)
        self.base = base

    def forward(self, q_pre, k_pre, v, scale=None, out_dtype=torch.float32):
        return one_pass_forward(q_pre, k_pre, v, self.layout, self.base, scale, out_dtype)

    def backward(self, q_rot, k_rot, v, o, do, lse, scale=None):
        return one_pass_backward(q_rot, k_rot, v, o, do, lse, self.layout, self.base, scale)


class OnePassAttentionLayer:
    """The attention layer from hidden states to hidden states, bf16.

    x [tokens, width] -> q, k, v = x w_qkv^T + b_qkv -> each head of q and k normed, weighted and rotated ->
    masked attention -> o w_o^T + b_o + residual.  w_qkv [(hq + 2 hkv) head_dim, width] holds the rows of q, k
    and v in that order, w_o [width, hq head_dim]; ``freq`` and ``rotary_scale`` come from
    opr_rotary_frequencies.

    >>> freq, s = opr.opr_rotary_frequencies(128, 1e6)
    >>> layer = OnePassAttentionLayer(turn_lens, conv_turn_ptr, seq_conv_ptr, 32, 8, 128, freq, s)
    >>> y, saved = layer.forward(x, w_qkv, w_o, q_weight, k_weight, residual=x_stream)
    >>> grads = layer.backward(dy, saved)            # the residual's gradient is dy
    """

    def __init__(self, turn_lens, conv_turn_ptr, seq_conv_ptr, hq: int, hkv: int, head_dim: int, freq: torch.Tensor,
                 rotary_scale: float = 1.0, interleaved: bool = False, eps: float = 1e-6, device="cuda"):
        self.layout = opr_build_layout(turn_lens, conv_turn_ptr, seq_conv_ptr, device=device)
        self.hq, self.hkv, self.head_dim = hq, hkv, head_dim
        self.rotation = dict(pos_id=self.layout.pos_id, freq=freq, eps=eps, interleaved=interleaved,
                             scale=rotary_scale)

    def forward(self, x, w_qkv, w_o, q_weight, k_weight, b_qkv=None, b_o=None, residual=None, scale=None):
        """(y, saved): saved is what backward takes (it refers to x and the weights, without copies)."""
        lay, hq, hkv, d = self.layout, self.hq, self.hkv, self.head_dim
        if x.dtype != torch.bfloat16:
            raise OprError("OnePassAttentionLayer: x must be bf16")
        if x.dim() != 2 or x.shape[0] != lay.total or w_qkv.shape[0] != (hq + 2 * hkv) * d:
            raise OprError("OnePassAttentionLayer: x must have the layout's tokens and w_qkv the rows of q, k and v")
        st, cut = lay.dev_status, (hq + hkv) * d
        bias = (None, None) if b_qkv is None else (b_qkv[:cut], b_qkv[cut:])
        # v apart from q and k: opr_attn_bwd takes it contiguous
        qk = opr_linear(x, w_qkv[:cut], bias[0], dev_status=st).view(-1, hq + hkv, d)
        v = opr_linear(x, w_qkv[cut:], bias[1], dev_status=st).view(-1, hkv, d)
        q_rot, k_rot, v16 = opr_qk_norm_rope(qk[:, :hq], qk[:, hq:], q_weight, k_weight, **self.rotation, v=v,
                                             row_map=lay.attn_pos, dev_status=st)
        o, lse = opr_attn_fwd(q_rot, k_rot, v16, lay, scale, torch.bfloat16)
        y = opr_linear(o.view(-1, hq * d), w_o, b_o, residual=residual, dev_status=st)
        saved = dict(x=x, w_qkv=w_qkv, w_o=w_o, q_weight=q_weight, k_weight=k_weight, qk=qk, v=v, q_rot=q_rot,
                     k_rot=k_rot, o=o, lse=lse, scale=scale, has_b_qkv=b_qkv is not None, has_b_o=b_o is not None)
        return y, saved

    def backward(self, dy, saved) -> dict:
        """Gradients of x, w_qkv, w_o, q_weight, k_weight and of the biases that forward was given."""
        lay, hq, hkv, d, s = self.layout, self.hq, self.hkv, self.head_dim, saved
        st, qk = lay.dev_status, s["qk"]
        do, dw_o, db_o = opr_linear_bwd(dy, s["o"].view(-1, hq * d), s["w_o"], bias=s["has_b_o"], dev_status=st)
        # no rope_base: the gradients w.r.t. the rotated q and k, rotated back below with the norm's gradient
        dq, dk, dv = opr_attn_bwd(s["q_rot"], s["k_rot"], s["v"], s["o"], do.view(-1, hq, d), s["lse"], lay,
                                  s["scale"])
        dqkv = torch.empty((lay.total, hq + 2 * hkv, d), dtype=torch.bfloat16, device=dy.device)
        *_, dq_weight, dk_weight = opr_qk_norm_rope_bwd(
            dq, dk, qk[:, :hq], qk[:, hq:], s["q_weight"], s["k_weight"], **self.rotation, dv=dv,
            out=(dqkv[:, :hq], dqkv[:, hq:hq + hkv], dqkv[:, hq + hkv:]), dev_status=st)
        dx, dw_qkv, db_qkv = opr_linear_bwd(dqkv.view(-1, (hq + 2 * hkv) * d), s["x"], s["w_qkv"],
                                            bias=s["has_b_qkv"], dev_status=st)
        return dict(x=dx, w_qkv=dw_qkv, w_o=dw_o, q_weight=dq_weight, k_weight=dk_weight, b_qkv=db_qkv, b_o=db_o)
