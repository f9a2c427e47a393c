"""The experts' block of a mixture-of-experts MLP whose layers are LiftQuant layers.

Each expert is two layers o = diag(s) . W_q . (blockdiag(M^T) . T^{-1} . a) (LiftQuant
paper note, "Key designs" 1, 3 and 4) with a gate between them. M is global and T belongs to
the layer, so all experts of a layer share them and a token is lifted once, whatever
number of experts it goes to:

    h = act(gate_e(u)) * up_e(u),   u = lift(x)
    o = x + sum_j weights[t][j] * down_{e_j}(lift(h))

The arithmetic is the library's kernels; this module only holds the weights and calls them.
"""

from __future__ import annotations


def interleave_rows(gate, up):
    """Packed signs [experts][out][K/32], or scales [experts][out], of the gate and the up layer ->
    one array of 2*out rows in the order gate 0, up 0, gate 1, up 1, ..."""
    import torch
    if gate.shape != up.shape or gate.dim() < 2:
        raise ValueError("gate and up must have the same shape, [experts][out] or [experts][out][K/32]")
    both = torch.stack((gate, up), dim=2)
    return both.reshape(gate.shape[0], 2 * gate.shape[1], *gate.shape[2:]).contiguous()


def _whitening(tinv, channels, M, name):
    """Checks T^{-1}: the lift takes its number of blocks from `channels` and reads them all."""
    import torch
    if tinv is None:
        return
    t = tinv.shape[-1] if tinv.dim() == 3 else 0
    if t < 1 or tuple(tinv.shape) != (channels // t, t, t) or channels % t:
        raise ValueError(f"{name} must be [{channels}/t][t][t]")
    if tinv.dtype != torch.float32 or not tinv.is_contiguous() or tinv.device != M.device:
        raise ValueError(f"{name} must be contiguous float32 on {M.device}")


class ExpertMLP:
    """Experts of one MLP block, all tensors on one device.

    gate_up    : int32 [experts][2*hidden][K1/32], rows interleaved (interleave_rows), K1 = lifted_dim(model)
    gate_up_s  : fp32 [experts][2*hidden]
    down       : int32 [experts][model][K2/32], K2 = lifted_dim(hidden); down_s: fp32 [experts][model]
    M          : fp32 [d][D]; tinv_in, tinv_hidden: T^{-1} of the two layers as fp32 blocks [model/t][t][t]
                 and [hidden/t][t][t], or None
    """

    def __init__(self, gate_up, gate_up_s, down, down_s, M, tinv_in=None, tinv_hidden=None, act="silu"):
        import torch

        from . import lifted_dim
        if gate_up.dim() != 3 or down.dim() != 3 or M.dim() != 2:
            raise ValueError("gate_up and down must be [experts][out][K/32] and M [d][D]")
        if M.dtype != torch.float32 or not M.is_contiguous():
            raise ValueError("M must be contiguous float32")
        self.gate_up, self.gate_up_s, self.down, self.down_s = gate_up, gate_up_s, down, down_s
        self.M, self.tinv_in, self.tinv_hidden, self.act = M, tinv_in, tinv_hidden, act
        self.experts, self.hidden, self.model = gate_up.shape[0], gate_up.shape[1] // 2, down.shape[1]
        d, D = M.shape
        self.K1, self.K2 = lifted_dim(self.model, d, D), lifted_dim(self.hidden, d, D)
        if gate_up.shape[2] * 32 != self.K1 or down.shape[2] * 32 != self.K2 or down.shape[0] != self.experts:
            raise ValueError("packed widths do not match the lifted sizes of M")
        _whitening(tinv_in, self.model, M, "tinv_in")
        _whitening(tinv_hidden, self.hidden, M, "tinv_hidden")

    def step(self, x, expert_ids, weights, residual=True, stream=None):
        """x bf16 [tokens][model], expert_ids int32 [tokens][topk], weights fp32 [tokens][topk] -> bf16 [tokens][model].

        Nothing is read back to the host, so the step can be captured in a CUDA graph. Ids
        outside 0..experts-1 are skipped."""
        import torch
        from . import _on, combine_rows, gemm_grouped, group_rows, lift_activations
        if x.dim() != 2 or x.shape[1] != self.model or expert_ids.dim() != 2 or expert_ids.shape[0] != x.shape[0]:
            raise ValueError(f"x must be [tokens][{self.model}] and expert_ids [tokens][topk]")
        if weights.shape != expert_ids.shape or x.dtype != torch.bfloat16:
            raise ValueError("x must be bfloat16 and weights [tokens][topk]")
        if x.device != self.M.device:
            raise ValueError(f"x must be on the block's device, {self.M.device}")
        n = expert_ids.numel()
        with _on(x, stream):
            u = lift_activations(x, self.M, self.K1, tinv=self.tinv_in, u_dtype="bf16")
            offsets, rows, slots = group_rows(expert_ids, self.experts)
            h = gemm_grouped(self.gate_up, self.gate_up_s, u, offsets, n, rows=rows, act=self.act, glu=True,
                             o_dtype="bf16")
            u = lift_activations(h, self.M, self.K2, tinv=self.tinv_hidden, u_dtype="bf16")
            y = gemm_grouped(self.down, self.down_s, u, offsets, n, o_dtype="bf16")
            return combine_rows(y, slots, weights, residual=x if residual else None)
