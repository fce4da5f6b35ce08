"""A GraphGPS layer's attention branch and what surrounds it, on libkmip.

k-Maximum Inner Product Attention for Graph Transformers and the Expressive
Power of GraphGPS (Figure 1: one GraphGPS layer): node features x [N, hidden]
are projected to queries, keys and values of H heads of width d (hidden =
H d), every query attends over its k best keys of its own graph, and the
heads are projected back and added to the input:

    [Q | K | V] = x W_qkv + b_qkv            one GEMM, [N, 3 H d]
    Q, K        = rotary(Q, K, positions)    optional: coordinates of the nodes
    A           = kmip_attention(Q, K, V)    libkmip (C ABI), [N, H, d]
    y           = x + A W_o + b_o

GraphTransformerLayer puts a group norm per graph before that branch and a
second one with a gated feed-forward block behind it, each added to its input.

The projections are plain GEMMs (torch / cuBLAS); attention, positions, norm
and feed-forward block run in libkmip's kernels through the ctypes binding,
forward and backward, and everything is trainable through torch autograd.  The
local (message-passing) branch of a GraphGPS layer is not part of this module.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import binding


def _packed(t):
    """t contiguous and 16-byte aligned, as the attention and the feed-forward
    block take it; a copy where it is not (part of a longer row, say)."""
    t = t.contiguous()
    return t if t.data_ptr() % 16 == 0 else t.clone()


class KmipAttentionFunction(torch.autograd.Function):
    """Autograd wrapper of kmip_attn_fwd / kmip_attn_bwd.

    Q, K, V: [N, H, d] CUDA tensors (bf16 or fp32); offsets: int32 [G+1]
    CUDA tensor or None.  Returns out [N, H, d] in the input dtype; the
    selection (idx) gets no gradient.  Gradients come back in the input
    dtype (the library computes them in fp32)."""

    @staticmethod
    def forward(ctx, Q, K, V, offsets, k: int, scale: float):
        Q, K, V = _packed(Q), _packed(K), _packed(V)
        out, idx, lse = binding.attn_fwd(Q, K, V, k, scale, offsets)
        ctx.save_for_backward(Q, K, V, idx, lse)
        ctx.scale = scale
        ctx.mark_non_differentiable(idx)
        return out, idx

    @staticmethod
    def backward(ctx, dout, _didx):
        Q, K, V, idx, lse = ctx.saved_tensors
        dQ, dK, dV = binding.attn_bwd(_packed(dout.to(Q.dtype)), Q, K, V, idx, lse,
                                      ctx.scale)
        return dQ.to(Q.dtype), dK.to(K.dtype), dV.to(V.dtype), None, None, None


def kmip_attention(Q, K, V, k: int, scale: float | None = None, offsets=None):
    """k-MIP attention with autograd; returns (out [N, H, d], idx [N, H, k])."""
    if scale is None:
        scale = 1.0 / math.sqrt(Q.shape[-1])
    return KmipAttentionFunction.apply(Q, K, V, offsets, int(k), float(scale))


def _turnable(x, interleaved: bool):
    """x [N, H, d], or a copy where kmip_rotary cannot take its layout: a
    head's elements adjacent and, interleaved, every pair aligned as one."""
    if x.stride(2) != 1 or interleaved and (
            x.data_ptr() % (2 * x.element_size()) or
            any(s % 2 for s, n in zip(x.stride()[:2], x.shape) if n > 1)):
        return x.clone(memory_format=torch.contiguous_format)
    return x


class RotaryFunction(torch.autograd.Function):
    """Autograd wrapper of kmip_rotary: the gradient is the inverse turn.
    Positions and frequencies get no gradient."""

    @staticmethod
    def forward(ctx, x, pos, freq, axis, interleaved: bool):
        ctx.save_for_backward(pos, freq, axis)
        ctx.interleaved = interleaved
        return binding.rotary(_turnable(x, interleaved), pos, freq, axis,
                              interleaved=interleaved)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        pos, freq, axis = ctx.saved_tensors
        dx = binding.rotary(_turnable(dout, ctx.interleaved), pos, freq, axis, inverse=True,
                            interleaved=ctx.interleaved)
        return dx, None, None, None, None


class AxisRotary(torch.nn.Module):
    """Rotary positions of heads of width d by several coordinates.

    The pairs of a head are dealt to the axes in runs (``sections``, by
    default as even as they go); axis a's pair j of n turns by
    coordinate * base ** (-j / n).  ``pairs`` < d / 2 leaves the rest of the
    head unturned.  Call with x [N, H, d] and positions [N, axes] (fp32, int32
    or int64)."""

    def __init__(self, d: int, axes: int, base: float = 10000.0, sections=None,
                 pairs: int | None = None, interleaved: bool = False):
        super().__init__()
        if axes < 1:
            raise ValueError("axes must be positive")
        if sections is None:
            pairs = d // 2 if pairs is None else pairs
            sections = [pairs // axes + (a < pairs % axes) for a in range(axes)]
        sections = [int(n) for n in sections]
        if len(sections) != axes or min(sections) < 0 or 2 * sum(sections) > d:
            raise ValueError("sections: one count of pairs per axis, at most d / 2 in all")
        self.d, self.axes, self.sections, self.interleaved = d, axes, sections, interleaved
        # kept on the host in fp64 (a module's .to(dtype) would round a buffer)
        # and copied to a device once
        self._freq = [base ** (-j / n) for n in sections for j in range(n)]
        self._axis = [a for a, n in enumerate(sections) for _ in range(n)]
        self._tables = {}

    def tables(self, device):
        """(freq, axis) on `device`."""
        device = torch.device(device)
        if device not in self._tables:
            # not inference tensors, even when first made there: training saves them
            with torch.inference_mode(False):
                self._tables[device] = (
                    torch.tensor(self._freq, dtype=torch.float64, device=device),
                    torch.tensor(self._axis, dtype=torch.int32, device=device))
        return self._tables[device]

    def forward(self, x, pos):
        if x.shape[-1] != self.d or pos.shape[-1] != self.axes:
            raise ValueError(f"expected heads of {self.d} and {self.axes} coordinates")
        if pos.requires_grad:
            raise ValueError("positions get no gradient")
        freq, axis = self.tables(x.device)
        return RotaryFunction.apply(x, pos.contiguous(), freq, axis, self.interleaved)


class GroupNormFunction(torch.autograd.Function):
    """Autograd wrapper of kmip_group_norm_fwd / kmip_group_norm_bwd."""

    @staticmethod
    def forward(ctx, x, weight, bias, offsets, groups: int, eps: float, act: str):
        x = x.contiguous()
        y, mean, rstd = binding.group_norm_fwd(x, weight, bias, groups, eps, act, offsets)
        ctx.save_for_backward(x, weight, bias, offsets, mean, rstd)
        ctx.groups, ctx.act = groups, act
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, weight, bias, offsets, mean, rstd = ctx.saved_tensors
        dx, dw, db = binding.group_norm_bwd(dy.contiguous(), x, weight, bias, mean, rstd,
                                            ctx.groups, ctx.act, offsets)
        return dx, dw, db, None, None, None, None


class GraphGroupNorm(torch.nn.Module):
    """Group norm over the nodes of each graph and the channels of each group,
    channels last, with an activation ("none", "silu", "gelu", "relu")."""

    def __init__(self, channels: int, groups: int, eps: float = 1e-5, act: str = "none",
                 affine: bool = True, dtype=torch.bfloat16, device=None):
        super().__init__()
        if groups < 1 or channels % groups:
            raise ValueError("channels must be a multiple of groups")
        binding._act_code(act)
        self.groups, self.eps, self.act = groups, eps, act
        self.weight = self.bias = None
        if affine:
            self.weight = torch.nn.Parameter(torch.ones(channels, dtype=dtype, device=device))
            self.bias = torch.nn.Parameter(torch.zeros(channels, dtype=dtype, device=device))

    def forward(self, x, offsets=None):
        return GroupNormFunction.apply(x, self.weight, self.bias, offsets, self.groups, self.eps,
                                       self.act)


class GatedFeedForwardFunction(torch.autograd.Function):
    """Autograd wrapper of kmip_ffn_fwd / kmip_ffn_bwd (which keeps nothing of
    the forward but its inputs)."""

    @staticmethod
    def forward(ctx, x, wg, wu, wd, act: str):
        x, wg, wu, wd = _packed(x), _packed(wg), _packed(wu), _packed(wd)
        ctx.save_for_backward(x, wg, wu, wd)
        ctx.act = act
        return binding.ffn_fwd(x, wg, wu, wd, act)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        x, wg, wu, wd = ctx.saved_tensors
        return (*binding.ffn_bwd(_packed(dy), x, wg, wu, wd, ctx.act), None)


class GatedFeedForward(torch.nn.Module):
    """y = (act(x Wg^T) * (x Wu^T)) Wd^T; hidden and width multiples of 8."""

    def __init__(self, hidden: int, width: int, act: str = "silu", dtype=torch.bfloat16,
                 device=None):
        super().__init__()
        if hidden % 8 or width % 8:
            raise ValueError("hidden and width must be multiples of 8")
        binding._act_code(act)
        self.act = act

        def weight(rows, cols):
            w = torch.empty(rows, cols, dtype=dtype, device=device)
            return torch.nn.Parameter(torch.nn.init.kaiming_uniform_(w, a=math.sqrt(5)))

        self.gate, self.up = weight(width, hidden), weight(width, hidden)
        self.down = weight(hidden, width)

    def forward(self, x):
        return GatedFeedForwardFunction.apply(x, self.gate, self.up, self.down, self.act)


class KmipGlobalAttention(torch.nn.Module):
    """GraphGPS global-attention block: fused QKV projection, k-MIP
    attention, output projection and residual (see the module docstring).
    With ``rotary`` (an AxisRotary of the head width) queries and keys are
    turned by the positions given to forward."""

    def __init__(self, hidden: int, heads: int, k: int, dtype=torch.bfloat16, device=None,
                 rotary: AxisRotary | None = None):
        super().__init__()
        if hidden % heads:
            raise ValueError("hidden must be a multiple of heads")
        self.hidden, self.heads, self.d, self.k = hidden, heads, hidden // heads, k
        self.scale = 1.0 / math.sqrt(self.d)
        self.qkv = torch.nn.Linear(hidden, 3 * hidden, dtype=dtype, device=device)
        self.proj = torch.nn.Linear(hidden, hidden, dtype=dtype, device=device)
        self.rotary = rotary

    def attend(self, x, offsets=None, pos=None):
        """The block without its residual."""
        if (pos is None) != (self.rotary is None):
            raise ValueError("positions go with rotary, and rotary needs positions")
        N = x.shape[0]
        qkv = self.qkv(x).view(N, 3, self.heads, self.d)
        q, k = qkv[:, 0], qkv[:, 1]
        if self.rotary is not None:
            q, k = self.rotary(q, pos), self.rotary(k, pos)
        a, idx = kmip_attention(q, k, qkv[:, 2], self.k, self.scale, offsets)
        self.last_idx = idx
        return self.proj(a.reshape(N, self.hidden))

    def forward(self, x, offsets=None, pos=None):
        return x + self.attend(x, offsets, pos)


class GraphTransformerLayer(torch.nn.Module):
    """x + attend(norm(x)), then + ffn(norm(.)): the attention branch and the
    feed-forward part of a GraphGPS layer, normalised per graph."""

    def __init__(self, hidden: int, heads: int, k: int, width: int, groups: int, axes: int = 0,
                 act: str = "silu", dtype=torch.bfloat16, device=None):
        super().__init__()
        rotary = AxisRotary(hidden // heads, axes) if axes else None
        self.norm1 = GraphGroupNorm(hidden, groups, dtype=dtype, device=device)
        self.attn = KmipGlobalAttention(hidden, heads, k, dtype=dtype, device=device,
                                        rotary=rotary)
        self.norm2 = GraphGroupNorm(hidden, groups, dtype=dtype, device=device)
        self.ffn = GatedFeedForward(hidden, width, act, dtype=dtype, device=device)

    def forward(self, x, offsets=None, pos=None):
        x = x + self.attn.attend(self.norm1(x, offsets), offsets, pos)
        return x + self.ffn(self.norm2(x, offsets))
