"""Caller-side glue around the VMoBA kernels: an autograd function over the C
ABI's forward / backward, and a self-attention module that places VMoBA where
a video DiT has full self-attention.

VMoBA notes, overall framework: VMoBA replaces the attention computation
itself (same input and output shapes as full attention); key design 1: layer
l partitions keys by mode l mod 3; training strategy: tau = 0.25, and the
first 25 % of denoising steps keep full attention.  The projections are plain
GEMMs (``torch.nn.Linear``); every attention step -- partition, pooling,
scores, selection, attention forward and backward -- runs in libvmoba.
"""
from __future__ import annotations

import math

import torch
from torch.autograd.function import once_differentiable

from . import _lib, norm_rope
from ._lib import LayerShape
from .layer import VMoBALayer
from .norm_rope import Act8, NormRope


def _all_pairs(layer: VMoBALayer) -> torch.Tensor:
    """The selection bitmap of dense attention over the layer's blocks."""
    bits = torch.full_like(layer.sel, -1)
    rem = layer.n_blocks % 32
    if rem:
        bits[..., -1] = (1 << rem) - 1
    return bits


class VMoBAFunction(torch.autograd.Function):
    """O = VMoBA(q, k, v) with the selection held constant for the backward
    (the selection is piecewise constant: no gradient flows through it).

    q, k, v: [s][n_heads][head_dim] contiguous CUDA tensors of the layer's
    dtype.  ``full`` selects every pair (dense attention over the blocks).

    The backward kernels read state the forward left in the layer's buffers
    (permuted keys and values, pair lists, LSE, the fp32 output copy).  Each
    call keeps its own selection bitmap and records the layer's generation; if
    another call wrote to that state in between (two micro-batches, activation
    checkpointing, a full-attention call, another selection), the backward
    first restores this call's state by re-running partition, plan and forward
    on its saved inputs and selection -- the same deterministic kernels, so the
    restored state is bit-identical -- and then runs.
    """

    @staticmethod
    def forward(ctx, q, k, v, layer: VMoBALayer, tau: float, full: bool, scale: float):
        if full:
            layer.partition_only(k, v)
            layer.use_selection(_all_pairs(layer))
        else:
            layer.select(q, k, v, tau, scale)
        out, _ = layer.forward(q, scale)
        ctx.layer, ctx.scale = layer, scale
        ctx.generation = layer.generation
        ctx.save_for_backward(q, k, v, layer.sel.clone())
        return out.clone()

    @staticmethod
    def backward(ctx, dout):
        q, k, v, sel = ctx.saved_tensors
        layer = ctx.layer
        if layer.generation != ctx.generation:
            # another call replaced a part of this one's state: rebuild it
            layer.partition_only(k, v)
            layer.use_selection(sel)
            layer.forward(q, ctx.scale)
            ctx.generation = layer.generation
        dq, dk, dv = layer.backward(q, dout.contiguous(), ctx.scale)
        return dq.clone(), dk.clone(), dv.clone(), None, None, None, None


class VMoBANormRopeFunction(torch.autograd.Function):
    """O = VMoBA(rot(norm(q)), rot(norm(k)), v) of the projection's raw rows
    qkv [s][3][n_heads][head_dim]; the norm weights are fp32 [head_dim] or
    None (ones), table and dims the rotation's (norm_rope.rope_table).

    Saved for the backward are the raw rows, or with ``checkpoint8`` their
    8-bit checkpoint (written by the forward's own pass), and the selection.
    The other state stays in the layer's buffers; if another call wrote to it
    in between, the backward rebuilds it from what was saved: from the raw
    rows bit for bit, from a checkpoint as the attention of the values it
    holds.  The gradients of the raw rows and norm weights are taken at the
    saved values in either case.
    """

    @staticmethod
    def forward(ctx, qkv, q_weight, k_weight, layer: VMoBALayer, table, dims, eps: float,
                tau: float, full: bool, scale: float, checkpoint8: bool):
        norm = NormRope(q_weight, k_weight, eps, table, dims)
        checkpoint8 = checkpoint8 and any(ctx.needs_input_grad[:3])
        ckpt = Act8.empty(qkv.shape, layer.shape.head_dim, qkv.device) if checkpoint8 else None
        layer.prologue(qkv, norm, ckpt)
        if full:
            layer.use_selection(_all_pairs(layer))
        else:
            layer.select_pooled(layer.q, tau, scale)
        out, _ = layer.forward(layer.q, scale)
        ctx.layer, ctx.scale, ctx.dims, ctx.eps = layer, scale, dims, eps
        ctx.generation = layer.generation
        ctx.has = q_weight is not None, k_weight is not None, table is not None, checkpoint8
        given = [t for t in (q_weight, k_weight, table) if t is not None]
        ctx.save_for_backward(layer.sel.clone(), *given,
                              *((ckpt.codes, ckpt.scales) if checkpoint8 else (qkv,)))
        return out.clone()

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        layer, saved = ctx.layer, list(ctx.saved_tensors)
        sel = saved.pop(0)
        q_weight, k_weight, table = (saved.pop(0) if has else None for has in ctx.has[:3])
        norm = NormRope(q_weight, k_weight, ctx.eps, table, ctx.dims)
        raw = Act8(*saved, layer.shape.head_dim) if ctx.has[3] else saved[0]
        if layer.generation != ctx.generation:
            # another call replaced a part of this one's state: rebuild it
            layer.prologue(raw, norm)
            layer.use_selection(sel)
            layer.forward(layer.q, ctx.scale)
            ctx.generation = layer.generation
        s, h, d = layer.shape.s, layer.shape.n_heads, layer.shape.head_dim
        dqkv = torch.empty((s, 3, h, d), dtype=layer.dtype, device=dout.device)
        need_q, need_k = ctx.needs_input_grad[1:3]
        dweight = torch.empty((2, d), dtype=torch.float32, device=dout.device) \
            if need_q or need_k else None
        layer.backward_raw(raw, norm, dout.contiguous(), dqkv, dweight, ctx.scale)
        return (dqkv, dweight[0] if need_q else None, dweight[1] if need_k else None) + (None,) * 8


class Linear8Function(torch.autograd.Function):
    """y = x W^T + b, x [...][cols] kept for the weight's gradient as an 8-bit
    checkpoint of its rows: dx = dy W, dW = dy^T x8, db = sum dy.  Without a
    gradient of W nothing is stored.  Under autocast the products of both
    passes are in the region's type, as the plain layer's."""

    @staticmethod
    @torch.amp.custom_fwd(device_type="cuda")
    def forward(ctx, x, weight, bias):
        kept = ()
        if ctx.needs_input_grad[1]:
            rows = x.reshape(-1, x.shape[-1])
            if rows.stride(1) != 1 or rows.stride(0) < rows.shape[1]:
                rows = rows.contiguous()
            ckpt = Act8.empty(rows.shape, 128 if rows.shape[1] % 128 == 0 else 64, x.device)
            norm_rope.act8_pack(rows, ckpt)
            ctx.group, ctx.x_dtype = ckpt.group, x.dtype
            kept = ckpt.codes, ckpt.scales
        ctx.save_for_backward(weight if ctx.needs_input_grad[0] else None, *kept)
        return torch.nn.functional.linear(x, weight, bias)

    @staticmethod
    @once_differentiable
    @torch.amp.custom_bwd(device_type="cuda")
    def backward(ctx, dy):
        weight, *kept = ctx.saved_tensors
        dx = dw = db = None
        if ctx.needs_input_grad[0]:
            dx = dy @ weight
        dy = dy.reshape(-1, dy.shape[-1])
        if ctx.needs_input_grad[1]:
            dtype = dy.dtype if dy.dtype in (torch.bfloat16, torch.float32) else ctx.x_dtype
            ckpt = Act8(*kept, ctx.group)
            x = torch.empty(ckpt.codes.shape, dtype=dtype, device=dy.device)
            norm_rope.act8_unpack(ckpt, x)
            dw = dy.t() @ x
        if ctx.needs_input_grad[2]:
            db = dy.sum(0)
        return dx, dw, db


class Linear8(torch.nn.Linear):
    """A linear layer that keeps its input for the weight's gradient in 8 bits
    while ``checkpoint8`` is set."""

    checkpoint8 = True

    def forward(self, x):
        if self.checkpoint8 and torch.is_grad_enabled():
            return Linear8Function.apply(x, self.weight, self.bias)
        return super().forward(x)


class VMoBASelfAttention(torch.nn.Module):
    """Self-attention of one DiT layer over a (T, H, W) video latent with
    VMoBA in place of full attention.

    x: [s][dim] tokens in (t, y, x) order -> [s][dim].  ``boxes`` gives the
    (bt, bh, bw) box of each partition mode (mode = layer_idx mod 3);
    ``full_attention=True`` in ``forward`` keeps every pair (the early
    denoising steps of the training strategy).

    ``qk_norm`` normalises each head's query and key (RMS norm with fp32
    weights ``q_norm``, ``k_norm`` of head_dim); ``rope`` then rotates them by
    the token's position, with that many of a head's dimensions for t, y and x
    (``True``: the usual split, norm_rope.rope_dims), frequencies
    ``rope_base`` ** (-2i / dim), positions counted from ``rope_origin``.
    ``checkpoint8`` keeps what the backward needs of the activations in 8 bits:
    the projections' inputs and the raw q, k, v (5 bytes and 5 scales of a
    group for each token and channel in place of 10 in bf16).  Rotation and
    checkpoints are part of the norm's pass, so both need ``qk_norm``.  A
    module put in a projection's place keeps what it keeps itself.

    ``layer`` shares another module's buffers (``other.layer``, of the same
    latent, heads, boxes and mode), which are far more than an activation: 14
    bytes a token and channel in bf16, and the workspace.  Every module but
    the last to run forward then rebuilds its state in the backward (one more
    attention forward).
    """

    def __init__(self, dim: int, n_heads: int, T: int, H: int, W: int, layer_idx: int,
                 boxes, tau: float = 0.25, dtype=torch.bfloat16, device="cuda", *,
                 qk_norm: bool = False, norm_eps: float = 1e-6, rope=None,
                 rope_base: float = 10000.0, rope_origin=(0, 0, 0), checkpoint8: bool = False,
                 layer: VMoBALayer | None = None):
        super().__init__()
        if not qk_norm and (rope or checkpoint8):
            raise ValueError("rope and checkpoint8 need qk_norm")
        if dim % n_heads:
            raise ValueError("dim must be a multiple of n_heads")
        self.n_heads, self.head_dim = n_heads, dim // n_heads
        self.mode = _lib.mode_for_layer(layer_idx)
        self.tau = float(tau)
        linear = Linear8 if qk_norm else torch.nn.Linear
        self.qkv = linear(dim, 3 * dim, bias=True, device=device, dtype=dtype)
        self.proj = linear(dim, dim, bias=True, device=device, dtype=dtype)
        bt, bh, bw = boxes[self.mode]
        dt = "bf16" if dtype == torch.bfloat16 else "f32"
        self.shape = LayerShape(T, H, W, n_heads, self.head_dim, self.mode, bt, bh, bw, dt)
        if layer is not None and layer.shape != self.shape:
            raise ValueError(f"layer: expected one of shape {self.shape}, got {layer.shape}")
        self.layer = VMoBALayer(self.shape, device=device) if layer is None else layer
        self.scale = 1.0 / math.sqrt(self.head_dim)
        self.norm_eps, self.checkpoint8 = float(norm_eps), checkpoint8
        # like the layer's buffers, the rotation's table is the module's own: fp32
        # whatever type the parameters are moved to
        self.rope_dims, self.rope_table = (0, 0, 0), None
        self.q_norm = self.k_norm = None
        if qk_norm:
            self.q_norm, self.k_norm = (
                torch.nn.Parameter(torch.ones(self.head_dim, dtype=torch.float32, device=device))
                for _ in range(2))
        if rope:
            self.rope_dims = norm_rope.rope_dims(self.head_dim) if rope is True else tuple(rope)
            self.rope_table = norm_rope.rope_table(self.shape, self.rope_dims, rope_base,
                                                   rope_origin, device)

    @property
    def checkpoint8(self) -> bool:
        return self._checkpoint8

    @checkpoint8.setter
    def checkpoint8(self, on):
        self._checkpoint8 = bool(on)
        for m in (self.qkv, self.proj):
            if isinstance(m, Linear8):
                m.checkpoint8 = self._checkpoint8

    def forward(self, x: torch.Tensor, full_attention: bool = False) -> torch.Tensor:
        s = x.shape[0]
        qkv = self.qkv(x).view(s, 3, self.n_heads, self.head_dim)
        if self.q_norm is not None:
            o = VMoBANormRopeFunction.apply(
                qkv, self.q_norm.float(), self.k_norm.float(), self.layer, self.rope_table,
                self.rope_dims, self.norm_eps, self.tau, bool(full_attention), self.scale,
                self.checkpoint8 and torch.is_grad_enabled())
            return self.proj(o.view(s, -1))
        q, k, v = (qkv[:, i].contiguous() for i in range(3))
        o = VMoBAFunction.apply(q, k, v, self.layer, self.tau, bool(full_attention), self.scale)
        return self.proj(o.reshape(s, self.n_heads * self.head_dim))


def full_attention_steps(n_steps: int, fraction: float = 0.25) -> int:
    """Denoising steps (from the first) that keep full attention: the notes'
    training strategy keeps it for the first 25 % of steps."""
    return int(math.ceil(fraction * n_steps))
