"""What stands around the attention of a layer: the norm of each head's queries
and keys with their (t, y, x) rotation, forward and backward, and activation
checkpoints in 8 bits (include/vmoba.h: vmoba_norm_rope, vmoba_act8_pack).

Binding only, as _lib: arguments are checked and passed on, every step runs in
libvmoba's kernels on the caller's buffers.  The checks are native
(csrc/calls.cpp) and raise ValueError; a call's tensors lie on one CUDA device,
which is made current during the call.  Importing loads neither the library nor
the native calls; the first call does, and raises if they are missing.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
from dataclasses import dataclass

from . import _lib
from ._lib import LayerShape


@dataclass(frozen=True, eq=False)
class NormRope:
    """Norm and rotation of a layer's queries and keys (include/vmoba.h:
    vmoba_norm_rope).  q_weight, k_weight: fp32 CUDA tensors [head_dim], or
    None for ones; table: from rope_table, or None if no pair turns; dims:
    how many of a head's dimensions turn with t, y and x."""
    q_weight: torch.Tensor | None = None
    k_weight: torch.Tensor | None = None
    eps: float = 1e-6
    table: torch.Tensor | None = None
    dims: tuple = (0, 0, 0)


@dataclass(frozen=True, eq=False)
class Act8:
    """An 8-bit activation checkpoint: int8 codes of the activation's shape and
    one fp32 scale for each group of neighbouring values of the last axis."""
    codes: torch.Tensor
    scales: torch.Tensor
    group: int

    @classmethod
    def empty(cls, shape, group: int, device="cuda") -> "Act8":
        import torch
        if group not in (64, 128):
            raise ValueError("group: expected 64 or 128")
        shape = tuple(shape)
        n = -(-shape[-1] // group)
        return cls(torch.empty(shape, dtype=torch.int8, device=device),
                   torch.empty(shape[:-1] + (n,), dtype=torch.float32, device=device), group)


def rope_dims(head_dim: int) -> tuple:
    """The usual split of a head's dimensions over (t, y, x): two of six parts
    of the pairs each for y and x, the rest for t (44, 42, 42 of 128)."""
    hw = 2 * (head_dim // 6)
    return head_dim - 2 * hw, hw, hw


_ENTRIES = ("vmoba_qk_norm_rope", "vmoba_qk_norm_rope_act8", "vmoba_qk_norm_rope_partition",
            "vmoba_qk_norm_rope_partition_act8", "vmoba_qk_norm_rope_bwd",
            "vmoba_qk_norm_rope_bwd_act8", "vmoba_act8_pack", "vmoba_act8_unpack")
_calls, _bound = None, False


def _bind() -> None:
    """Load the native calls and hand them the library's entries (at the first one)."""
    global _calls, _bound
    from .build import calls_path
    path = calls_path()
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with "
                           "`python -m block_sparse_attention_layer_b200.build`")
    loader = importlib.machinery.ExtensionFileLoader(__package__ + "._calls", path)
    spec = importlib.util.spec_from_file_location(loader.name, path, loader=loader)
    native = importlib.util.module_from_spec(spec)
    loader.exec_module(native)
    _calls, L = native, _lib.lib()
    native.bind({n: ctypes.cast(getattr(L, n), ctypes.c_void_p).value for n in _ENTRIES}, Act8)
    _bound = True


def rope_table(shape: LayerShape, dims, base: float = 10000.0, origin=(0, 0, 0), device="cuda",
               stream=None) -> torch.Tensor:
    """The rotation table of the shape's grid: (cos, sin) of each position and
    pair of the three axes, [T dims[0]/2 + H dims[1]/2 + W dims[2]/2][2] fp32,
    positions counted from ``origin`` (a chunk of a longer video)."""
    import torch
    t, h, w = (int(n) for n in dims)
    if min(t, h, w) < 0 or (t | h | w) & 1 or t + h + w > shape.head_dim:
        raise ValueError(f"dims: expected three even numbers >= 0 of sum <= {shape.head_dim}, "
                         f"got {dims}")
    table = torch.empty(((shape.T * t + shape.H * h + shape.W * w) // 2, 2), dtype=torch.float32,
                        device=device)
    if not table.is_cuda:
        raise ValueError("device: expected a CUDA device")
    with torch.cuda.device(table.device):
        _lib._check("vmoba_rope_table", _lib.lib().vmoba_rope_table(
            shape._ref, t, h, w, float(base), *(int(o) for o in origin), table.data_ptr(),
            _lib._stream(stream)))
    return table


def qk_norm_rope(shape, nr, qkv, q, k, v, ckpt=None, stream=None) -> None:
    """Norm of each head's query and key and their rotation, token order: raw
    rows -> q, k, v [s][heads][d] (v is copied).  qkv: the projection's output
    [s][3][heads][d] (tokens any stride apart), three [s][heads][d] tensors, or
    an Act8 checkpoint of it; ckpt: an Act8 to store the raw rows in (groups
    of head_dim), in the same pass."""
    native = shape._native
    rc = _calls.forward(native, nr, qkv, q, k, v, None, ckpt, stream)
    if rc:
        _lib._check("vmoba_qk_norm_rope", rc)


def qk_norm_rope_partition(shape, nr, qkv, q, k_perm, v_perm, blocks, ckpt=None,
                           stream=None) -> None:
    """As qk_norm_rope, into the sparse layer's buffers (in place of
    partition): q in token order, k_perm, v_perm in partition order and the
    fp32 means ``blocks`` of the rotated keys (before rounding to storage)."""
    if blocks is None:
        raise ValueError("blocks: expected a tensor")
    native = shape._native
    rc = _calls.forward(native, nr, qkv, q, k_perm, v_perm, blocks, ckpt, stream)
    if rc:
        _lib._check("vmoba_qk_norm_rope_partition", rc)


def qk_norm_rope_bwd_workspace_size(shape: LayerShape) -> int:
    return _lib.lib().vmoba_qk_norm_rope_bwd_workspace_size(shape._ref)


def qk_norm_rope_bwd(shape, nr, qkv, dq, dk, dv, dqkv, dweight, ws, stream=None) -> None:
    """Backward of qk_norm_rope and qk_norm_rope_partition: gradients of q, k, v
    (token order) -> of the raw rows (dqkv, laid out like qkv) and of the two
    norm weights (dweight [2][d] fp32, or None: then ws may be None too).  qkv:
    the forward's raw rows or their Act8 checkpoint."""
    native = shape._native
    rc = _calls.backward(native, nr, qkv, dq, dk, dv, dqkv, dweight, ws, stream)
    if rc:
        _lib._check("vmoba_qk_norm_rope_bwd", rc)


def act8_pack(x, ckpt, stream=None) -> None:
    """Store an activation in 8 bits: x (bf16 or fp32, [rows][cols] with rows
    any stride apart, or contiguous with more axes) into ``ckpt``."""
    if not _bound:
        _bind()
    rc = _calls.act8(True, x, ckpt, stream)
    if rc:
        _lib._check("vmoba_act8_pack", rc)


def act8_unpack(ckpt, out, stream=None) -> None:
    """Read an 8-bit checkpoint back into ``out`` (bf16 or fp32, laid out as
    act8_pack's x)."""
    if not _bound:
        _bind()
    rc = _calls.act8(False, out, ckpt, stream)
    if rc:
        _lib._check("vmoba_act8_unpack", rc)
