"""What stands around the attention of a layer: the norm of each head's queries
and keys with their (t, y, x) rotation, forward and backward, and activation
checkpoints in 8 bits (include/vmoba.h: vmoba_norm_rope, vmoba_act8_pack).

Binding only, as _lib: arguments are checked and passed on, every step runs in
libvmoba's kernels on the caller's buffers.  A call's tensors lie on one CUDA
device, which is made current during the call.
"""
from __future__ import annotations

import ctypes
from dataclasses import dataclass

import torch

from . import _lib
from ._lib import CNormRope, LayerShape

_F32, _I8, _BF16 = torch.float32, torch.int8, torch.bfloat16


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
        if group not in (64, 128):
            raise ValueError("group: expected 64 or 128")
        shape = tuple(shape)
        n = -(-shape[-1] // group)
        return cls(torch.empty(shape, dtype=_I8, device=device),
                   torch.empty(shape[:-1] + (n,), dtype=_F32, device=device), group)


def rope_dims(head_dim: int) -> tuple:
    """The usual split of a head's dimensions over (t, y, x): two of six parts
    of the pairs each for y and x, the rest for t (44, 42, 42 of 128)."""
    hw = 2 * (head_dim // 6)
    return head_dim - 2 * hw, hw, hw


# ---------------------------------------------------------------- checks

def _device(t, name) -> int:
    d = t.get_device()
    if d < 0:
        raise ValueError(f"{name}: expected a CUDA tensor")
    return d


def _at(t, size, dtype, device, name) -> int:
    """Address of a contiguous tensor of the call."""
    if t.shape == size and t.dtype is dtype and t.get_device() == device and t.is_contiguous():
        return t.data_ptr()
    _layout(t, size, dtype, device, name)
    raise ValueError(f"{name}: expected a contiguous tensor")


def _layout(t, size, dtype, device, name) -> None:
    if t.shape != size:
        raise ValueError(f"{name}: expected shape {tuple(size)}, got {tuple(t.shape)}")
    if t.dtype is not dtype:
        raise ValueError(f"{name}: expected dtype {dtype}, got {t.dtype}")
    if _device(t, name) != device:
        raise ValueError(f"{name}: expected a tensor on cuda:{device}, got {t.device}")


def _stride(t, least, dense, name) -> int:
    """The token stride of rows whose other axes are dense."""
    st = t.stride()
    if st[0] >= least and st[1:] == dense and t.shape[0] != 1:
        return st[0]
    if st[1:] != dense and any(n > 1 and have != want
                               for n, have, want in zip(t.shape[1:], st[1:], dense)):
        raise ValueError(f"{name}: expected dense rows, got strides {tuple(st)}")
    if t.shape[0] == 1:
        return least
    if st[0] < least:
        raise ValueError(f"{name}: rows overlap, strides {tuple(st)}")
    return st[0]


def _raw(shape: LayerShape, x, device, name):
    """(q, k, v addresses, token stride) of raw rows: a [s][3][heads][d] tensor
    or three [s][heads][d] ones, the last two axes dense."""
    token, _, raw, _, dtype = shape._sizes
    d, row = token[2], token[1] * token[2]
    if isinstance(x, (tuple, list)):
        if len(x) != 3:
            raise ValueError(f"{name}: expected one tensor or three")
        for t in x:
            _layout(t, token, dtype, device, name)
        ld = _stride(x[0], row, (d, 1), name)
        if _stride(x[1], row, (d, 1), name) != ld or _stride(x[2], row, (d, 1), name) != ld:
            raise ValueError(f"{name}: expected one token stride, got "
                             f"{[t.stride(0) for t in x]}")
        return x[0].data_ptr(), x[1].data_ptr(), x[2].data_ptr(), ld
    if x.shape != raw or x.dtype is not dtype or x.get_device() != device:
        _layout(x, raw, dtype, device, name)
    p, step = x.data_ptr(), row * dtype.itemsize
    return p, p + step, p + 2 * step, _stride(x, 3 * row, (row, d, 1), name)


def _first(x):
    """The tensor whose device a call runs on."""
    if isinstance(x, Act8):
        return x.codes
    return x[0] if isinstance(x, (tuple, list)) and x else x


def _ckpt(c: Act8, size, group, device, name):
    if c.group != group:
        raise ValueError(f"{name}: expected groups of {group}, got {c.group}")
    return (_at(c.codes, size, _I8, device, name + ".codes"),
            _at(c.scales, (*size[:-1], -(-size[-1] // group)), _F32, device, name + ".scales"))


def _dims(shape: LayerShape, dims) -> tuple:
    """(dims, table rows), checked."""
    ok = isinstance(dims, (tuple, list)) and len(dims) == 3 and \
        all(isinstance(n, int) for n in dims)
    if not ok or min(dims) < 0 or any(n & 1 for n in dims) or sum(dims) > shape.head_dim:
        raise ValueError(f"dims: expected three even numbers >= 0 of sum <= {shape.head_dim}, "
                         f"got {dims}")
    t, h, w = dims
    return t, h, w, (shape.T * t + shape.H * h + shape.W * w) // 2


def _norm(shape: LayerShape, nr: NormRope, device):
    """The norm and rotation as the ABI takes them.  nr's tensors are checked
    when they are first used with the shape, and again once one's memory has
    moved; what they hold is read by each call's kernels."""
    gq, gk, table = nr.q_weight, nr.k_weight, nr.table
    at = (shape, device, gq if gq is None else gq.data_ptr(), gk if gk is None else gk.data_ptr(),
          table if table is None else table.data_ptr())
    made = nr.__dict__.get("_made")
    if made is not None and made[0] == at:
        return made[1]
    t, h, w, rows = _dims(shape, nr.dims)
    d = (shape.head_dim,)
    g = [0 if x is None else _at(x, d, _F32, device, name)
         for name, x in (("q_weight", gq), ("k_weight", gk))]
    if rows and table is None:
        raise ValueError("table: expected a rotation table (rope_table)")
    c = ctypes.byref(CNormRope(*g, nr.eps, _at(table, (rows, 2), _F32, device, "table")
                               if rows else 0, t, h, w))
    nr.__dict__["_made"] = at, c
    return c


def _stream(device, stream) -> int:
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device)
    if stream.device.index != device:
        raise ValueError(f"stream: expected one of cuda:{device}, got {stream.device}")
    return stream.cuda_stream


def _run(name, device, *args) -> None:
    fn = getattr(_lib._LIB or _lib.lib(), name)
    if device == torch._C._cuda_getDevice():
        rc = fn(*args)
    else:
        with torch.cuda.device(device):
            rc = fn(*args)
    if rc:
        _lib._check(name, rc)


# ---------------------------------------------------------------- calls

def rope_table(shape: LayerShape, dims, base: float = 10000.0, origin=(0, 0, 0), device="cuda",
               stream=None) -> torch.Tensor:
    """The rotation table of the shape's grid: (cos, sin) of each position and
    pair of the three axes, [T dims[0]/2 + H dims[1]/2 + W dims[2]/2][2] fp32,
    positions counted from ``origin`` (a chunk of a longer video)."""
    t, h, w, rows = _dims(shape, dims)
    table = torch.empty((rows, 2), dtype=_F32, device=device)
    on = _device(table, "table")
    _run("vmoba_rope_table", on, shape._ref, t, h, w, float(base), *(int(o) for o in origin),
         table.data_ptr(), _stream(on, stream))
    return table


def _source(shape, qkv, ckpt, device):
    """The forward's leading arguments and the checkpoint's trailing ones."""
    if isinstance(qkv, Act8):
        if ckpt is not None:
            raise ValueError("ckpt: the raw values already come from a checkpoint")
        return _ckpt(qkv, shape._sizes[2], shape.head_dim, device, "qkv"), ()
    if ckpt is None:
        return _raw(shape, qkv, device, "qkv"), (0, 0)
    return (_raw(shape, qkv, device, "qkv"),
            _ckpt(ckpt, shape._sizes[2], shape.head_dim, device, "ckpt"))


def qk_norm_rope(shape, nr, qkv, q, k, v, ckpt=None, stream=None) -> None:
    """Norm of each head's query and key and their rotation, token order: raw
    rows -> q, k, v [s][heads][d] (v is copied).  qkv: the projection's output
    [s][3][heads][d] (tokens any stride apart), three [s][heads][d] tensors, or
    an Act8 checkpoint of it; ckpt: an Act8 to store the raw rows in (groups
    of head_dim), in the same pass."""
    token, _, _, _, dtype = shape._sizes
    device = _device(q, "q")
    src, more = _source(shape, qkv, ckpt, device)
    _run("vmoba_qk_norm_rope" if more else "vmoba_qk_norm_rope_act8", device, shape._ref,
         _norm(shape, nr, device), *src, _at(q, token, dtype, device, "q"),
         _at(k, token, dtype, device, "k"), _at(v, token, dtype, device, "v"), *more,
         _stream(device, stream))


def qk_norm_rope_partition(shape, nr, qkv, q, k_perm, v_perm, blocks, ckpt=None,
                           stream=None) -> None:
    """As qk_norm_rope, into the sparse layer's buffers (in place of
    partition): q in token order, k_perm, v_perm in partition order and the
    fp32 means ``blocks`` of the rotated keys (before rounding to storage)."""
    token, head, _, means, dtype = shape._sizes
    device = _device(q, "q")
    src, more = _source(shape, qkv, ckpt, device)
    _run("vmoba_qk_norm_rope_partition" if more else "vmoba_qk_norm_rope_partition_act8", device,
         shape._ref, _norm(shape, nr, device), *src, _at(q, token, dtype, device, "q"),
         _at(k_perm, head, dtype, device, "k_perm"), _at(v_perm, head, dtype, device, "v_perm"),
         _at(blocks, means, _F32, device, "blocks"), *more, _stream(device, stream))


def qk_norm_rope_bwd_workspace_size(shape: LayerShape) -> int:
    return _lib.lib().vmoba_qk_norm_rope_bwd_workspace_size(shape._ref)


def qk_norm_rope_bwd(shape, nr, qkv, dq, dk, dv, dqkv, dweight, ws, stream=None) -> None:
    """Backward of qk_norm_rope and qk_norm_rope_partition: gradients of q, k, v
    (token order) -> of the raw rows (dqkv, laid out like qkv) and of the two
    norm weights (dweight [2][d] fp32, or None: then ws may be None too).  qkv:
    the forward's raw rows or their Act8 checkpoint."""
    token, _, raw, _, dtype = shape._sizes
    device = _device(dq, "dq")
    if isinstance(qkv, Act8):
        name = "vmoba_qk_norm_rope_bwd_act8"
        src = _ckpt(qkv, raw, token[2], device, "qkv")
    else:
        name = "vmoba_qk_norm_rope_bwd"
        q, k, _, ld = _raw(shape, qkv, device, "qkv")
        src = q, k, ld
    dw = p_ws = n_ws = 0
    if dweight is not None:
        dw = _at(dweight, (2, token[2]), _F32, device, "dweight")
        p_ws, n_ws = _at(ws, ws.shape, ws.dtype, device, "ws"), ws.nbytes
    _run(name, device, shape._ref, _norm(shape, nr, device), *src,
         _at(dq, token, dtype, device, "dq"), _at(dk, token, dtype, device, "dk"),
         _at(dv, token, dtype, device, "dv"), *_raw(shape, dqkv, device, "dqkv"), dw, p_ws, n_ws,
         _stream(device, stream))


def _rows(x, name):
    """(dtype code, rows, cols, row stride) of a tensor whose leading axes are
    rows."""
    if x.dtype is _BF16:
        code = _lib.VMOBA_BF16
    elif x.dtype is _F32:
        code = _lib.VMOBA_F32
    else:
        raise ValueError(f"{name}: expected dtype bfloat16 or float32, got {x.dtype}")
    size = x.shape
    if len(size) < 2:
        raise ValueError(f"{name}: expected at least two axes")
    cols = size[-1]
    if x.is_contiguous():
        return code, x.numel() // cols if cols else 0, cols, cols
    row, step = x.stride() if len(size) == 2 else (0, 0)
    if (cols > 1 and step != 1) or (size[0] > 1 and row < cols):
        raise ValueError(f"{name}: expected dense rows, got strides {tuple(x.stride())}")
    return code, size[0], cols, row if size[0] > 1 else cols


def act8_pack(x, ckpt, stream=None) -> None:
    """Store an activation in 8 bits: x (bf16 or fp32, [rows][cols] with rows
    any stride apart, or contiguous with more axes) into ``ckpt``."""
    code, rows, cols, ld = _rows(x, "x")
    device = _device(x, "x")
    codes, scales = _ckpt(ckpt, x.shape, ckpt.group, device, "ckpt")
    _run("vmoba_act8_pack", device, code, x.data_ptr(), rows, cols, ld, ckpt.group, codes, scales,
         _stream(device, stream))


def act8_unpack(ckpt, out, stream=None) -> None:
    """Read an 8-bit checkpoint back into ``out`` (bf16 or fp32, laid out as
    act8_pack's x)."""
    code, rows, cols, ld = _rows(out, "out")
    device = _device(out, "out")
    codes, scales = _ckpt(ckpt, out.shape, ckpt.group, device, "ckpt")
    _run("vmoba_act8_unpack", device, code, codes, scales, rows, cols, ckpt.group, out.data_ptr(),
         ld, _stream(device, stream))
