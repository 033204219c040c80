"""Plain fp64 numpy forms of the operators around the attention (norm +
rotation, its gradients, 8-bit checkpoints), and the error bounds that the
kernels' fp32 arithmetic is held to.  U = 2^-24 is the relative error of one
fp32 operation."""
from __future__ import annotations

import numpy as np

U = 2.0 ** -24
STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}      # half a step of the storage type, relative
# Below the least normal number 2^-126 a half step is absolute: 2^-134 for bf16
# (7 fraction bits), 2^-150 for fp32, and each of the at most 16 fp32
# operations behind a result adds 2^-150.
TINY = {"bf16": 2.0 ** -134 + 2.0 ** -146, "f32": 2.0 ** -145}


def table(T, H, W, dims, base=10000.0, origin=(0, 0, 0)):
    """(cos, sin) entries in fp64, axis after axis."""
    parts = []
    for n, dim, o in zip((T, H, W), dims, origin):
        a = (np.arange(n, dtype=np.float64)[:, None] + o) * \
            np.float64(base) ** (-2.0 * np.arange(dim // 2) / max(dim, 1))[None, :]
        parts.append(np.stack((np.cos(a), np.sin(a)), -1).reshape(-1, 2))
    return np.concatenate(parts)


def phases(T, H, W, d, dims, tab):
    """[s][d/2] complex factors of every token's pairs."""
    out = np.ones((T, H, W, d // 2), dtype=np.complex128)
    col = at = 0
    for axis, (n, dim) in enumerate(zip((T, H, W), dims)):
        p = dim // 2
        rows = (tab[at:at + n * p, 0] + 1j * tab[at:at + n * p, 1]).reshape(n, p)
        shape = [1, 1, 1, p]
        shape[axis] = n
        out[..., col:col + p] = rows.reshape(shape)
        col, at = col + p, at + n * p
    return out.reshape(T * H * W, d // 2)


def rotate(y, z):
    """[s][h][d] rows turned by z [s][d/2]."""
    c = y[..., 0::2] + 1j * y[..., 1::2]
    c = c * z[:, None, :]
    return np.stack((c.real, c.imag), -1).reshape(y.shape)


def pair_abs(y):
    """|y0| + |y1| of the pair each element belongs to."""
    a = np.abs(y[..., 0::2]) + np.abs(y[..., 1::2])
    return np.repeat(a, 2, axis=-1)


def forward(x, g, eps, z):
    """(rotated rows, bound of a kernel's error before storage).

    fp32: the sum of squares of d <= 128 values is added over eight terms and
    four halvings (12 U), halved by the root (6 U) with rsqrt's own 2 ulp (4 U):
    10 U; two products for x r g (2 U); two products and a sum per rotated
    value (3 U of |y0| + |y1|): 15 U, and second-order terms."""
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = x * r if g is None else x * r * g
    return rotate(y, z), 16 * U * pair_abs(y)


def backward(x, g, eps, z, dy):
    """(dx, bound, dg, bound).

    u is two products and a sum (3 U of its pair's |d|); x r is 11 U; the
    mean of w x r adds eight terms and four halvings: (3 + 1 + 11 + 1 + 12) U
    of the mean of absolute products; dx adds two operations and r's 10 U:
    under 48 U of r (|w| + |xh| mean|w xh|).  dg: each term 15 U, fp32 sums of
    at most 64 rows a lane, the CTAs' fp64 totals rounded once: under 96 U of
    the sum of absolute terms."""
    d = x.shape[-1]
    r = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    xh = x * r
    u = rotate(dy, np.conj(z))
    w = u if g is None else u * g
    dx = r * (w - xh * (w * xh).mean(-1, keepdims=True))
    pu = pair_abs(dy)
    pw = pu if g is None else pu * np.abs(g)
    bound = 48 * U * r * (pw + np.abs(xh) * (pw * np.abs(xh)).mean(-1, keepdims=True))
    dg = (u * xh).reshape(-1, d).sum(0)
    return dx, bound, dg, 96 * U * (pu * np.abs(xh)).reshape(-1, d).sum(0)


def encode8(x, group):
    """Codes (int) and fp32 scales of x [..., cols] (exactly representable in
    fp32).  127 x / a in fp64 has the exact quotient's rounding: a tie is
    representable, and any other quotient is at least 2^-25 relative from one."""
    cols = x.shape[-1]
    n = -(-cols // group)
    pad = np.zeros(x.shape[:-1] + (n * group,))
    pad[..., :cols] = x
    pad = pad.reshape(x.shape[:-1] + (n, group))
    a = np.abs(pad).max(-1)
    bad = ~np.isfinite(pad).all(-1)
    small = a < 2.0 ** -119
    use = np.where(bad | small, 1.0, a)
    codes = np.rint(np.where((bad | small)[..., None], 0.0, 127.0 * pad) / use[..., None])
    scales = (use.astype(np.float32) / np.float32(127.0)).astype(np.float32)
    with np.errstate(over="ignore"):       # 127 scale must not read back as infinite
        over = np.isinf(scales * np.float32(127.0))
    scales[over] = np.nextafter(scales[over], np.float32(0.0))
    scales[small] = 0.0
    scales[bad] = np.nan
    return codes.reshape(x.shape[:-1] + (n * group,))[..., :cols].astype(np.int8), scales


def decode8(codes, scales, group):
    """code * scale with its one fp32 rounding, as fp64."""
    cols = codes.shape[-1]
    s = np.repeat(scales, group, axis=-1)[..., :cols]
    return (codes.astype(np.float32) * s).astype(np.float64)
