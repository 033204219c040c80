"""8-bit activation checkpoints: codes and scales bit for bit against the
plain form, and what they read back as."""
import numpy as np
import pytest

from . import norm_rope_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_sparse_attention_layer_b200 as V  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _roundtrip(x, group):
    ckpt = V.Act8.empty(tuple(x.shape), group)
    ckpt.codes.fill_(99)
    V.act8_pack(x, ckpt)
    out = torch.full(tuple(x.shape), 3.0, dtype=x.dtype, device="cuda")
    V.act8_unpack(ckpt, out)
    return ckpt, out


def _check(x, group):
    ckpt, out = _roundtrip(x, group)
    exact = x.double().cpu().numpy()
    codes, scales = R.encode8(exact, group)
    assert np.array_equal(ckpt.codes.cpu().numpy(), codes)
    assert np.array_equal(ckpt.scales.cpu().numpy(), scales, equal_nan=True)
    want = torch.from_numpy(R.decode8(codes, scales, group)).to(x.dtype)
    assert torch.equal(torch.nan_to_num(out.cpu(), nan=-5.0), torch.nan_to_num(want, nan=-5.0))
    return exact, out.double().cpu().numpy(), scales


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("group", [64, 128])
@pytest.mark.parametrize("rows,cols,pad", [
    (1, 1, 0), (1, 64, 0), (1, 129, 0), (3, 7, 0), (5, 200, 8), (17, 1003, 2), (33, 1536, 0),
    (64, 8, 0), (129, 96, 0), (2, 8192, 64), (1001, 72, 1)])
def test_codes_scales_and_values(dtype, group, rows, cols, pad):
    gen = torch.Generator(device="cuda").manual_seed(rows * cols + group)
    whole = torch.randn((rows, cols + pad), generator=gen, device="cuda") * \
        torch.exp(2 * torch.randn(cols + pad, generator=gen, device="cuda"))
    x = whole.to(DT[dtype])[:, :cols]
    exact, back, scales = _check(x, group)
    # half a code, the scale's rounding over 127 codes, the product's and the storage's
    s = np.repeat(scales.astype(np.float64), group, axis=-1)[:, :cols]
    assert (np.abs(back - exact) <= s * 0.5 * (1 + 2.0 ** -15) + R.STEP[dtype] * np.abs(back)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_rounding_borders(dtype):
    """Groups in which half of the quotients lie exactly between two codes
    (max |x| = 127 and 254 steps), next to one, or at half the largest."""
    rows = []
    for a in (127.0, 254.0, 1.0, 128.0, 190.0, 2.0 ** -20 * 127):
        v = np.zeros(128)
        v[0] = a
        v[1] = -a
        v[2] = a / 2
        n = np.arange(125)
        v[3:] = (n - 62 + 0.5) * a / 127 if dtype == "f32" else (n - 62 + 0.5) * (a / 128)
        rows.append(v)
    x = torch.tensor(np.array(rows)).to(DT[dtype])
    if dtype == "f32":       # neighbours of the borders too
        up = torch.nextafter(x, torch.full_like(x, np.inf))
        down = torch.nextafter(x, torch.full_like(x, -np.inf))
        x = torch.cat((x, up, down))
    _check(x.cuda(), 128)
    _check(x.cuda(), 64)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_extremes(dtype):
    """Zeros, the least and the largest magnitudes, infinities and NaN: each
    affects its own group only."""
    gen = torch.Generator(device="cuda").manual_seed(4)
    x = torch.randn((12, 256), generator=gen, device="cuda").to(DT[dtype])
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 200] = float("inf")
    x[3, 64] = -float("inf")
    x[4, :64] = 3e38 * torch.sign(x[4, :64].float()).to(x.dtype)
    x[5] *= 1e-37
    x[6] = 2.0 ** -119
    x[7] = 2.0 ** -120
    x[8] = 1e-40
    x[9, :] = 0.0
    x[9, 255] = 5.0
    x[10] = -1.0
    x[11, ::2] = torch.finfo(x.dtype).max
    for group in (64, 128):
        _check(x, group)
    ckpt, out = _roundtrip(x, 64)
    assert torch.isnan(out[1, :64]).all() and torch.isfinite(out[1, 64:]).all()
    assert torch.isnan(out[2, 192:]).all() and torch.isfinite(out[2, :192]).all()
    assert (out[7] == 0).all() and (out[6] != 0).all()
    assert torch.isfinite(out[11]).all()


def test_more_axes_no_rows_and_padding_kept():
    x = torch.randn((3, 5, 4, 128), device="cuda").to(torch.bfloat16)
    a, out = _roundtrip(x, 128)
    b, out2 = _roundtrip(x.view(60, 128), 128)
    assert torch.equal(a.codes.view(60, 128), b.codes) and torch.equal(out.view(60, 128), out2)
    empty = torch.empty((0, 64), device="cuda")
    n0 = V.kernel_launches()
    _roundtrip(empty, 64)
    assert V.kernel_launches() == n0
    ckpt, _ = _roundtrip(x.view(60, 128), 64)
    wide = torch.full((60, 160), 3.0, dtype=torch.bfloat16, device="cuda")
    V.act8_unpack(ckpt, wide[:, 8:136])
    assert (wide[:, :8] == 3.0).all() and (wide[:, 136:] == 3.0).all()
    odd = torch.full((60, 161), 3.0, dtype=torch.bfloat16, device="cuda")
    V.act8_unpack(ckpt, odd[:, 1:129])           # the unaligned form gives the same values
    assert torch.equal(odd[:, 1:129], wide[:, 8:136])
    assert (odd[:, 0] == 3.0).all() and (odd[:, 129:] == 3.0).all()


def test_side_stream_and_graph():
    x = torch.randn((300, 1536), device="cuda").to(torch.bfloat16)
    want, out_want = _roundtrip(x, 128)
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        got, out = _roundtrip(x, 128)
    torch.cuda.synchronize()
    assert torch.equal(got.codes, want.codes) and torch.equal(out, out_want)
    ckpt, out = V.Act8.empty((300, 1536), 128), torch.zeros_like(x)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        V.act8_pack(x, ckpt)
        V.act8_unpack(ckpt, out)
    x.mul_(-3.0)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, _roundtrip(x, 128)[1])


def test_offsets_beyond_32_bits():
    """More than 2^32 values: the last rows are those of a call on them alone."""
    rows, cols = 2 ** 22 + 3, 1032
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    part = torch.randn((2 ** 16, cols), device="cuda").to(torch.bfloat16)
    for i in range(0, rows, 2 ** 16):
        x[i:i + 2 ** 16] = (part * (1 + i))[:rows - i]
    ckpt = V.Act8.empty((rows, cols), 128)
    V.act8_pack(x, ckpt)
    tail = V.Act8.empty((1000, cols), 128)
    V.act8_pack(x[-1000:], tail)
    assert torch.equal(ckpt.codes[-1000:], tail.codes)
    assert torch.equal(ckpt.scales[-1000:], tail.scales)
    out = torch.empty((1000, cols), dtype=x.dtype, device="cuda")
    V.act8_unpack(tail, out)
    V.act8_unpack(ckpt, x)
    assert torch.equal(x[-1000:], out)


@pytest.mark.parametrize("cols", [2 ** 31 - 128, 2 ** 31 - 8, 2 ** 31 - 1])
@pytest.mark.parametrize("group", [64, 128])
def test_widest_rows(cols, group):
    """One row of nearly 2^31 values: its whole groups are those of the same
    values as rows of one group, the short last one the plain form's."""
    x = torch.empty((1, cols), dtype=torch.bfloat16, device="cuda")
    part = torch.randn(2 ** 24 + 1, device="cuda").to(torch.bfloat16)
    for i in range(0, cols, part.numel()):
        x[0, i:i + part.numel()] = (part * (1 + i // part.numel()))[:cols - i]
    ckpt = V.Act8.empty((1, cols), group)
    V.act8_pack(x, ckpt)
    whole = cols // group * group
    rows = V.Act8.empty((whole // group, group), group)
    V.act8_pack(x[0, :whole].view(-1, group), rows)
    assert torch.equal(ckpt.codes[0, :whole], rows.codes.view(-1))
    assert torch.equal(ckpt.scales[0, :whole // group], rows.scales.view(-1))
    last = x[:, -1000:].double().cpu().numpy()[:, -(cols - whole):] if cols > whole else None
    out = torch.empty_like(x)
    V.act8_unpack(ckpt, out)
    del x
    want = torch.empty((whole // group, group), dtype=out.dtype, device="cuda")
    V.act8_unpack(rows, want)
    assert torch.equal(out[0, :whole], want.view(-1))
    if last is not None:
        codes, scales = R.encode8(last, group)
        assert np.array_equal(ckpt.codes[:, whole:].cpu().numpy(), codes)
        assert np.array_equal(ckpt.scales[:, -1:].cpu().numpy(), scales)
        back = torch.from_numpy(R.decode8(codes, scales, group)).to(out.dtype)
        assert torch.equal(out[:, whole:].cpu(), back)


def _bf16_pairs():
    """(values [n][64] bf16, codes) of groups whose largest value has each of
    the 128 bf16 significands, at some exponents, and whose others run over
    every significand at every exponent down to a code of zero, both signs:
    the code is round-half-even of 127 x / a, in whole numbers."""
    m = np.arange(128, 256)
    x, e = np.meshgrid(m, np.arange(10), indexing="ij")
    x, e = (np.concatenate((t.ravel(), t.ravel())) for t in (x, e))
    sign = np.where(np.arange(x.size) < x.size // 2, 1, -1)
    groups, codes = [], []
    for a in m:
        keep = (x <= a) | (e > 0)                        # |x| <= a 2^e / 2^e
        num, den = 127 * x[keep], a << e[keep]           # 127 |x| / a, exactly
        c, rest = num // den, 2 * (num % den)
        c = c + ((rest > den) | ((rest == den) & (c % 2 == 1)))
        v, c = sign[keep] * x[keep] * 2.0 ** -e[keep], sign[keep] * c
        pad = -v.size % 63
        v, c = np.pad(v, (0, pad)).reshape(-1, 63), np.pad(c, (0, pad)).reshape(-1, 63)
        groups.append(np.insert(v, 0, a, 1))
        codes.append(np.insert(c, 0, 127, 1))
    return np.concatenate(groups), np.concatenate(codes)


def test_every_pair_of_bf16_significands():
    """The one rounding that a bf16 group's codes go through is the exact
    quotient's, for every value against every largest one."""
    values, codes = _bf16_pairs()
    for shift in (-100, -7, 0, 60, 92, 110):
        x = torch.from_numpy(values * 2.0 ** shift).to(torch.bfloat16)
        assert torch.equal(x.double(), torch.from_numpy(values * 2.0 ** shift))
        ckpt = V.Act8.empty(tuple(x.shape), 64)
        V.act8_pack(x.cuda(), ckpt)
        assert np.array_equal(ckpt.codes.cpu().numpy(), codes)


def test_every_fp32_scale():
    """a / 127 is correctly rounded for every significand of a: the host's
    division is, and no exponent changes it while the results are normal."""
    for shift in (-110, 0, 100):
        for first in range(1 << 23, 1 << 24, 1 << 21):
            a = torch.arange(first, first + (1 << 21), dtype=torch.float64) * 2.0 ** (shift - 23)
            a = a.float()
            x = torch.zeros((a.numel(), 64), device="cuda")
            x[:, 5] = -a.cuda()
            ckpt = V.Act8.empty(tuple(x.shape), 64)
            V.act8_pack(x, ckpt)
            want = torch.from_numpy(a.numpy() / np.float32(127.0))
            assert torch.equal(ckpt.scales[:, 0].cpu(), want)
            assert (ckpt.codes[:, 5] == -127).all()
