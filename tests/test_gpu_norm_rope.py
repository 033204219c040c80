"""Norm + rotation of queries and keys (forward in token and partition order,
backward) against plain fp64 forms, on values, odd sizes, strides, extreme
inputs, checkpoints, streams and graphs.  Bounds: norm_rope_ref."""
import weakref

import numpy as np
import pytest

import oracle as O

from . import norm_rope_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_sparse_attention_layer_b200 as V  # noqa: E402

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS = 1e-6


class Case:
    """One problem: tensors on the device and their exact values in fp64."""

    def __init__(self, grid, h, d, dtype, mode=2, box=None, dims=None, weights=True,
                 layout="packed", seed=0, scale=1.0, origin=(0, 0, 0), eps=EPS):
        T, H, W = grid
        box = box or grid
        self.sh = V.LayerShape(T, H, W, h, d, mode, *box, dtype)
        self.s, self.h, self.d, self.dtype, self.dt, self.eps = T * H * W, h, d, dtype, DT[dtype], eps
        self.dims = V.rope_dims(d) if dims is None else dims
        gen = torch.Generator(device="cuda").manual_seed(seed)
        s, shape = self.s, (self.s, 3, h, d)
        val = torch.randn(shape, generator=gen, device="cuda") * scale * \
            torch.exp(torch.randn(shape[1:], generator=gen, device="cuda"))
        self.layout = layout
        self.whole, self.qkv = self.buffer()
        self.fill(val.to(self.dt))
        self.gq = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if weights else None
        self.gk = 1 + 0.2 * torch.randn(d, generator=gen, device="cuda") if weights else None
        self.table = V.rope_table(self.sh, self.dims, origin=origin)
        self.nr = V.NormRope(self.gq, self.gk, eps, self.table, self.dims)
        self.z = R.phases(T, H, W, d, self.dims, self.table.double().cpu().numpy())
        self.grads = [torch.randn((s, h, d), generator=gen, device="cuda").to(self.dt)
                      for _ in range(3)]
        self.box = O.mode_box(mode, T, H, W, *box)

    def buffer(self):
        """(allocation, raw rows) in the case's layout."""
        s, h, d = self.s, self.h, self.d
        if self.layout == "separate":
            t = torch.zeros((3, s, h, d), dtype=self.dt, device="cuda")
            return t, (t[0], t[1], t[2])
        pad = 8 if self.layout == "padded" else 0
        t = torch.full((s, 3 * h * d + pad), 7.0, dtype=self.dt, device="cuda")
        return t, t.as_strided((s, 3, h, d), (3 * h * d + pad, h * d, d, 1))

    def parts(self, qkv=None):
        qkv = self.qkv if qkv is None else qkv
        return list(qkv) if isinstance(qkv, tuple) else [qkv[:, i] for i in range(3)]

    def fill(self, val):
        for i, p in enumerate(self.parts()):
            p.copy_(val[:, i])
        self.x = [p.double().cpu().numpy() for p in self.parts()]

    def g(self, i):
        w = (self.gq, self.gk)[i]
        return None if w is None else w.double().cpu().numpy()

    def token(self):
        return torch.full((self.s, self.h, self.d), 9.0, dtype=self.dt, device="cuda")

    def head(self):
        return torch.full((self.h, self.s, self.d), 9.0, dtype=self.dt, device="cuda")

    def means(self):
        return torch.full((self.h, V.num_blocks(self.sh), self.d), 9.0, device="cuda")

    def order(self):
        return O.partition_order(self.sh.T, self.sh.H, self.sh.W, self.box)

    def forward(self, src=None, ckpt=None):
        out = [self.token(), self.token(), self.token()]
        V.qk_norm_rope(self.sh, self.nr, self.qkv if src is None else src, *out, ckpt=ckpt)
        return out

    def partition(self, src=None, ckpt=None):
        out = [self.token(), self.head(), self.head(), self.means()]
        V.qk_norm_rope_partition(self.sh, self.nr, self.qkv if src is None else src, *out,
                                 ckpt=ckpt)
        return out

    def backward(self, src=None, weights=True):
        whole, raw = self.buffer()
        dw = torch.full((2, self.d), 9.0, device="cuda") if weights else None
        ws = torch.full((V.qk_norm_rope_bwd_workspace_size(self.sh),), 0x7F, dtype=torch.uint8,
                        device="cuda") if weights else None
        V.qk_norm_rope_bwd(self.sh, self.nr, self.qkv if src is None else src, *self.grads, raw, dw,
                           ws)
        return whole, self.parts(raw), dw

    def empty_ckpt(self):
        return V.Act8.empty((self.s, 3, self.h, self.d), self.d)

    def close(self, got, want, bound):
        got = got.double().cpu().numpy()
        assert got.shape == want.shape
        err = np.abs(got - want) - R.STEP[self.dtype] * np.abs(want) - R.TINY[self.dtype] - bound
        assert err.max() <= 0, f"beyond the bound by {err.max()}"

    def check_forward(self, got, x=None):
        x = self.x if x is None else x
        (q, bq), (k, bk) = (R.forward(x[i], self.g(i), self.eps, self.z) for i in range(2))
        self.close(got[0], q, bq)
        self.close(got[1], k, bk)

    def check_partition(self, got, x=None):
        x = self.x if x is None else x
        (q, bq), (k, bk) = (R.forward(x[i], self.g(i), self.eps, self.z) for i in range(2))
        o = self.order()
        self.close(got[0], q, bq)
        kp, bp = k[o].transpose(1, 0, 2), bk[o].transpose(1, 0, 2)
        self.close(got[1], kp, bp)
        nb = got[3].shape[1]
        cut = lambda a: a.reshape(self.h, nb, self.s // nb, self.d)     # noqa: E731
        # the rows' own bound, fp32 sums over at most 64 rows (64 U of the mean
        # |k|), and the division and rounding of the result
        mean = cut(kp).mean(2)
        bound = cut(bp).mean(2) + 64 * R.U * np.abs(cut(kp)).mean(2) + 2 * R.U * np.abs(mean)
        err = np.abs(got[3].double().cpu().numpy() - mean) - bound
        assert err.max() <= 0, f"block means beyond the bound by {err.max()}"

    def check_backward(self, parts, dw, x=None):
        x = self.x if x is None else x
        for i in range(2):
            dy = self.grads[i].double().cpu().numpy()
            dx, b, dg, bg = R.backward(x[i], self.g(i), self.eps, self.z, dy)
            self.close(parts[i], dx, b)
            if dw is not None:
                assert (np.abs(dw[i].double().cpu().numpy() - dg) <= bg + R.U * np.abs(dg)).all()
        assert torch.equal(parts[2], self.grads[2])


CASES = {
    "one token": dict(grid=(1, 1, 1), h=1, d=64, dtype="bf16"),
    "one token, 40 heads": dict(grid=(1, 1, 1), h=40, d=128, dtype="bf16", origin=(70000, 0, 3)),
    "three tokens f32": dict(grid=(1, 1, 3), h=2, d=64, dtype="f32", layout="padded"),
    "17 tokens": dict(grid=(1, 1, 17), h=3, d=128, dtype="bf16", layout="separate"),
    "odd grid": dict(grid=(7, 9, 11), h=5, d=64, dtype="bf16", box=(7, 3, 11), mode=2),
    "odd grid f32": dict(grid=(3, 5, 7), h=3, d=128, dtype="f32", box=(1, 5, 1), mode=2,
                         layout="padded", dims=(2, 126, 0)),
    "blocks of one token": dict(grid=(2, 3, 5), h=2, d=128, dtype="bf16", box=(1, 1, 1)),
    "temporal blocks": dict(grid=(6, 5, 13), h=12, d=128, dtype="bf16", box=(2, 1, 1), mode=0),
    "spatial blocks f32": dict(grid=(5, 6, 8), h=4, d=64, dtype="f32", box=(1, 3, 4), mode=1,
                               layout="separate", weights=False),
    "no rotation": dict(grid=(2, 4, 8), h=2, d=128, dtype="bf16", dims=(0, 0, 0)),
    "partial rotation": dict(grid=(4, 4, 4), h=8, d=128, dtype="bf16", dims=(16, 0, 34),
                             box=(2, 2, 2), weights=False, layout="padded"),
    "long block": dict(grid=(2, 40, 60), h=1, d=64, dtype="bf16", box=(2, 40, 60)),
    "2048 tokens": dict(grid=(8, 16, 16), h=4, d=64, dtype="bf16", box=(2, 4, 4)),
    "huge rows and eps": dict(grid=(2, 4, 4), h=2, d=64, dtype="f32", eps=1e33, scale=1e16),
    "large eps": dict(grid=(2, 4, 4), h=2, d=64, dtype="f32", eps=10.0),
}


@pytest.fixture(params=sorted(CASES))
def case(request):
    return Case(**CASES[request.param], seed=sorted(CASES).index(request.param))


def test_table_is_the_angles(case):
    sh = case.sh
    for dims, base, origin in ((case.dims, 10000.0, (0, 0, 0)), ((2, 4, 6), 256.0, (-9, 2 ** 31, 7)),
                               ((0, 64, 0), 1e6, (0, 123456789, 0))):
        got = V.rope_table(sh, dims, base, origin).double().cpu().numpy()
        want = R.table(sh.T, sh.H, sh.W, dims, base, origin)
        assert got.shape == want.shape
        # the fp64 angle is off by a few of its own 2^-53 (power, division and
        # product on either side: 8 are allowed), then one fp32 rounding
        largest = max(abs(o) + n for o, n in zip(origin, (sh.T, sh.H, sh.W)))
        assert np.abs(got - want).max(initial=0.0) <= R.U + 8 * 2.0 ** -53 * max(largest, 1)


def test_forward_token_order(case):
    got = case.forward()
    case.check_forward(got)
    assert torch.equal(got[2], case.parts()[2])


def test_forward_into_partition(case):
    got = case.partition()
    case.check_partition(got)
    o = torch.from_numpy(case.order()).cuda()
    assert torch.equal(got[2], case.parts()[2][o].transpose(0, 1))
    # the same rotated keys, whichever way they leave
    q, k, _ = case.forward()
    assert torch.equal(got[0], q) and torch.equal(got[1], k[o].transpose(0, 1))


def test_backward(case):
    whole, parts, dw = case.backward()
    case.check_backward(parts, dw)
    if case.layout == "padded":        # nothing is written between the rows
        assert (whole[:, 3 * case.h * case.d:] == 7.0).all()
    again = case.backward(weights=False)[1]
    assert all(torch.equal(a, b) for a, b in zip(parts, again))
    assert torch.equal(case.backward()[2], dw)       # a fixed order of sums


def test_checkpoint_written_and_used(case):
    ckpt = case.empty_ckpt()
    plain = case.forward()
    assert all(torch.equal(a, b) for a, b in zip(plain, case.forward(ckpt=ckpt)))
    want = [R.encode8(x, case.d) for x in case.x]
    for i, (codes, scales) in enumerate(want):
        assert np.array_equal(ckpt.codes[:, i].cpu().numpy(), codes)
        assert np.array_equal(ckpt.scales[:, i].cpu().numpy(), scales)
    ckpt2 = case.empty_ckpt()
    part = case.partition()
    assert all(torch.equal(a, b) for a, b in zip(part, case.partition(ckpt=ckpt2)))
    assert torch.equal(ckpt.codes, ckpt2.codes) and torch.equal(ckpt.scales, ckpt2.scales)
    x8 = [R.decode8(c, s, case.d) for c, s in want]
    v8 = torch.from_numpy(x8[2]).to(case.dt).cuda()
    got = case.forward(ckpt)
    case.check_forward(got, x8)
    assert torch.equal(got[2], v8)
    got = case.partition(ckpt)
    case.check_partition(got, x8)
    assert torch.equal(got[2], v8[torch.from_numpy(case.order()).cuda()].transpose(0, 1))
    _, parts, dw = case.backward(ckpt)
    case.check_backward(parts, dw, x8)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_large_and_small_rows(dtype):
    """Squares beyond fp32's range, rows far below eps, and zero rows."""
    c = Case((2, 3, 4), 2, 128, dtype, dims=(44, 42, 42), seed=5)
    val = torch.stack([p.float() for p in c.parts()], 1)
    # lifts the row's largest to about 3e38 and 1e30, lowers others to 1e-30, 0
    top = val.abs().amax(-1, keepdim=True)
    for n, size in ((3, 3e38), (4, 1e30), (5, 2e19), (6, 1e-30), (7, 0.0), (8, 1e-38)):
        val[n] = val[n] / top[n] * size
    c.fill(val.to(c.dt))
    c.check_forward(c.forward())
    c.check_partition(c.partition())
    _, parts, dw = c.backward()
    for i in range(2):
        dy = c.grads[i].double().cpu().numpy()
        dx, b, _, _ = R.backward(c.x[i], c.g(i), c.eps, c.z, dy)
        # r dx below fp32's normal range loses bits: 2^-126 absolute
        c.close(parts[i], dx, b + 2.0 ** -126)
    assert torch.isfinite(dw).all()


def test_nan_and_inf_stay_in_their_row():
    c = Case((4, 4, 4), 2, 64, "bf16", box=(2, 2, 2), seed=6)
    clean_f, clean_p, (_, clean_b, _) = c.forward(), c.partition(), c.backward()
    val = torch.stack([p.clone() for p in c.parts()], 1)
    val[5, 0, 1, 7] = float("nan")
    val[9, 1, 0, 3] = float("inf")
    c.fill(val)
    q, k, v = c.forward()
    assert torch.isnan(q[5, 1]).all() and torch.isnan(k[9, 0]).any()
    for got, want, n, h in ((q, clean_f[0], 5, 1), (k, clean_f[1], 9, 0)):
        keep = torch.ones_like(got, dtype=torch.bool)
        keep[n, h] = False
        assert torch.equal(got[keep], want[keep])
    blocks, want = c.partition()[3], clean_p[3]
    where = int(np.nonzero(c.order() == 9)[0][0]) // 8
    keep = torch.ones(blocks.shape[:2], dtype=torch.bool)
    keep[0, where] = False
    assert torch.equal(blocks[keep], want[keep]) and not torch.isfinite(blocks[0, where]).all()
    _, parts, dw = c.backward()
    keep = torch.ones_like(parts[0], dtype=torch.bool)
    keep[5, 1] = False
    assert torch.equal(parts[0][keep], clean_b[0][keep])
    assert torch.isnan(dw[0]).any()
    # a checkpoint gives the whole group back as NaN and leaves the others alone
    ckpt = c.empty_ckpt()
    c.forward(ckpt=ckpt)
    assert torch.isnan(ckpt.scales).nonzero().tolist() == [[5, 0, 1, 0], [9, 1, 0, 0]]


@pytest.mark.parametrize("weights", [True, False])
def test_gradient_matches_differences(weights):
    """The kernel's gradients along random directions against central
    differences of the plain fp64 forward."""
    c = Case((2, 3, 5), 2, 64, "f32", seed=8, weights=weights, eps=1e-2)
    _, parts, dw = c.backward()
    rng = np.random.default_rng(1)
    for i in range(2):
        dy, g = c.grads[i].double().cpu().numpy(), c.g(i)
        g0 = np.ones(c.d) if g is None else g
        dx, bx, dg, bg = R.backward(c.x[i], g, c.eps, c.z, dy)
        for _ in range(4):
            vx, vg = rng.normal(size=c.x[i].shape), rng.normal(size=c.d)
            step = 1e-5
            f = [(R.forward(c.x[i] + e * vx, g0 + e * vg, c.eps, c.z)[0] * dy).sum()
                 for e in (step, -step)]
            got = (parts[i].double().cpu().numpy() * vx).sum() + \
                (dw[i].double().cpu().numpy() * vg).sum()
            # the kernel's own bounds, and the differences' (step^2 and 2^-53 / step)
            allowed = ((bx + R.U * np.abs(dx)) * np.abs(vx)).sum() + \
                ((bg + R.U * np.abs(dg)) * np.abs(vg)).sum() + 1e-6 * np.abs(dy).sum()
            assert abs((f[0] - f[1]) / (2 * step) - got) <= allowed


def test_streams_and_graphs():
    """Calls on a side stream, two streams at once with a workspace each, and a
    captured pass replayed on new inputs."""
    a = Case((8, 16, 16), 4, 64, "bf16", box=(2, 4, 4), seed=10)
    b = Case((6, 8, 16), 3, 128, "bf16", box=(3, 4, 4), seed=11)
    want = [(c.partition(), c.backward()) for c in (a, b)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for i, c in enumerate((a, b)):
            with torch.cuda.stream(streams[i]):
                got[i].append((c.partition(), c.backward()))
    torch.cuda.synchronize()
    for i in range(2):
        for part, back in got[i]:
            assert all(torch.equal(x, y) for x, y in zip(part, want[i][0]))
            assert all(torch.equal(x, y) for x, y in zip(back[1], want[i][1][1]))
            assert torch.equal(back[2], want[i][1][2])
    # an explicit stream argument
    out = a.forward()
    again = [a.token() for _ in range(3)]
    streams[0].wait_stream(torch.cuda.current_stream())
    V.qk_norm_rope(a.sh, a.nr, a.qkv, *again, stream=streams[0])
    streams[0].synchronize()
    assert all(torch.equal(x, y) for x, y in zip(out, again))

    ckpt, part = a.empty_ckpt(), [a.token(), a.head(), a.head(), a.means()]
    raw, dw = a.buffer()[1], torch.zeros((2, a.d), device="cuda")
    ws = torch.empty((V.qk_norm_rope_bwd_workspace_size(a.sh),), dtype=torch.uint8, device="cuda")

    def passes():
        V.qk_norm_rope_partition(a.sh, a.nr, a.qkv, *part, ckpt=ckpt)
        V.qk_norm_rope_bwd(a.sh, a.nr, ckpt, *a.grads, raw, dw, ws)

    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        passes()
    for seed in (1, 2):
        val = torch.randn((a.s, 3, a.h, a.d), device="cuda",
                          generator=torch.Generator(device="cuda").manual_seed(seed)).to(a.dt)
        a.fill(val)
        graph.replay()
        torch.cuda.synchronize()
        kept = [x.clone() for x in part + a.parts(raw) + [dw]]
        passes()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, part + a.parts(raw) + [dw]))


def test_full_size_sampled():
    """The 55296-token training layer with 3D blocks: sampled rows of every
    output, the block means in full, and the weight gradients."""
    c = Case((24, 36, 64), 12, 128, "bf16", box=(4, 6, 8), seed=12)
    part = c.partition()
    ckpt = c.empty_ckpt()
    assert all(torch.equal(x, y) for x, y in zip(part, c.partition(ckpt=ckpt)))
    c.check_partition(part)
    _, parts, dw = c.backward()
    c.check_backward(parts, dw)
    codes, scales = R.encode8(c.x[1], c.d)
    assert np.array_equal(ckpt.codes[:, 1].cpu().numpy(), codes)
    assert np.array_equal(ckpt.scales[:, 1].cpu().numpy(), scales)


def test_offsets_beyond_32_bits():
    """Raw rows, outputs and checkpoint of more than 2^32 bytes: the last and
    middle blocks equal those of a small run on the same rows."""
    grid, h, d = (64, 64, 64), 24, 128
    dims = (0, 0, 0)
    sh = V.LayerShape(*grid, h, d, 0, 4, 64, 64, "bf16")
    s = sh.s
    qkv = torch.empty((s, 3, h, d), dtype=torch.bfloat16, device="cuda")
    assert qkv.nbytes > 2 ** 32
    gen = torch.Generator(device="cuda").manual_seed(3)
    part = torch.randn((4096, 3, h, d), generator=gen, device="cuda").to(torch.bfloat16)
    for i in range(s // 4096):
        qkv[i * 4096:(i + 1) * 4096] = part * (1 + i)
    nr = V.NormRope(dims=dims)
    q = torch.empty((s, h, d), dtype=torch.bfloat16, device="cuda")
    k, v = torch.empty((h, s, d), dtype=q.dtype, device="cuda"), torch.empty((h, s, d), dtype=q.dtype,
                                                                             device="cuda")
    blocks = torch.empty((h, 16, d), device="cuda")
    ckpt = V.Act8.empty((s, 3, h, d), d)
    V.qk_norm_rope_partition(sh, nr, qkv, q, k, v, blocks, ckpt=ckpt)
    dqkv = torch.empty_like(qkv)
    V.qk_norm_rope_bwd(sh, nr, qkv, q, q, q, dqkv, None, None)
    small = V.LayerShape(4, 64, 64, h, d, 0, 4, 64, 64, "bf16")
    n = small.s
    for j in (0, 7, 15):
        rows = slice(j * n, (j + 1) * n)
        out = [torch.empty_like(q[:n]), torch.empty((h, n, d), dtype=q.dtype, device="cuda"),
               torch.empty((h, n, d), dtype=q.dtype, device="cuda"),
               torch.empty((h, 1, d), device="cuda")]
        c = V.Act8.empty((n, 3, h, d), d)
        V.qk_norm_rope_partition(small, nr, qkv[rows], *out, ckpt=c)
        assert torch.equal(q[rows], out[0]) and torch.equal(k[:, rows], out[1])
        assert torch.equal(v[:, rows], out[2]) and torch.equal(ckpt.codes[rows], c.codes)
        assert torch.equal(ckpt.scales[rows], c.scales)
        # fp32 sums of at most 64 rows a lane, cut differently
        assert (blocks[:, j] - out[3][:, 0]).abs().max() <= 2 * 64 * R.U * out[1].abs().max()
        back = torch.empty_like(qkv[rows])
        V.qk_norm_rope_bwd(small, nr, qkv[rows], q[rows], q[rows], q[rows], back, None, None)
        assert torch.equal(dqkv[rows], back)


def test_refusals_leave_outputs_alone():
    c = Case((2, 4, 4), 2, 64, "bf16", seed=13)
    out = [c.token(), c.head(), c.head(), c.means()]
    n0 = V.kernel_launches()
    bad = V.NormRope(c.gq, c.gk, 0.0, c.table, c.dims)
    with pytest.raises(V.VmobaError, match="VMOBA_ERR_ARG"):
        V.qk_norm_rope_partition(c.sh, bad, c.qkv, *out)
    odd = torch.zeros(c.s * c.h * c.d + 1, dtype=c.dt, device="cuda")[1:].view(c.s, c.h, c.d)
    with pytest.raises(V.VmobaError, match="VMOBA_ERR_ARG"):
        V.qk_norm_rope_partition(c.sh, c.nr, (odd, odd, odd), *out)
    with pytest.raises(V.VmobaError, match="VMOBA_ERR_WORKSPACE"):
        V.qk_norm_rope_bwd(c.sh, c.nr, c.qkv, *c.grads, c.buffer()[1],
                           torch.zeros((2, 64), device="cuda"),
                           torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="v: expected a CUDA"):
        V.qk_norm_rope(c.sh, c.nr, c.qkv, c.token(), c.token(), c.token().cpu())
    with pytest.raises(ValueError, match="table: expected a CUDA"):
        V.qk_norm_rope(c.sh, V.NormRope(c.gq, c.gk, EPS, c.table.cpu(), c.dims), c.qkv, c.token(),
                       c.token(), c.token())
    torch.cuda.synchronize()
    assert V.kernel_launches() == n0
    assert all((t == 9.0).all() for t in out)


@pytest.mark.parametrize("grid,h,d", [((2, 3, 5), 2, 64), ((9, 16, 17), 4, 128)])
def test_chain_reads_what_the_last_call_wrote(grid, h, d):
    """Calls behind one another on a stream, each set up while the one before
    still runs: weights, rows, codes and scales are what that one wrote into
    buffers that held other values before, bit for bit as with waits between."""
    c = Case(grid, h, d, "bf16", seed=21)
    gen = torch.Generator(device="cuda").manual_seed(22)
    n, u = 12, (c.s, 3, c.h, c.d)
    weights = [V.Act8.empty((2, d), d) for _ in range(n)]
    rows = [V.Act8.empty(u, d) for _ in range(n)]
    for w, r in zip(weights, rows):
        V.act8_pack(1 + torch.randn((2, d), generator=gen, device="cuda"), w)
        V.act8_pack(torch.randn(u, generator=gen, device="cuda").to(c.dt), r)
    g = torch.zeros((2, d), device="cuda")
    raw = torch.zeros(u, dtype=c.dt, device="cuda")
    ckpt = V.Act8.empty(u, d)
    ws = torch.zeros(V.qk_norm_rope_bwd_workspace_size(c.sh), dtype=torch.uint8, device="cuda")
    nr = V.NormRope(g[0], g[1], c.eps, c.table, c.dims)

    def chain(between):
        outs = []
        for w, r in zip(weights, rows):
            first, second, grads = ([c.token() for _ in range(3)] for _ in range(3))
            d_raw, d_raw8 = torch.empty_like(raw), torch.empty_like(raw)
            dw, dw8 = torch.empty_like(g), torch.empty_like(g)
            between()
            for call in (
                    lambda: V.act8_unpack(r, raw),
                    lambda: V.act8_unpack(w, g),
                    lambda: V.qk_norm_rope(c.sh, nr, raw, *first, ckpt=ckpt),
                    lambda: V.qk_norm_rope(c.sh, nr, ckpt, *second),
                    lambda: V.qk_norm_rope_bwd(c.sh, nr, raw, *second, d_raw, dw, ws),
                    lambda: V.qk_norm_rope_bwd(c.sh, nr, ckpt, *first, d_raw8, dw8, ws),
                    lambda: V.act8_pack(d_raw8, ckpt),
                    lambda: V.act8_unpack(ckpt, raw),
                    lambda: V.qk_norm_rope(c.sh, nr, raw, *grads)):
                call()
                between()
            outs.append([*first, *second, *grads, d_raw, d_raw8, dw, dw8])
        torch.cuda.synchronize()
        return outs

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        for a, b in zip(chain(lambda: None), want):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_weights_made_at_each_access_live_through_the_call():
    """A norm whose tensors are made when they are read: still alive when the
    last of a call's arguments is read, and what the call computes with."""
    c = Case((3, 4, 5), 2, 64, "bf16", seed=71)
    made, alive = [], []

    def fresh(t):
        t = t.clone()
        made.append(weakref.ref(t))
        return t

    class Norm:
        q_weight = property(lambda self: fresh(c.gq))
        k_weight = property(lambda self: fresh(c.gk))
        table = property(lambda self: fresh(c.table))
        eps, dims = c.eps, c.dims

    class Stream:                      # read after every tensor
        cuda_stream = property(lambda self: torch.cuda.current_stream().cuda_stream)

        @property
        def device(self):
            alive.append([r() is not None for r in made])
            return torch.device("cuda", torch.cuda.current_device())

    out = [c.token(), c.token(), c.token()]
    V.qk_norm_rope(c.sh, Norm(), c.qkv, *out, stream=Stream())
    made.clear()
    assert all(torch.equal(a, b) for a, b in zip(out, c.forward()))
    _, want, dw = c.backward()
    whole, raw = c.buffer()
    got = torch.empty_like(dw)
    ws = torch.empty((V.qk_norm_rope_bwd_workspace_size(c.sh),), dtype=torch.uint8, device="cuda")
    V.qk_norm_rope_bwd(c.sh, Norm(), c.qkv, *c.grads, raw, got, ws, stream=Stream())
    assert all(torch.equal(a, b) for a, b in zip(c.parts(raw), want)) and torch.equal(got, dw)
    assert alive == [[True] * 3] * 2


def test_calls_behind_two_branches_of_a_graph():
    """A captured call whose stream has just joined another branch waits for
    both: its rows come from one, its weights from the other; and a call in a
    branch of its own runs beside the first."""
    c = Case((8, 16, 16), 4, 64, "bf16", box=(2, 4, 4), seed=31)
    raw, g = torch.zeros_like(c.qkv), torch.zeros((2, c.d), device="cuda")
    rows, weights = V.Act8.empty(raw.shape, c.d), V.Act8.empty(g.shape, c.d)
    nr = V.NormRope(g[0], g[1], c.eps, c.table, c.dims)
    one, two = ([c.token(), c.head(), c.head(), c.means()] for _ in range(2))
    draw, dw = torch.zeros_like(raw), torch.zeros_like(g)
    ws = torch.empty((V.qk_norm_rope_bwd_workspace_size(c.sh),), dtype=torch.uint8, device="cuda")
    side = torch.cuda.Stream()

    def passes():
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            V.act8_unpack(weights, g)
        V.act8_unpack(rows, raw)
        main.wait_stream(side)
        V.qk_norm_rope_partition(c.sh, nr, raw, *one)
        side.wait_stream(main)
        with torch.cuda.stream(side):
            V.qk_norm_rope_partition(c.sh, nr, rows, *two)
        V.qk_norm_rope_bwd(c.sh, nr, raw, *c.grads, draw, dw, ws)
        main.wait_stream(side)

    def new(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        V.act8_pack(torch.randn(raw.shape, generator=gen, device="cuda").to(c.dt), rows)
        V.act8_pack(1 + torch.randn((2, c.d), generator=gen, device="cuda"), weights)

    new(1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        passes()
    every = [*one, *two, draw, dw]
    for seed in (2, 3, 4):
        new(seed)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in every]
        for t in (raw, g, *every):
            t.zero_()
        passes()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(kept, every))
        want = [c.token(), c.head(), c.head(), c.means()]
        V.qk_norm_rope_partition(c.sh, nr, raw, *want)
        assert all(torch.equal(x, y) for x, y in zip(want, one))
