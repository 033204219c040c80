"""The linear layer that keeps its input in 8 bits takes what the plain layer
takes and keeps no more than its backward reads."""
import pytest

from . import norm_rope_ref as R

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_sparse_attention_layer_b200 as V  # noqa: E402
from block_sparse_attention_layer_b200 import attention  # noqa: E402
from block_sparse_attention_layer_b200.attention import (Linear8Function,  # noqa: E402
                                                         VMoBASelfAttention)

DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _stored(x, dtype):
    """What x [rows][cols] reads back as from 8 bits."""
    group = 128 if x.shape[1] % 128 == 0 else 64
    codes, scales = R.encode8(x.detach().double().cpu().numpy(), group)
    return torch.from_numpy(R.decode8(codes, scales, group)).to(dtype).cuda()


def _tensors(rows, cols, out_cols, xt, wt, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *size: torch.randn(size, generator=g, device="cuda")    # noqa: E731
    x = normal(rows, cols).to(DT[xt]).requires_grad_(True)
    w, b = (t.to(DT[wt]).requires_grad_(True) for t in (normal(out_cols, cols), normal(out_cols)))
    return x, w, b, normal(rows, out_cols).to(torch.bfloat16)


@pytest.mark.parametrize("xt,wt", [("f32", "f32"), ("f32", "bf16"), ("bf16", "f32"),
                                   ("bf16", "bf16")])
def test_under_autocast(xt, wt):
    """Products in the region's type as the plain layer's, forward and
    backward (which runs outside of the region); gradients in the type of what
    they belong to.  dW is dy^T times the stored values in bf16."""
    x, w, b, dy = _tensors(37, 256, 64, xt, wt)
    with torch.autocast("cuda", dtype=torch.bfloat16):
        y = Linear8Function.apply(x, w, b)
        plain = torch.nn.functional.linear(x, w, b)
    assert y.dtype == torch.bfloat16 and torch.equal(y, plain)
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    px, _, _ = torch.autograd.grad(plain, (x, w, b), dy)
    assert dx.dtype == x.dtype and dw.dtype == w.dtype and db.dtype == b.dtype
    assert torch.equal(dx, px)
    want = dy.t() @ _stored(x, x.dtype).to(torch.bfloat16)
    assert torch.equal(dw, want.to(w.dtype))
    # a sum of 37 bf16 values in fp32, rounded to bf16 or not at all
    exact = dy.double().sum(0)
    allowed = dy.double().abs().sum(0) * 37 * R.U + exact.abs() * R.STEP["bf16"]
    assert ((db.double() - exact).abs() <= allowed).all()


def test_module_with_fp32_tokens_under_autocast():
    """A bf16 module on fp32 tokens: the region casts them for the projection."""
    torch.manual_seed(0)
    m = VMoBASelfAttention(256, 2, 4, 8, 8, 2, ((1, 8, 8), (4, 4, 4), (2, 4, 4)), qk_norm=True,
                           rope=True, checkpoint8=True)
    x = torch.randn((256, 256), device="cuda", requires_grad=True)
    with torch.autocast("cuda", dtype=torch.bfloat16):
        y = m(x)
    y.float().square().mean().backward()
    assert x.grad.dtype == torch.float32 and torch.isfinite(x.grad).all()
    assert all(torch.isfinite(p.grad).all() for p in m.parameters())


@pytest.mark.parametrize("layout", ["transposed", "expanded", "every other", "padded", "axes",
                                    "swapped axes", "one row"])
def test_any_layout(layout):
    """Gradients are those of the same rows laid out densely."""
    g = torch.Generator(device="cuda").manual_seed(5)
    normal = lambda *size: torch.randn(size, generator=g, device="cuda").bfloat16()  # noqa: E731
    x = {"transposed": lambda: normal(192, 6).t(), "expanded": lambda: normal(1, 192).expand(6, 192),
         "every other": lambda: normal(6, 384)[:, ::2], "padded": lambda: normal(6, 200)[:, :192],
         "axes": lambda: normal(2, 3, 192), "swapped axes": lambda: normal(3, 2, 192).transpose(0, 1),
         "one row": lambda: normal(192)}[layout]().requires_grad_(True)
    w, b = normal(64, 192).requires_grad_(True), normal(64).requires_grad_(True)
    dy = normal(*x.shape[:-1], 64)
    y = Linear8Function.apply(x, w, b)
    assert torch.equal(y, torch.nn.functional.linear(x, w, b))
    dx, dw, db = torch.autograd.grad(y, (x, w, b), dy)
    rows = x.detach().reshape(-1, 192).contiguous().requires_grad_(True)
    flat = dy.reshape(-1, 64)
    rx, rw, rb = torch.autograd.grad(Linear8Function.apply(rows, w, b), (rows, w, b), flat)
    assert torch.equal(dx, rx.view(x.shape)) and torch.equal(dw, rw) and torch.equal(db, rb)
    assert torch.equal(dw, flat.t() @ _stored(rows, torch.bfloat16))


def _module(**kw):
    torch.manual_seed(0)
    return VMoBASelfAttention(256, 2, 4, 8, 8, 2, ((1, 8, 8), (4, 4, 4), (2, 4, 4)), qk_norm=True,
                              rope=True, **kw)


def test_frozen_modules_keep_no_codes():
    """Projection weights frozen: only the raw q, k, v are stored; everything
    frozen: nothing, and no kernel stores them."""
    x = torch.randn((256, 256), device="cuda").bfloat16()
    plain, m = _module(), _module(checkpoint8=True)

    def run(m, x):
        codes, n0 = [], V.kernel_launches()

        def keep(t):
            if t.dtype == torch.int8:
                codes.append(t.numel())
            return t

        with torch.autograd.graph.saved_tensors_hooks(keep, lambda t: t):
            y = m(x)
        return y, codes, V.kernel_launches() - n0

    y0, none, n0 = run(plain, x)
    y1, every, n1 = run(m, x)
    assert torch.equal(y0, y1) and none == [] and sorted(every) == [256 * 256] * 2 + [3 * 256 * 256]
    assert n1 == n0 + 2                                   # the two inputs' own passes
    for p in (m.qkv.weight, m.proj.weight):
        p.requires_grad_(False)
    y2, codes, n2 = run(m, x)
    assert codes == [3 * 256 * 256] and n2 == n0 and torch.equal(y2, y0)
    y2.float().square().mean().backward()
    assert m.q_norm.grad is not None and m.qkv.weight.grad is None
    for p in m.parameters():
        p.requires_grad_(False)
    y3, codes, n3 = run(m, x)
    assert codes == [] and n3 == n0 and torch.equal(y3, y0) and not y3.requires_grad


def test_nothing_to_differentiate_writes_no_checkpoint():
    """Rows and weights without gradients: the forward's pass is the one
    without a checkpoint (its own kernel would store 1.03 bytes a value)."""
    m = _module(checkpoint8=True)
    for p in m.parameters():
        p.requires_grad_(False)
    x = torch.randn((256, 256), device="cuda").bfloat16()
    made = []
    empty = attention.Act8.empty
    attention.Act8.empty = lambda *a, **kw: (made.append(a), empty(*a, **kw))[1]
    try:
        m(x)
    finally:
        attention.Act8.empty = empty
    assert made == []


class _Scaled(torch.nn.Module):
    """A module put in a projection's place."""

    def __init__(self, inner):
        super().__init__()
        self.inner = inner

    @property
    def weight(self):
        return self.inner.weight

    @property
    def bias(self):
        return self.inner.bias

    def forward(self, x):
        return 2 * self.inner(x)


@pytest.mark.parametrize("ckpt", [False, True])
def test_projections_are_called_as_modules(ckpt):
    """Hooks on the projections run, modules put in their place are used, and
    the switch can be set later."""
    x = torch.randn((256, 256), device="cuda").bfloat16()
    m = _module(checkpoint8=ckpt)
    y0, seen = m(x), []
    for name in ("qkv", "proj"):
        getattr(m, name).register_forward_hook(lambda mod, i, o, name=name: seen.append(name))
    doubled = m.proj.register_forward_hook(lambda mod, i, o: 2 * o)
    y1 = m(x)
    assert seen == ["qkv", "proj"] and torch.equal(y1, 2 * y0)
    y1.float().square().mean().backward()
    with torch.no_grad():
        assert torch.equal(m(x), y1)
    doubled.remove()
    grads = {n: p.grad for n, p in m.named_parameters()}
    other = _module(checkpoint8=ckpt)
    other.proj = _Scaled(other.proj)
    y2 = other(x)
    assert torch.equal(y2, y1)
    y2.float().square().mean().backward()
    for n, p in other.named_parameters():
        assert torch.equal(p.grad, grads[n.replace("proj.inner", "proj")])
    late = _module(checkpoint8=not ckpt)
    late.checkpoint8 = ckpt
    assert late.checkpoint8 is ckpt
    late.proj.register_forward_hook(lambda mod, i, o: 2 * o)
    late(x).float().square().mean().backward()
    assert all(torch.equal(p.grad, grads[n]) for n, p in late.named_parameters())


@pytest.mark.parametrize("ckpt", [False, True])
def test_modules_share_one_layer(ckpt):
    """Two modules on one layer's buffers: the outputs of modules with their
    own, and their gradients too (from a checkpoint for the second one only:
    the first one's attention is then rebuilt from the stored values)."""
    x = torch.randn((256, 256), device="cuda").bfloat16()
    own = [_module(checkpoint8=ckpt), _module(checkpoint8=ckpt)]
    shared = [_module(checkpoint8=ckpt)]
    shared.append(_module(checkpoint8=ckpt, layer=shared[0].layer))
    assert shared[1].layer is shared[0].layer
    for m in (own[1], shared[1]):
        with torch.no_grad():
            m.proj.bias.add_(1.0)
    ys = [m[1](m[0](x)) for m in (own, shared)]
    assert torch.equal(*ys)
    for y in ys:
        y.float().square().mean().backward()
    for i in ((1,) if ckpt else (0, 1)):
        for (n, p), q in zip(own[i].named_parameters(), shared[i].parameters()):
            assert torch.equal(p.grad, q.grad), n
    # rebuilt from stored values: there and finite
    for p, q in zip(own[0].parameters(), shared[0].parameters()):
        assert torch.isfinite(q.grad).all() and p.grad.abs().max() > 0
    other = V.LayerShape(4, 8, 8, 2, 128, 1, 4, 4, 4, "bf16")
    with pytest.raises(ValueError, match="layer: expected one of shape"):
        _module(layer=attention.VMoBALayer(other))
