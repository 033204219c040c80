"""Norm, rotation and 8-bit checkpoints as the self-attention module runs them:
the whole run against the fp64 oracle, against the single operators bit for
bit, with the layer's buffers shared between forwards, and in a graph."""
import math

import numpy as np
import pytest

import oracle as O

from . import norm_rope_attn_ref as A
from . import norm_rope_ref as R
from .gpu_util import TOL, from_device, out_err, unpack_bits

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover
    pytest.skip("needs a CUDA device", allow_module_level=True)

import block_sparse_attention_layer_b200 as V  # noqa: E402
from block_sparse_attention_layer_b200.attention import (Linear8Function,  # noqa: E402
                                                         VMoBANormRopeFunction,
                                                         VMoBASelfAttention)
from block_sparse_attention_layer_b200.layer import VMoBALayer  # noqa: E402

T, H, W, NH, D = 8, 16, 16, 2, 128
S = T * H * W
BOXES = ((1, 16, 16), (8, 4, 4), (2, 4, 4))
DIMS = V.rope_dims(D)
SCALE = 1 / math.sqrt(D)
EPS = 1e-6


def _layer(mode=2):
    return VMoBALayer(V.LayerShape(T, H, W, NH, D, mode, *BOXES[mode], "bf16"))


def _inputs(seed, leaf=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *size: torch.randn(size, generator=g, device="cuda")    # noqa: E731
    qkv = normal(S, 3, NH, D).to(torch.bfloat16)
    w = [1 + 0.2 * normal(D) for _ in range(2)]
    dout = normal(S, NH, D).to(torch.bfloat16)
    if leaf:
        qkv.requires_grad_(True)
        for t in w:
            t.requires_grad_(True)
    return qkv, w[0], w[1], dout


def _apply(layer, qkv, gq, gk, table, tau=0.4, full=False, ckpt=False):
    return VMoBANormRopeFunction.apply(qkv, gq, gk, layer, table, DIMS, EPS, tau, full, SCALE, ckpt)


def _table():
    return V.rope_table(_layer().shape, DIMS)


def _by_hand(layer, qkv, gq, gk, dout, table, tau=0.4, start=None, at=None, sel=None):
    """The same run by the single operators: rows from `start` (default qkv),
    norm gradient at `at` (default qkv)."""
    nr = V.NormRope(gq, gk, EPS, table, DIMS)
    layer.prologue(qkv if start is None else start, nr)
    if sel is None:
        layer.select_pooled(layer.q, tau, SCALE)
    else:
        layer.use_selection(sel)
    out = layer.forward(layer.q, SCALE)[0].clone()
    layer.backward(layer.q, dout, SCALE)
    dqkv, dw = torch.empty_like(qkv), torch.empty((2, D), device="cuda")
    V.qk_norm_rope_bwd(layer.shape, nr, qkv if at is None else at, layer.dq, layer.dk, layer.dv,
                       dqkv, dw, layer.ws_norm)
    return out, dqkv, dw


@pytest.mark.parametrize("mode,full", [(0, False), (1, False), (2, False), (2, True)])
def test_run_matches_oracle(mode, full):
    """Selection, output and gradients: the oracle's attention on the rows that
    the forward pass made (these themselves within their own bound), then the
    plain norm backward; an error e of dq and dk reaches the raw gradients as
    r (|g| e' + |xh| mean(|g| e' |xh|)) at most, e' over its rotated pair."""
    layer, table = _layer(mode), _table()
    qkv, gq, gk, dout = _inputs(20 + mode)
    out = _apply(layer, qkv, gq, gk, table, full=full)
    out.backward(dout)
    torch.cuda.synchronize()
    z = R.phases(T, H, W, D, DIMS, table.double().cpu().numpy())
    box = O.mode_box(mode, T, H, W, *BOXES[mode])
    order = O.partition_order(T, H, W, box)
    raw = qkv.detach().double().cpu().numpy()
    g = [t.detach().double().cpu().numpy() for t in (gq, gk)]
    back = np.empty_like(order)
    back[order] = np.arange(S)
    q = from_device(layer.q)
    k, v = (from_device(t).transpose(1, 0, 2)[back] for t in (layer.k_perm, layer.v_perm))
    for got, want, b in zip((q, k), *zip(*(R.forward(raw[:, i], g[i], EPS, z) for i in range(2)))):
        assert (np.abs(got - want) <= R.STEP["bf16"] * np.abs(want) + b).all()
    assert np.array_equal(v, raw[:, 2])
    sel = unpack_bits(layer.sel.cpu().numpy(), layer.n_blocks)
    if full:
        assert sel.all()
    blk = O.block_of_token(T, H, W, box)
    o_ref, _ = O.attention_fwd(q, k, v, sel, blk, SCALE)
    ref = O.attention_bwd(q, k, v, sel, blk, SCALE, dout.double().cpu().numpy())
    assert out_err(from_device(out.detach()), o_ref, "bf16") <= TOL["bf16"]
    got = qkv.grad.double().cpu().numpy()
    for i in range(2):
        dx, b, dg, bg = R.backward(raw[:, i], g[i], EPS, z, ref[i])
        r = 1 / np.sqrt((raw[:, i] ** 2).mean(-1, keepdims=True) + EPS)
        xh = np.abs(raw[:, i] * r)
        e = R.pair_abs(TOL["bf16"] + R.STEP["bf16"] * np.abs(ref[i]))
        w = e * np.abs(g[i])
        allowed = b + r * (w + xh * (w * xh).mean(-1, keepdims=True))
        assert (np.abs(got[:, i] - dx) <= allowed + R.STEP["bf16"] * (np.abs(dx) + allowed)).all()
        dgot = (gq, gk)[i].grad.double().cpu().numpy()
        assert (np.abs(dgot - dg) <= bg + (e * xh).reshape(-1, D).sum(0) + R.U * np.abs(dg)).all()
    assert out_err(got[:, 2], ref[2], "bf16") <= TOL["bf16"]


@pytest.mark.parametrize("ckpt", [False, True])
def test_function_is_the_operators(ckpt):
    """The autograd function against the operators called one by one; with a
    checkpoint only the norm's gradient is taken at the stored values."""
    table = _table()
    qkv, gq, gk, dout = _inputs(30)
    out = _apply(_layer(), qkv, gq, gk, table, ckpt=ckpt)
    out.backward(dout)
    raw = qkv.detach()
    c = V.Act8.empty(raw.shape, D)
    V.act8_pack(raw, c)
    want, dqkv, dw = _by_hand(_layer(), raw, gq.detach(), gk.detach(), dout, table,
                              at=c if ckpt else None)
    assert torch.equal(out.detach(), want) and torch.equal(qkv.grad, dqkv)
    assert torch.equal(gq.grad, dw[0]) and torch.equal(gk.grad, dw[1])


@pytest.mark.parametrize("ckpt", [False, True])
def test_shared_layer_rebuilds(ckpt):
    """Two forwards through one layer, backwards in either order: the second
    one's state is still there, the first one's is rebuilt from what it saved."""
    table, shared = _table(), _layer()
    runs = [_inputs(seed) for seed in (40, 41)]
    outs = [_apply(shared, q, a, b, table, ckpt=ckpt) for q, a, b, _ in runs]
    for i in (1, 0):
        outs[i].backward(runs[i][3])
    torch.cuda.synchronize()
    for i, (qkv, gq, gk, dout) in enumerate(runs):
        raw, c, fresh = qkv.detach(), V.Act8.empty(qkv.shape, D), _layer()
        V.act8_pack(raw, c)
        out, dqkv, dw = _by_hand(fresh, raw, gq.detach(), gk.detach(), dout, table,
                                 at=c if ckpt else None)
        assert torch.equal(outs[i].detach(), out)
        if ckpt and i == 0:                # rebuilt: the attention of the stored values
            sel = fresh.sel.clone()
            _, dqkv, dw = _by_hand(_layer(), raw, gq.detach(), gk.detach(), dout, table, start=c,
                                   at=c, sel=sel)
        assert torch.equal(qkv.grad, dqkv)
        assert torch.equal(gq.grad, dw[0]) and torch.equal(gk.grad, dw[1])


def test_prologue_without_a_forward_ends_the_state():
    """A prologue on the same layer between forward and backward (nothing else)
    overwrites keys and queries: the backward must rebuild, not use them."""
    table, layer = _table(), _layer()
    qkv, gq, gk, dout = _inputs(45)
    out = _apply(layer, qkv, gq, gk, table)
    other = _inputs(46, leaf=False)
    layer.prologue(other[0], V.NormRope(other[1], other[2], EPS, table, DIMS))
    out.backward(dout)
    _, dqkv, dw = _by_hand(_layer(), qkv.detach(), gq.detach(), gk.detach(), dout, table)
    assert torch.equal(qkv.grad, dqkv) and torch.equal(gq.grad, dw[0])


def test_weights_may_be_absent_or_frozen():
    table = _table()
    qkv, gq, gk, dout = _inputs(50)
    out = _apply(_layer(), qkv, None, None, table)
    out.backward(dout)
    ones = torch.ones(D, device="cuda")
    want, dqkv, _ = _by_hand(_layer(), qkv.detach(), ones, ones, dout, table)
    assert torch.equal(out.detach(), want) and torch.equal(qkv.grad, dqkv)
    qkv.grad = None
    frozen = gq.detach()
    _apply(_layer(), qkv, frozen, gk, table).backward(dout)
    assert frozen.grad is None and gk.grad is not None
    with pytest.raises(RuntimeError, match="once_differentiable"):
        x = qkv.detach().requires_grad_(True)
        (gx,) = torch.autograd.grad(_apply(_layer(), x, None, None, table).float().square().sum(),
                                    x, create_graph=True)
        gx.float().sum().backward()


@pytest.mark.parametrize("rows,cols,out_cols", [(1, 64, 8), (37, 256, 64), (300, 200, 24)])
def test_linear8(rows, cols, out_cols):
    """dW is dy^T times the stored values, everything else the plain layer's."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x, w, b, dy = (torch.randn(size, generator=g, device="cuda").to(torch.bfloat16)
                   for size in ((rows, cols), (out_cols, cols), (out_cols,), (rows, out_cols)))
    for t in (x, w, b):
        t.requires_grad_(True)
    y = Linear8Function.apply(x, w, b)
    y.backward(dy)
    assert torch.equal(y, torch.nn.functional.linear(x, w, b))
    group = 128 if cols % 128 == 0 else 64
    codes, scales = R.encode8(x.detach().double().cpu().numpy(), group)
    x8 = torch.from_numpy(R.decode8(codes, scales, group)).to(torch.bfloat16).cuda()
    assert torch.equal(w.grad, dy.t() @ x8)
    assert torch.equal(x.grad, dy @ w.detach()) and torch.equal(b.grad, dy.sum(0))


def _module(ckpt, **kw):
    torch.manual_seed(0)
    return VMoBASelfAttention(NH * D, NH, T, H, W, 2, BOXES, tau=0.3, qk_norm=True, rope=True,
                              checkpoint8=ckpt, **kw)


def _saved_bytes(m, x):
    """What autograd holds for the backward, without parameters and tables."""
    kept = {id(p) for p in m.parameters()} | {id(m.rope_table)}
    size = []
    with torch.autograd.graph.saved_tensors_hooks(
            lambda t: (size.append(0 if id(t) in kept or t.dim() < 2 else
                                   t.numel() * t.element_size()), t)[1], lambda t: t):
        y = m(x)
    return y, sum(size)


def test_module_trains_with_and_without_checkpoints():
    x = (torch.randn((S, NH * D), device="cuda") * 0.5).to(torch.bfloat16)
    plain, small = _module(False), _module(True)
    weights = sum(p.numel() * p.element_size() for p in plain.parameters() if p.dim() > 1)
    y0, n0 = _saved_bytes(plain, x)
    y1, n1 = _saved_bytes(small, x)
    assert torch.equal(y0, y1)             # the forward is the same
    # bf16: x, qkv, o; 8 bits: a code for each and a scale of 4 bytes for 128
    sel = plain.layer.sel.numel() * 4
    assert n0 - sel >= 10 * S * NH * D
    assert n1 - sel <= 5 * S * NH * D * (1 + 4 / 128) + weights
    for m, y in ((plain, y0), (small, y1)):
        y.float().square().mean().backward()
        assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in m.parameters())
    # gradients that no checkpoint touches: the last layer's bias
    assert torch.equal(plain.proj.bias.grad, small.proj.bias.grad)
    with torch.no_grad():
        assert torch.equal(small(x), y0.detach())
        full = small(x, full_attention=True)
    assert full.shape == x.shape and torch.isfinite(full).all()


def test_module_moved_to_another_type():
    """Norm weights moved to bf16 with the rest: used and trained in fp32."""
    x = (torch.randn((S, NH * D), device="cuda") * 0.5).to(torch.bfloat16)
    m, moved = _module(False), _module(False).to(torch.bfloat16)
    assert moved.q_norm.dtype == torch.bfloat16 and moved.rope_table.dtype == torch.float32
    assert torch.equal(m(x), moved(x))
    moved(x).float().square().mean().backward()
    assert moved.q_norm.grad.dtype == torch.bfloat16 and torch.isfinite(moved.q_norm.grad).all()


def test_module_arguments():
    with pytest.raises(ValueError, match="need qk_norm"):
        VMoBASelfAttention(NH * D, NH, T, H, W, 2, BOXES, rope=True)
    with pytest.raises(ValueError, match="need qk_norm"):
        VMoBASelfAttention(NH * D, NH, T, H, W, 2, BOXES, checkpoint8=True)
    with pytest.raises(ValueError, match="dims"):
        _module(False).__class__(NH * D, NH, T, H, W, 2, BOXES, qk_norm=True, rope=(1, 2, 3))
    old = VMoBASelfAttention(NH * D, NH, T, H, W, 2, BOXES)
    assert set(old.state_dict()) == {"qkv.weight", "qkv.bias", "proj.weight", "proj.bias"}
    assert set(_module(False).state_dict()) == set(old.state_dict()) | {"q_norm", "k_norm"}


def test_forward_and_backward_in_a_graph():
    """A whole step captured and replayed on new inputs gives what the same
    calls give outside; no eager graph of the same leaves is alive meanwhile."""
    table, layer = _table(), _layer()
    qkv, gq, gk, dout = _inputs(60)

    def step():
        out = _apply(layer, qkv, gq, gk, table, ckpt=True)
        return (out.detach(), *torch.autograd.grad(out, (qkv, gq, gk), dout))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for seed in (61, 62):
        with torch.no_grad():
            qkv.copy_(_inputs(seed, leaf=False)[0])
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in captured]
        eager = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(kept, eager))


@pytest.mark.parametrize("between", ["select_pooled", "select", "select_variant", "use_selection",
                                     "partition_only"])
def test_a_selection_in_between_ends_the_state(between):
    """A selection or partition on the layer between forward and backward, with
    no forward after it: the gradients are still the first call's."""
    table, layer = _table(), _layer()
    qkv, gq, gk, dout = _inputs(47)
    out = _apply(layer, qkv, gq, gk, table)
    a, b, c = (t.contiguous() for t in _inputs(48, leaf=False)[0].unbind(1))
    args = dict(select_pooled=(layer.q, 0.1, SCALE), select=(a, b, c, 0.1, SCALE),
                select_variant=(a, b, c, "topk_global", 100, SCALE),
                use_selection=(torch.zeros_like(layer.sel),), partition_only=(b, c))[between]
    getattr(layer, between)(*args)
    out.backward(dout)
    _, dqkv, dw = _by_hand(_layer(), qkv.detach(), gq.detach(), gk.detach(), dout, table)
    assert torch.equal(qkv.grad, dqkv) and torch.equal(gq.grad, dw[0])


@pytest.mark.parametrize("mode,full", [(0, False), (1, False), (2, False), (2, True)])
def test_gradients_of_the_run_within_their_own_bounds(mode, full):
    """The two halves of the backward, each against its own formula: the
    attention's dq and dk against the oracle's at the rows that the forward
    made, within the bound of their fp16 operands; then the raw rows' and the
    norm weights' gradients against the plain norm backward of those very dq
    and dk, within the norm's own fp32 bounds.  Gradients that are zero,
    negated or a tenth off are outside of either."""
    layer, table = _layer(mode), _table()
    qkv, gq, gk, dout = _inputs(70 + mode)
    _apply(layer, qkv, gq, gk, table, full=full).backward(dout)
    torch.cuda.synchronize()
    z = R.phases(T, H, W, D, DIMS, table.double().cpu().numpy())
    box = O.mode_box(mode, T, H, W, *BOXES[mode])
    order = O.partition_order(T, H, W, box)
    back = np.empty_like(order)
    back[order] = np.arange(S)
    q = from_device(layer.q)
    k, v = (from_device(t).transpose(1, 0, 2)[back] for t in (layer.k_perm, layer.v_perm))
    sel, blk = unpack_bits(layer.sel.cpu().numpy(), layer.n_blocks), O.block_of_token(T, H, W, box)
    dy = dout.double().cpu().numpy()
    lse = O.attention_fwd(q, k, v, sel, blk, SCALE)[1]
    some = sel.any(-1)
    assert (np.abs(layer.lse.double().cpu().numpy()[some] - lse[some]) <= A.LSE).all()
    ref = O.attention_bwd(q, k, v, sel, blk, SCALE, dy)
    bounds = A.attention_bounds(q, k, v, sel[:, :, blk], SCALE, dy)

    def within(got, want, bound):
        return np.abs(got - want) <= bound + R.STEP["bf16"] * (np.abs(want) + bound) + \
            R.TINY["bf16"]

    def rejects(check, got):
        return not check(0 * got).all() and not check(-got).all() and not check(1.1 * got).all()

    grads = [from_device(layer.dq), from_device(layer.dk)]
    for i in range(2):
        check = lambda g: within(g, ref[i], bounds[i])                  # noqa: E731
        assert check(grads[i]).all()
        assert rejects(check, grads[i]) and check(0 * grads[i]).mean() < 0.5
    raw = qkv.detach().double().cpu().numpy()
    got = qkv.grad.double().cpu().numpy()
    for i, g in enumerate((gq, gk)):
        dx, b, dg, bg = R.backward(raw[:, i], g.detach().double().cpu().numpy(), EPS, z, grads[i])
        check = lambda x: within(x, dx, b)                              # noqa: E731
        assert check(got[:, i]).all()
        assert rejects(check, got[:, i]) and check(0 * dx).mean() < 0.5     # rows without a pair are zero
        check = lambda w: np.abs(w - dg) <= bg + R.U * np.abs(dg)       # noqa: E731
        dgot = g.grad.double().cpu().numpy()
        assert check(dgot).all()
        assert rejects(check, dgot) and check(0 * dgot).mean() < 0.05
    assert np.array_equal(got[:, 2], from_device(layer.dv))
