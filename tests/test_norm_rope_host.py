"""Host-side checks of the norm + rotation and 8-bit checkpoint calls: every
refusal happens before anything is launched (no GPU needed), and the plain
forms that the GPU tests compare with are themselves checked."""
import copy
import ctypes
import dataclasses
import gc
import os
import pickle
import subprocess
import sys
import weakref

import numpy as np
import pytest

import block_sparse_attention_layer_b200 as V
from block_sparse_attention_layer_b200 import _lib

from . import norm_rope_ref as R

torch = pytest.importorskip("torch")

OK = ctypes.c_void_p(0x100000)     # aligned, never dereferenced: the calls fail validation
ODD = ctypes.c_void_p(0x100004)


def _shape(**kw):
    base = dict(T=4, H=8, W=8, n_heads=2, head_dim=64, mode=2, bt=2, bh=4, bw=4, dtype="bf16")
    base.update(kw)
    return V.LayerShape(**base)


def _nr(eps=1e-6, table=0x100000, dims=(24, 20, 20), q=0, k=0):
    return ctypes.byref(_lib.CNormRope(q, k, eps, table, *dims))


def _sh(**kw):
    return ctypes.byref(_shape(**kw).c())


def _fwd(sh=None, nr=None, q_in=OK, ld=384, q=OK, blocks=OK, codes=None, scales=None):
    return V.lib().vmoba_qk_norm_rope_partition(sh or _sh(), nr or _nr(), q_in, OK, OK, ld, q, OK,
                                                OK, blocks, codes, scales, None)


def _bwd(sh=None, nr=None, q_in=OK, ld=384, dq=OK, out=OK, ld_out=384, dw=OK, ws=OK,
         n=1 << 30):
    return V.lib().vmoba_qk_norm_rope_bwd(sh or _sh(), nr or _nr(), q_in, OK, ld, dq, OK, OK, out,
                                          OK, OK, ld_out, dw, ws, n, None)


@pytest.mark.parametrize("call", [_fwd, _bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(sh=_sh(bt=3)), -2), (dict(sh=_sh(head_dim=96)), -2), (dict(sh=_sh(mode=5)), -1),
    (dict(nr=_nr(dims=(3, 2, 2))), -2), (dict(nr=_nr(dims=(-2, 2, 2))), -2),
    (dict(nr=_nr(dims=(64, 2, 0))), -2), (dict(nr=_nr(dims=(2 ** 31 - 2, 2 ** 31 - 2, 6))), -2),
    (dict(nr=_nr(table=0)), -1), (dict(nr=_nr(table=0x100008)), -1),
    (dict(nr=_nr(q=0x100004)), -1), (dict(nr=_nr(k=0x100004)), -1),
    (dict(nr=_nr(eps=0.0)), -1), (dict(nr=_nr(eps=-1.0)), -1), (dict(nr=_nr(eps=float("nan"))), -1),
    (dict(nr=_nr(eps=float("inf"))), -1),
    (dict(q_in=None), -1), (dict(q_in=ODD), -1), (dict(ld=127), -1), (dict(ld=388), -1),
    (dict(ld=0), -1), (dict(ld=1 << 50), -1),
])
def test_layer_calls_refuse(call, kw, code):
    assert call(**kw) == code


@pytest.mark.parametrize("kw", [dict(q=None), dict(q=ODD), dict(blocks=None), dict(blocks=ODD),
                                dict(codes=OK), dict(scales=OK), dict(codes=ODD, scales=OK)])
def test_forward_refuses(kw):
    assert _fwd(**kw) == -1


@pytest.mark.parametrize("kw,code", [
    (dict(dq=None), -1), (dict(dq=ODD), -1), (dict(out=None), -1), (dict(out=ODD), -1),
    (dict(ld_out=64), -1), (dict(ld_out=130), -1), (dict(dw=ODD), -1), (dict(ws=None), -4),
    (dict(ws=ODD), -4), (dict(n=1024), -4)])
def test_backward_refuses(kw, code):
    assert _bwd(**kw) == code


def test_checkpoint_sources_refuse():
    L = V.lib()
    for codes, scales in ((None, OK), (OK, None), (ODD, OK), (OK, ODD)):
        assert L.vmoba_qk_norm_rope_act8(_sh(), _nr(), codes, scales, OK, OK, OK, None) == -1
        assert L.vmoba_qk_norm_rope_partition_act8(_sh(), _nr(), codes, scales, OK, OK, OK, OK,
                                                   None) == -1
        assert L.vmoba_qk_norm_rope_bwd_act8(_sh(), _nr(), codes, scales, OK, OK, OK, OK, OK, OK,
                                             384, None, None, 0, None) == -1
    assert L.vmoba_qk_norm_rope(_sh(), None, OK, OK, OK, 384, OK, OK, OK, None, None, None) == -1


@pytest.mark.parametrize("args,code", [
    (dict(dtype=2), -3), (dict(rows=-1), -2), (dict(cols=0), -2), (dict(ld=9), -2),
    (dict(group=32), -2), (dict(group=0), -2), (dict(rows=1 << 40), -2),
    (dict(rows=1 << 25, ld=1 << 39), -2), (dict(x=None), -1), (dict(codes=None), -1),
    (dict(scales=None), -1), (dict(x=ctypes.c_void_p(0x100001)), -1),
    (dict(scales=ctypes.c_void_p(0x100002)), -1), (dict(rows=0), 0)])
def test_act8_refuses(args, code):
    a = dict(dtype=0, x=OK, rows=4, cols=10, ld=10, group=64, codes=OK, scales=OK)
    a.update(args)
    L = V.lib()
    assert L.vmoba_act8_pack(a["dtype"], a["x"], a["rows"], a["cols"], a["ld"], a["group"],
                             a["codes"], a["scales"], None) == code
    assert L.vmoba_act8_unpack(a["dtype"], a["codes"], a["scales"], a["rows"], a["cols"],
                               a["group"], a["x"], a["ld"], None) == code


@pytest.mark.parametrize("args,code", [
    ((23, 20, 20, 1e4, 0, 0, 0, OK), -2), ((24, 20, 22, 1e4, 0, 0, 0, OK), -2),
    ((24, 20, 20, 0.0, 0, 0, 0, OK), -1), ((24, 20, 20, float("nan"), 0, 0, 0, OK), -1),
    ((24, 20, 20, float("inf"), 0, 0, 0, OK), -1), ((24, 20, 20, 1e4, 1 << 32, 0, 0, OK), -1),
    ((24, 20, 20, 1e4, 0, 0, -(1 << 32), OK), -1), ((24, 20, 20, 1e4, 0, 0, 0, None), -1),
    ((24, 20, 20, 1e4, 0, 0, 0, ODD), -1), ((0, 0, 0, 1e4, 0, 0, 0, None), 0)])
def test_rope_table_refuses(args, code):
    assert V.lib().vmoba_rope_table(_sh(), *args, None) == code


def test_workspace_sizes():
    for d in (64, 128):
        n = V.qk_norm_rope_bwd_workspace_size(_shape(head_dim=d))
        assert n >= 2 * d * 4 and n % 256 == 0
    assert V.qk_norm_rope_bwd_workspace_size(_shape(bt=3)) == 0


def test_binding_refuses_before_the_call():
    """Everything about a tensor is checked before its device, so host tensors
    reach each check; a call that is right but for the device is refused last."""
    sh = _shape()
    s, h, d = sh.s, 2, 64
    bf = torch.bfloat16
    t, qkv = torch.zeros((s, h, d), dtype=bf), torch.zeros((s, 3, h, d), dtype=bf)
    head = t.view(h, s, d)
    wide = torch.zeros((s, 3 * h * d + 64), dtype=bf)
    padded = wide.as_strided((s, 3, h, d), (wide.stride(0), h * d, d, 1))
    nr, table = V.NormRope(), torch.zeros(((4 * 2 + 8 * 4 + 8 * 6) // 2, 2))
    c, x = V.Act8.empty((s, 3, h, d), d, "cpu"), torch.zeros((4, 8))
    means, dw = torch.zeros((h, 8, d)), torch.zeros((2, d))
    ws = torch.zeros(V.qk_norm_rope_bwd_workspace_size(sh), dtype=torch.uint8)

    def fwd(qkv=qkv, q=t, k=t, v=t, nr=nr, **kw):
        V.qk_norm_rope(sh, nr, qkv, q, k, v, **kw)

    def part(q=t, k=head, v=head, blocks=means):
        V.qk_norm_rope_partition(sh, nr, qkv, q, k, v, blocks)

    def bwd(qkv=qkv, dq=t, dk=t, dv=t, out=qkv, dweight=dw, ws=ws):
        V.qk_norm_rope_bwd(sh, nr, qkv, dq, dk, dv, out, dweight, ws)

    def norm(**kw):
        fwd(nr=V.NormRope(**kw))

    for match, call in (
            ("qkv: expected a CUDA", fwd), ("qkv: expected a CUDA", part),
            ("qkv: expected a CUDA", bwd),
            ("qkv: expected a CUDA", lambda: fwd(qkv=padded)),
            ("qkv: expected a CUDA", lambda: fwd(qkv=(t, t, t))),
            ("qkv: expected a CUDA", lambda: fwd(qkv=[qkv[:, i] for i in range(3)])),
            ("qkv.codes: expected a CUDA", lambda: fwd(qkv=c)),
            ("qkv: expected a tensor", lambda: fwd(qkv=3)),
            ("qkv: expected shape", lambda: fwd(qkv=qkv[1:])),
            ("qkv: expected dtype torch.bfloat16, got torch.float32",
             lambda: fwd(qkv=qkv.float())),
            ("qkv: expected one tensor or three", lambda: fwd(qkv=(t, t))),
            ("qkv: expected one token stride", lambda: fwd(qkv=(t, t, qkv[:, 2]))),
            ("qkv: rows overlap", lambda: fwd(qkv=qkv[:1].expand(s, 3, h, d))),
            ("qkv: expected dense rows",
             lambda: fwd(qkv=torch.zeros((s, h, 3, d), dtype=bf).transpose(1, 2))),
            ("qkv: expected dense rows",
             lambda: fwd(qkv=torch.zeros((s, 3, d, h), dtype=bf).transpose(2, 3))),
            ("q: expected shape", lambda: fwd(q=t[1:])),
            ("k: expected a contiguous", lambda: fwd(k=qkv[:, 0])),
            ("v: expected dtype", lambda: fwd(v=t.float())),
            ("checkpoint", lambda: fwd(qkv=c, ckpt=c)),
            ("ckpt: expected an Act8", lambda: fwd(ckpt=t)),
            ("ckpt.codes: expected shape",
             lambda: fwd(ckpt=V.Act8.empty((s, 2, h, d), d, "cpu"))),
            ("ckpt.scales: expected shape",
             lambda: fwd(ckpt=V.Act8(c.codes, c.scales[1:], d))),
            ("ckpt.scales: expected dtype", lambda: fwd(ckpt=V.Act8(c.codes, c.scales.int(), d))),
            ("ckpt.codes: expected a contiguous",
             lambda: fwd(ckpt=V.Act8(torch.zeros((s, 3, h, 2 * d), dtype=torch.int8)[..., :d],
                                     c.scales, d))),
            ("groups of 64, got 128", lambda: fwd(ckpt=V.Act8.empty((s, 3, h, d), 128, "cpu"))),
            ("k_perm: expected shape", lambda: part(k=t)),
            ("blocks: expected shape", lambda: part(blocks=means[:, 1:])),
            ("blocks: expected a tensor", lambda: part(blocks=None)),
            ("dk: expected shape", lambda: bwd(dk=t[1:])),
            ("dqkv: rows overlap", lambda: bwd(out=qkv[:1].expand(s, 3, h, d))),
            ("dweight: expected shape", lambda: bwd(dweight=dw[:1])),
            ("ws: expected a tensor", lambda: bwd(ws=None)),
            ("dims", lambda: norm(dims=(1, 2, 2))), ("dims", lambda: norm(dims=(64, 2, 0))),
            ("dims", lambda: norm(dims=(2, 2))), ("dims", lambda: norm(dims=(2.0, 2, 2))),
            ("dims", lambda: norm(dims=(1 << 70, 2, 2))), ("dims", lambda: norm(dims=None)),
            ("dims", lambda: norm(dims=(-2, 2, 2))),
            ("table: expected a rotation table", lambda: norm(dims=(2, 2, 2))),
            ("table: expected shape", lambda: norm(dims=(2, 2, 2), table=table)),
            ("qkv: expected a CUDA", lambda: norm(dims=[2, 4, 6], table=table)),
            ("q_weight: expected shape", lambda: norm(q_weight=torch.zeros(32))),
            ("k_weight: expected dtype", lambda: norm(k_weight=torch.zeros(64, dtype=bf))),
            ("64 or 128", lambda: V.Act8.empty((4, 4), 32, "cpu")),
            ("bfloat16 or float32",
             lambda: V.act8_pack(x.half(), V.Act8.empty((4, 8), 64, "cpu"))),
            ("two axes", lambda: V.act8_pack(torch.zeros(4), V.Act8.empty((4,), 64, "cpu"))),
            ("dense rows", lambda: V.act8_pack(x.t(), V.Act8.empty((8, 4), 64, "cpu"))),
            ("dense rows",
             lambda: V.act8_unpack(V.Act8.empty((4, 8), 64, "cpu"), x[:1].expand(4, 8))),
            ("groups of 64 or 128", lambda: V.act8_pack(x, V.Act8(c.codes, c.scales, 32))),
            ("ckpt.codes: expected shape",
             lambda: V.act8_pack(x, V.Act8.empty((4, 9), 64, "cpu"))),
            ("x: expected a CUDA", lambda: V.act8_pack(x, V.Act8.empty((4, 8), 64, "cpu"))),
            ("dims", lambda: V.rope_table(sh, (2, 3, 4))),
            ("CUDA", lambda: V.rope_table(sh, (2, 4, 4), device="cpu"))):
        with pytest.raises(ValueError, match=match):
            call()
    with pytest.raises(AttributeError):
        V.qk_norm_rope(sh, None, qkv, t, t, t)
    with pytest.raises(V.VmobaError, match="SHAPE"):
        V.qk_norm_rope(_shape(bt=3), nr, qkv, t, t, t)


def test_a_used_shape_is_copied_and_pickled():
    sh = _shape()
    assert sh._native is not None and sh._ref is not None
    for other in (copy.deepcopy(sh), pickle.loads(pickle.dumps(sh)),
                  dataclasses.replace(sh, n_heads=2)):
        assert other == sh and hash(other) == hash(sh) and "_native" not in other.__dict__
        assert other._native is not sh._native


def test_rope_dims():
    assert V.rope_dims(128) == (44, 42, 42) and V.rope_dims(64) == (24, 20, 20)


def test_plain_gradients_match_differences():
    """The plain backward against central differences of the plain forward."""
    rng = np.random.default_rng(3)
    s, h, d = 6, 2, 8
    z = R.phases(1, 2, 3, d, (2, 4, 2), R.table(1, 2, 3, (2, 4, 2)))
    x, g, dy = rng.normal(size=(s, h, d)), rng.normal(size=d) + 1, rng.normal(size=(s, h, d))
    dx, _, dg, _ = R.backward(x, g, 1e-3, z, dy)
    step = 1e-5
    for _ in range(8):
        vx, vg = rng.normal(size=x.shape), rng.normal(size=d)
        f = [(R.forward(x + e * vx, g + e * vg, 1e-3, z)[0] * dy).sum() for e in (step, -step)]
        assert abs((f[0] - f[1]) / (2 * step) - (dx * vx).sum() - (dg * vg).sum()) < 1e-7


def test_plain_rotation_is_the_stated_one():
    """Brute force: each pair turned by its axis position's angle."""
    T, H, W, d, dims, o = 2, 3, 4, 16, (4, 6, 2), (5, 0, 100)
    z = R.phases(T, H, W, d, dims, R.table(T, H, W, dims, 100.0, o))
    for t in range(T):
        for y in range(H):
            for x in range(W):
                want = []
                for pos, dim in zip((t + o[0], y + o[1], x + o[2]), dims):
                    want += [pos * 100.0 ** (-2 * i / dim) for i in range(dim // 2)]
                want += [0.0] * (d // 2 - len(want))
                got = z[(t * H + y) * W + x]
                assert np.allclose(got, np.exp(1j * np.array(want)), atol=1e-12)


_WIDEST = """
import ctypes, sys
import block_sparse_attention_layer_b200 as V
L, p = V.lib(), ctypes.c_void_p(0x100000)
for cols in (2 ** 31 - 128, 2 ** 31 - 127, 2 ** 31 - 64, 2 ** 31 - 63, 2 ** 31 - 8, 2 ** 31 - 1):
    for group in (64, 128):
        for dtype in (0, 1):
            print(L.vmoba_act8_pack(dtype, p, 1, cols, cols, group, p, p, None),
                  L.vmoba_act8_unpack(dtype, p, p, 1, cols, group, p, cols, None))
"""


def test_act8_takes_the_widest_rows():
    """Rows up to the widest that an int counts reach the launch, which fails
    here for want of a device (none is visible to the process)."""
    env = dict(os.environ, CUDA_VISIBLE_DEVICES="")
    done = subprocess.run([sys.executable, "-c", _WIDEST], env=env, timeout=100, text=True,
                          capture_output=True, cwd=os.path.dirname(os.path.dirname(__file__)))
    assert done.returncode == 0, done.stderr
    assert done.stdout.split() == ["-5"] * 48


def test_a_call_holds_its_tensors():
    """Tensors that an argument makes anew at each access live as long as the
    call that was given them."""
    sh = _shape()
    size, d = (sh.s, 3, 2, 64), 64
    made = []

    def fresh(*a, **kw):
        t = torch.zeros(*a, **kw)
        made.append(weakref.ref(t))
        return t

    class Made(V.Act8):
        codes = property(lambda self: fresh(size, dtype=torch.int8))
        scales = property(lambda self: fresh(size[:3] + (1,)))
        group = d

        def __init__(self):
            pass

    class Seen(Exception):
        pass

    class Norm:                        # its attributes are read after the rows
        @property
        def dims(self):
            raise Seen([r() is not None for r in made])

    t = torch.zeros((sh.s, 2, d), dtype=torch.bfloat16)
    out = torch.zeros(size, dtype=torch.bfloat16)
    for call in (lambda: V.qk_norm_rope(sh, Norm(), Made(), t, t, t),
                 lambda: V.qk_norm_rope_bwd(sh, Norm(), Made(), t, t, t, out, None, None)):
        made.clear()
        with pytest.raises(Seen) as e:
            call()
        assert e.value.args[0] == [True, True]
        del e
        gc.collect()
        assert [r() for r in made] == [None, None]


def test_the_call_with_the_most_tensors():
    """Separate rows and gradients, weights, table, totals and workspace: all
    fourteen are compared, the first one named."""
    sh = _shape()
    bf = torch.bfloat16
    t = [torch.zeros((sh.s, 2, 64), dtype=bf) for _ in range(9)]
    w = [torch.ones(64) for _ in range(2)]
    nr = V.NormRope(*w, 1e-6, torch.zeros(((4 * 24 + 8 * 20 + 8 * 20) // 2, 2)), (24, 20, 20))
    ws = torch.zeros(V.qk_norm_rope_bwd_workspace_size(sh), dtype=torch.uint8)
    dw = torch.zeros((2, 64))
    every = [*t, *w, nr.table, dw, ws]
    before = [sys.getrefcount(x) for x in every]
    for _ in range(3):
        with pytest.raises(ValueError, match="qkv: expected a CUDA tensor"):
            V.qk_norm_rope_bwd(sh, nr, tuple(t[:3]), *t[3:6], tuple(t[6:]), dw, ws)
    assert len(every) == 14 and [sys.getrefcount(x) for x in every] == before


def test_linear8_takes_any_layout():
    """Transposed, expanded and spread inputs and ones with other than two axes
    get as far as a dense one: to the device check."""
    from block_sparse_attention_layer_b200.attention import Linear8Function
    dense = torch.zeros((6, 64))
    w = torch.zeros((8, 64), requires_grad=True)
    for x in (dense, torch.zeros((64, 6)).t(), dense[:1].expand(6, 64), dense[:, :1].expand(6, 64),
              torch.zeros((6, 128))[:, ::2], torch.zeros((6, 96))[:, :64], torch.zeros((2, 3, 64)),
              torch.zeros((3, 2, 64)).transpose(0, 1), dense[0]):
        with pytest.raises(ValueError, match="x: expected a CUDA tensor"):
            Linear8Function.apply(x, w, None)


def test_linear8_with_a_frozen_weight_stores_nothing():
    """Without a gradient of the weight x is neither stored (which would need a
    device) nor kept."""
    from block_sparse_attention_layer_b200.attention import Linear8Function
    w, b = torch.randn(8, 64), torch.randn(8, requires_grad=True)
    for x in (torch.randn(6, 64), torch.randn(6, 64, requires_grad=True)):
        kept = []
        with torch.autograd.graph.saved_tensors_hooks(lambda t: (kept.append(t), t)[1], lambda t: t):
            y = Linear8Function.apply(x, w, b)
        assert [t.data_ptr() for t in kept] == ([w.data_ptr()] if x.requires_grad else [])
        wanted = [t for t in (x, b) if t.requires_grad]
        want = torch.autograd.grad(torch.nn.functional.linear(x, w, b).square().sum(), wanted)
        got = torch.autograd.grad(y.square().sum(), wanted)
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    assert not Linear8Function.apply(x.detach(), w, b.detach()).requires_grad


_WITHOUT = """
import importlib.abc, sys
class Blocked(importlib.abc.MetaPathFinder):
    def find_spec(self, name, path=None, target=None):
        if name.split('.')[-1].startswith('_calls') or name == BLOCK:
            raise ImportError(name + ' is blocked')
sys.meta_path.insert(0, Blocked())
import os.path
exists = os.path.exists
os.path.exists = lambda p: '_calls' not in str(p) and exists(p)
"""


def _python(code):
    return subprocess.run([sys.executable, "-c", code], timeout=100, text=True, capture_output=True,
                          cwd=os.path.dirname(os.path.dirname(__file__)))


def test_the_plain_layer_imports_without_the_native_calls():
    """The attention, its module and the names of the package load without
    _calls; the first call of what needs it raises."""
    done = _python("BLOCK = None" + _WITHOUT + """
import block_sparse_attention_layer_b200 as V
from block_sparse_attention_layer_b200 import attention, layer, norm_rope
from block_sparse_attention_layer_b200 import *
import torch
c, x = V.Act8.empty((4, 64), 64, 'cpu'), torch.zeros(4, 64)
sh = V.LayerShape(4, 8, 8, 2, 64, 2, 2, 4, 4, 'bf16')
for call in (lambda: V.act8_pack(x, c), lambda: V.act8_unpack(c, x),
             lambda: V.qk_norm_rope(sh, V.NormRope(), x, x, x, x)):
    try:
        call()
    except (ImportError, RuntimeError) as e:
        assert '_calls' in str(e)
        print('raised')
""")
    assert done.stdout.split() == ["raised"] * 3, done.stderr


def test_the_package_names_load_without_torch():
    done = _python("BLOCK = 'torch'" + _WITHOUT + """
from block_sparse_attention_layer_b200 import *
print(lib() is not None, rope_dims(128) == (44, 42, 42), 'torch' in sys.modules)
""")
    assert done.stdout.split() == ["True", "True", "False"], done.stderr


@pytest.fixture
def fake_tools(tmp_path, monkeypatch):
    """The build script with its outputs in a folder of its own and compilers
    that only make their output file; the list of what they were asked for."""
    from block_sparse_attention_layer_b200 import build as B
    ran, broken = [], []

    def run(cmd, **kw):
        out = os.path.basename(cmd[cmd.index("-o") + 1])
        ran.append(out)
        if any(out.startswith(b) for b in broken):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name in ("LIB", "OBJ", "CALLS", "PKG"):
        if hasattr(B, name):
            monkeypatch.setattr(B, name, str(tmp_path / os.path.basename(getattr(B, name))))
    os.makedirs(B.PKG, exist_ok=True)
    return B, ran, broken


def test_the_library_builds_without_the_native_calls(fake_tools):
    """Where the Python calls cannot be compiled the library is there all the
    same, and the reason is told."""
    B, ran, broken = fake_tools
    broken.append("_calls")
    with pytest.warns(RuntimeWarning, match="no such header"):
        assert B.build(jobs=1) == B.LIB
    assert os.path.exists(B.LIB) and ran[-1].startswith("_calls")
    broken.clear()
    ran.clear()
    B.build(jobs=1)
    assert len(ran) == 1 and ran[0].startswith("_calls")
    B.build(jobs=1)
    assert len(ran) == 1


def test_native_calls_belong_to_one_torch(fake_tools, monkeypatch):
    """What was built against another torch is neither current nor loaded."""
    B, ran, _ = fake_tools
    B.build(jobs=1)
    assert len([r for r in ran if r.startswith("_calls")]) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    with monkeypatch.context() as m:
        from block_sparse_attention_layer_b200 import norm_rope
        m.setattr(norm_rope, "_bound", False)
        with pytest.raises(RuntimeError, match="missing: build it"):
            norm_rope._bind()
    B.build(jobs=1)
    assert len([r for r in ran if r.startswith("_calls")]) == 2


@pytest.mark.parametrize("call", ["prologue", "select_pooled", "select", "select_variant",
                                  "use_selection", "partition_only", "forward"])
def test_every_call_that_changes_the_state_counts(call, monkeypatch):
    """The forward state of a layer (keys, selection, plan, LSE) ends with any
    call that writes a part of it; a backward tells so by the generation."""
    from block_sparse_attention_layer_b200 import layer as lay
    for name in ("partition", "score_select", "score_select_variant", "build_plan", "attn_fwd"):
        monkeypatch.setattr(_lib, name, lambda *a, **kw: None)
    monkeypatch.setattr(lay.norm_rope, "qk_norm_rope_partition", lambda *a, **kw: None)
    layer = lay.VMoBALayer(_shape(), device="cpu", max_pair_fraction=0.1)
    t, before = torch.zeros(1), layer.generation
    args = dict(prologue=(t, None), select_pooled=(t, 0.3), select=(t, t, t, 0.3),
                select_variant=(t, t, t, "topk_global", 2), use_selection=(layer.sel.clone(),),
                partition_only=(t, t), forward=(t,))[call]
    getattr(layer, call)(*args)
    assert layer.generation > before
