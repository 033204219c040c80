"""Cases and plain forms of the operators around the attention layer: the norm
of each head's queries and keys with the 3D position rotation (token order, or
straight into the layer's key blocks), its backward pass, and activation
checkpoints in 8 bits with their use in both.

kinds of cases
  rotate     raw q, k, v of the projection -> normalised and rotated q, k and a
             copy of v, all in token order (what dense attention takes)
  partition  the same into the sparse layer's buffers: q in token order, K' and
             V' in partition order and the block means B
  backward   dq, dk, dv -> gradients of the raw q, k, v and of the norm weights
  train      one layer's use of an 8-bit checkpoint around its attention: the
             forward also writes the checkpoint of raw q, k, v, the backward
             first rebuilds q, K', V', B from it and then takes the gradients
             with the checkpoint in place of the raw values
  act8       an activation is stored in 8 bits and read back (the input of the
             projection, kept for its weight gradient)

Definitions.  Token n = (t, y, x) in frame-major order.  Norm of a head's row:
y = x g / sqrt(mean(x^2) + eps).  Rotation of the adjacent pairs (2p, 2p+1):
the first dt/2 pairs turn with t, the next dh/2 with y, the next dw/2 with x,
the rest stay; the table holds (cos, sin) for each axis position and pair.
B is the mean over a block of the rotated keys before they are rounded to the
storage type.  8 bits: per group of consecutive values a = max |x|,
code = round-half-even(127 x / a), scale = a / 127, value = code * scale.
"""
import torch

own = False

EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _layer(name, kind, grid, heads, d, dtype, box, mode, dims, weights=True, layout="packed",
           origin=0):
    T, H, W = grid
    return {"name": name, "kind": kind, "T": T, "H": H, "W": W, "n_heads": heads, "head_dim": d,
            "dtype": dtype, "mode": mode, "bt": box[0], "bh": box[1], "bw": box[2],
            "dt": dims[0], "dh": dims[1], "dw": dims[2], "weights": weights, "layout": layout,
            "origin": origin}


def listed():
    full, half = (44, 42, 42), (24, 20, 20)
    return [
        # one token appended to a stream: nothing but the cost of the call
        _layer("rotate one token", "rotate", (1, 1, 1), 12, 128, "bf16", (1, 1, 1), 2, full,
               origin=40000),
        # the 11520-token latent, separate q / k / v projections, dense attention
        _layer("rotate 11520 tokens", "rotate", (10, 32, 36), 12, 128, "bf16", (2, 8, 12), 2, full,
               layout="separate"),
        # the smallest workload of the repository, fp32 storage
        _layer("partition 256 tokens f32", "partition", (4, 8, 8), 2, 64, "f32", (2, 4, 4), 2,
               half),
        # the 2048-token workload, 3D blocks of 32 keys
        _layer("partition 2048 tokens", "partition", (8, 16, 16), 4, 64, "bf16", (2, 4, 4), 2,
               half),
        # the inference workload, 2D blocks (20 positions in each of 21 frames)
        _layer("partition 32760 tokens", "partition", (21, 30, 52), 12, 128, "bf16", (21, 5, 4), 1,
               full),
        # the training workload with eight blocks of three frames: few, long blocks
        _layer("partition 55296 tokens", "partition", (24, 36, 64), 12, 128, "bf16", (3, 36, 64),
               0, full),
        # odd grid, three heads, rows inside a wider buffer, fp32
        _layer("backward 693 tokens f32", "backward", (7, 9, 11), 3, 64, "f32", (7, 3, 11), 2,
               (16, 24, 14), layout="padded"),
        # the largest latent of the repository
        _layer("backward 75600 tokens", "backward", (21, 45, 80), 12, 128, "bf16", (3, 9, 8), 2,
               full),
        # the 2048-token workload trained with checkpoints
        _layer("train 2048 tokens", "train", (8, 16, 16), 4, 64, "bf16", (8, 4, 4), 1, half),
        # the headline training layer, 3D blocks of 192 keys
        _layer("train 55296 tokens", "train", (24, 36, 64), 12, 128, "bf16", (4, 6, 8), 2, full),
        # the projection's input of the training layer: 12 heads of 128
        {"name": "act8 55296 x 1536", "kind": "act8", "rows": 55296, "cols": 1536, "group": 128,
         "dtype": "bf16", "pad": 0},
        # ragged: the last group is short, rows are not aligned to vectors
        {"name": "act8 1001 x 1003 f32", "kind": "act8", "rows": 1001, "cols": 1003, "group": 64,
         "dtype": "f32", "pad": 2},
    ]


LARGEST = 55296 * 12 * 128       # tokens x channels of the largest training layer


def draw(rng):
    kind = rng.choice(["rotate", "partition", "partition", "backward", "backward", "train", "train",
                       "act8"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    most = LARGEST if dtype == "bf16" else LARGEST // 2
    if kind == "act8":
        while True:
            rows = int(2 ** rng.uniform(0, 16.2))
            cols = int(2 ** rng.uniform(5, 13))
            cols = cols // 8 * 8 if rng.random() < 0.7 else cols
            if 0 < rows * cols <= most:
                return {"kind": kind, "rows": rows, "cols": cols, "group": rng.choice([64, 128]),
                        "dtype": dtype, "pad": rng.choice([0, 0, 1, 8, 64])}
    d = rng.choice([64, 128, 128])
    while True:
        bt, bh, bw = (int(2 ** rng.uniform(0, 3.4)) for _ in range(3))
        nt, nh, nw = (int(2 ** rng.uniform(0, 3.4)) for _ in range(3))
        heads = rng.choice([1, 2, 3, 4, 5, 8, 12, 16, 24, 40])
        grid = (bt * nt, bh * nh, bw * nw)
        mode = rng.randrange(3)
        blocks = (nt, nh * nw, nt * nh * nw)[mode]
        if blocks <= 1024 and grid[0] * grid[1] * grid[2] * heads * d <= most:
            break
    left, dims = d // 2, []
    for _ in range(3):                          # any even split, parts of zero among them
        n = rng.choice([0, left, rng.randint(0, left), rng.randint(0, left), left // 2])
        dims.append(2 * n)
        left -= n
    rng.shuffle(dims)
    c = _layer("", kind, grid, heads, d, dtype, (bt, bh, bw), mode, dims,
               weights=rng.random() < 0.8, layout=rng.choice(["packed", "separate", "padded"]),
               origin=rng.choice([0, 0, rng.randrange(1 << 20)]))
    del c["name"]
    return c


def _sizes(case):
    T, H, W = case["T"], case["H"], case["W"]
    return T * H * W, case["n_heads"], case["head_dim"], (T, H, W)


def _box(case):
    """The block box of the case's partition mode."""
    T, H, W = case["T"], case["H"], case["W"]
    return ((case["bt"], H, W), (T, case["bh"], case["bw"]),
            (case["bt"], case["bh"], case["bw"]))[case["mode"]]


def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    if case["kind"] == "act8":
        n, groups = case["rows"] * case["cols"], -(-case["cols"] // case["group"])
        # the values are read, codes and scales written and read, the values written
        return {"bytes": 2 * n * e + 2 * (n + 4 * case["rows"] * groups), "flops": 5 * n}
    s, h, d, grid = _sizes(case)
    u = s * h * d
    bt, bh, bw = _box(case)
    blocks = 4 * h * d * (s // (bt * bh * bw))
    table = 4 * (grid[0] * case["dt"] + grid[1] * case["dh"] + grid[2] * case["dw"])
    weights = 8 * d if case["weights"] else 0
    small = table + weights
    ckpt = 3 * u + 12 * s * h
    if case["kind"] == "rotate":
        return {"bytes": 6 * u * e + small, "flops": 2 * u * 10}
    if case["kind"] == "partition":
        return {"bytes": 6 * u * e + small + blocks, "flops": 2 * u * 10 + u}
    if case["kind"] == "backward":                 # raw v is not needed
        return {"bytes": 8 * u * e + small + 8 * d, "flops": 2 * u * 18}
    # forward (writes the checkpoint), rebuild (reads it), gradients (read its q and k parts)
    forward = 6 * u * e + ckpt + small + blocks
    again = ckpt + 3 * u * e + small + blocks
    backward = 2 * u + 8 * s * h + 6 * u * e + small + 8 * d
    return {"bytes": forward + again + backward, "flops": 2 * u * 40}


def _raw_buffers(case):
    """(whole buffer or buffers, [q, k, v] views of [s][heads][d]) in the case's layout."""
    s, h, d, _ = _sizes(case)
    dt = DTYPES[case["dtype"]]
    if case["layout"] == "separate":
        parts = [torch.empty((s, h, d), dtype=dt, device="cuda") for _ in range(3)]
        return tuple(parts), parts
    ld = 3 * h * d + (64 if case["layout"] == "padded" else 0)
    whole = torch.zeros((s, ld), dtype=dt, device="cuda")
    qkv = whole[:, :3 * h * d].view(s, 3, h, d) if ld == 3 * h * d else \
        whole.as_strided((s, 3, h, d), (ld, h * d, d, 1))
    return qkv, [qkv[:, i] for i in range(3)]


def _axis_tables(case):
    """(cos, sin) of each axis position and pair, [T*dt/2 + H*dh/2 + W*dw/2][2] fp32,
    from angles in 64 bits."""
    _, _, _, grid = _sizes(case)
    parts = []
    for n, dim in zip(grid, (case["dt"], case["dh"], case["dw"])):
        pos = torch.arange(n, dtype=torch.float64, device="cuda") + case["origin"]
        i = torch.arange(dim // 2, dtype=torch.float64, device="cuda")
        a = (pos[:, None] * 10000.0 ** (-2.0 * i / max(dim, 1))).reshape(-1)
        parts.append(torch.stack((a.cos(), a.sin()), 1))
    return torch.cat(parts).float().contiguous()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    dt = DTYPES[case["dtype"]]
    st = {"case": case}
    if case["kind"] == "act8":
        rows, cols = case["rows"], case["cols"]
        whole = torch.zeros((rows, cols + case["pad"]), dtype=dt, device="cuda")
        x = whole[:, :cols]
        # activations: channels of unlike size, a few far larger than the rest
        gain = torch.exp(0.5 * normal(cols)) * torch.where(normal(cols) > 2.3, 10.0, 1.0)
        x.copy_(normal(rows, cols) * gain)
        st["x"] = x
        if own:
            import block_sparse_attention_layer_b200 as V
            st["V"], st["ckpt"] = V, V.Act8.empty((rows, cols), case["group"], "cuda")
            st["out"] = torch.empty((rows, cols), dtype=dt, device="cuda")
        return st

    s, h, d, _ = _sizes(case)
    st["raw"], parts = _raw_buffers(case)
    for p in parts:
        gain = torch.exp(0.5 * normal(h, d)) * torch.where(normal(h, d) > 2.3, 8.0, 1.0)
        p.copy_(normal(s, h, d) * gain)
    st["parts"] = parts
    st["gq"] = (1.0 + 0.2 * normal(d)) if case["weights"] else None
    st["gk"] = (1.0 + 0.2 * normal(d)) if case["weights"] else None
    st["table"] = _axis_tables(case)
    if case["kind"] in ("backward", "train"):
        st["grads"] = [(normal(s, h, d) * 0.02).to(dt) for _ in range(3)]
    if own:
        import block_sparse_attention_layer_b200 as V
        st["V"] = V
        st["shape"] = V.LayerShape(case["T"], case["H"], case["W"], h, d, case["mode"], case["bt"],
                                   case["bh"], case["bw"], case["dtype"])
        st["norm"] = V.NormRope(st["gq"], st["gk"], EPS, st["table"],
                                (case["dt"], case["dh"], case["dw"]))
        token = lambda: torch.empty((s, h, d), dtype=dt, device="cuda")       # noqa: E731
        head = lambda: torch.empty((h, s, d), dtype=dt, device="cuda")        # noqa: E731
        means = lambda: torch.empty((h, V.num_blocks(st["shape"]), d), device="cuda")  # noqa: E731
        if case["kind"] == "rotate":
            st["out"] = [token(), token(), token()]
        if case["kind"] in ("partition", "train"):
            st["out"] = [token(), head(), head(), means()]
        if case["kind"] == "train":
            st["again"] = [token(), head(), head(), means()]
            st["ckpt"] = V.Act8.empty((s, 3, h, d), d, "cuda")
        if case["kind"] in ("backward", "train"):
            st["graw"], _ = _raw_buffers(case)
            st["dweight"] = torch.empty((2, d), device="cuda")
            st["ws"] = torch.empty((V.qk_norm_rope_bwd_workspace_size(st["shape"]),),
                                   dtype=torch.uint8, device="cuda")
    return st


# ------------------------------------------------------------- the framework's calls

def _run_own(st):
    V, kind = st["V"], st["case"]["kind"]
    if kind == "act8":
        V.act8_pack(st["x"], st["ckpt"])
        V.act8_unpack(st["ckpt"], st["out"])
        return st["out"]
    sh, nr = st["shape"], st["norm"]
    if kind == "rotate":
        V.qk_norm_rope(sh, nr, st["raw"], *st["out"])
        return st["out"]
    if kind == "partition":
        V.qk_norm_rope_partition(sh, nr, st["raw"], *st["out"])
        return st["out"]
    if kind == "backward":
        V.qk_norm_rope_bwd(sh, nr, st["raw"], *st["grads"], st["graw"], st["dweight"], st["ws"])
        return [_three(st["graw"]), st["dweight"]]
    V.qk_norm_rope_partition(sh, nr, st["raw"], *st["out"], ckpt=st["ckpt"])
    V.qk_norm_rope_partition(sh, nr, st["ckpt"], *st["again"])
    V.qk_norm_rope_bwd(sh, nr, st["ckpt"], *st["grads"], st["graw"], st["dweight"], st["ws"])
    return [st["out"], st["again"], _three(st["graw"]), st["dweight"]]


def _three(raw):
    return list(raw) if isinstance(raw, tuple) else [raw[:, 0], raw[:, 1], raw[:, 2]]


# ------------------------------------------------------------- the plain forms

def _codes(x, group):
    """x [..., cols] fp32 -> (codes as fp32, scales) by groups of the last axis; the
    quotients in 64 bits, since many lie on a rounding border."""
    cols = x.shape[-1]
    n = -(-cols // group)
    x = torch.nn.functional.pad(x, (0, n * group - cols)).view(*x.shape[:-1], n, group)
    a = x.abs().amax(-1, keepdim=True)
    a = torch.where(a < 2.0 ** -119, torch.zeros_like(a), a)
    quotient = torch.where(a > 0, x.double() * 127.0 / a.double(), torch.zeros_like(x).double())
    return quotient.round().float(), a / 127.0


def _plain_act8(x, group):
    """What x [..., cols] reads back as from 8 bits, in fp32."""
    c, scale = _codes(x.float(), group)
    return (c * scale).flatten(-2)[..., :x.shape[-1]]


def _cos_sin(st):
    """[s][1][d/2] cosines and sines; pairs without a position have cos 1, sin 0."""
    case, table = st["case"], st["table"]
    s, _, d, (T, H, W) = _sizes(case)
    halves = (case["dt"] // 2, case["dh"] // 2, case["dw"] // 2)
    parts, at = [], 0
    for axis, (n, p) in enumerate(zip((T, H, W), halves)):
        view = [1, 1, 1, p, 2]
        view[axis] = n
        parts.append(table[at:at + n * p].view(view).expand(T, H, W, p, 2))
        at += n * p
    still = torch.zeros((T, H, W, d // 2 - sum(halves), 2), device=table.device)
    still[..., 0] = 1.0
    cs = torch.cat(parts + [still], 3).view(s, 1, d // 2, 2)
    return cs[..., 0], cs[..., 1]


def _turn(y, cos, sin):
    y0, y1 = y[..., 0::2], y[..., 1::2]
    return torch.stack((y0 * cos - y1 * sin, y0 * sin + y1 * cos), -1).flatten(-2)


def _norm(x, g):
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    return y if g is None else y * g


def _blocked(x, case):
    """[s][heads][d] -> [heads][s][d] in partition order."""
    s, h, d, (T, H, W) = _sizes(case)
    bt, bh, bw = _box(case)
    x = x.reshape(T // bt, bt, H // bh, bh, W // bw, bw, h, d)
    return x.permute(6, 0, 2, 4, 1, 3, 5, 7).reshape(h, s, d)


def _plain_forward(st, q, k, v, cos, sin):
    """q, k, v [s][heads][d] fp32 -> the forward's outputs for the case's kind."""
    case = st["case"]
    dt = DTYPES[case["dtype"]]
    q = _turn(_norm(q, st["gq"]), cos, sin).to(dt)
    k = _turn(_norm(k, st["gk"]), cos, sin)
    if case["kind"] == "rotate":
        return [q, k.to(dt), v.to(dt)]
    k = _blocked(k, case)
    bt, bh, bw = _box(case)
    means = k.view(k.shape[0], -1, bt * bh * bw, k.shape[-1]).mean(2)
    return [q, k.to(dt), _blocked(v.to(dt), case), means]


def _plain_grad(x, g, dy, cos, sin):
    """(gradient of the raw rows, gradient of the weight) in fp32."""
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS)
    xh = x * r
    u = _turn(dy.float(), cos, -sin)
    w = u if g is None else u * g
    dx = r * (w - xh * (w * xh).mean(-1, keepdim=True))
    return dx, (u * xh).sum((0, 1))


def _plain_backward(st, q, k, cos, sin):
    dt = DTYPES[st["case"]["dtype"]]
    dq, dk, dv = st["grads"]
    rq, wq = _plain_grad(q, st["gq"], dq, cos, sin)
    rk, wk = _plain_grad(k, st["gk"], dk, cos, sin)
    return [rq.to(dt), rk.to(dt), dv.clone()], torch.stack((wq, wk))


def _run_plain(st):
    case = st["case"]
    if case["kind"] == "act8":
        return _plain_act8(st["x"], case["group"]).to(st["x"].dtype)
    cos, sin = _cos_sin(st)
    q, k, v = (p.float() for p in st["parts"])
    if case["kind"] in ("rotate", "partition"):
        return _plain_forward(st, q, k, v, cos, sin)
    if case["kind"] == "backward":
        return list(_plain_backward(st, q, k, cos, sin))
    first = _plain_forward(st, q, k, v, cos, sin)
    q, k, v = (_plain_act8(x, case["head_dim"]) for x in (q, k, v))
    return [first, _plain_forward(st, q, k, v, cos, sin), *_plain_backward(st, q, k, cos, sin)]


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ------------------------------------------------------------- in 64 bits

def exact(case, seed):
    """The definition in 64 bits, with complex numbers for the rotation and an explicit
    list of each block's tokens."""
    st = prepare(case, seed)
    f8 = torch.float64

    def from8(x, group):
        out = torch.empty_like(x)
        for at in range(0, x.shape[-1], group):
            part = x[..., at:at + group]
            a = part.abs().max(-1, keepdim=True).values
            a[a < 2.0 ** -119] = 0.0
            step = (a / 127).clamp_min(1e-300)
            out[..., at:at + group] = torch.round(127 * part / a.clamp_min(1e-300)) * step
        return out

    if case["kind"] == "act8":
        return from8(st["x"].to(f8), case["group"])

    s, h, d, (T, H, W) = _sizes(case)
    n = torch.arange(s, device="cuda")
    t, y, x = n // (H * W), n // W % H, n % W
    table = torch.complex(*st["table"].to(f8).unbind(1))
    phase = torch.ones((s, d // 2), dtype=torch.complex128, device="cuda")
    column = start = 0
    for pos, count, dim in ((t, T, case["dt"]), (y, H, case["dh"]), (x, W, case["dw"])):
        p = dim // 2
        phase[:, column:column + p] = table[start:start + count * p].view(count, p)[pos]
        column, start = column + p, start + count * p
    phase = phase[:, None, :]

    bt, bh, bw = _box(case)
    block = ((t // bt) * (H // bh) + y // bh) * (W // bw) + x // bw
    order = torch.argsort(block, stable=True)
    length = bt * bh * bw

    def rotated(rows, g):
        rows = rows / torch.sqrt((rows * rows).sum(-1, keepdim=True) / d + EPS)
        rows = rows if g is None else rows * g.to(f8)
        z = torch.view_as_complex(rows.reshape(s, h, d // 2, 2)) * phase
        return torch.view_as_real(z).reshape(s, h, d)

    def forward(q, k, v):
        q, k = rotated(q, st["gq"]), rotated(k, st["gk"])
        if case["kind"] == "rotate":
            return [q, k, v]
        k, v = k[order].transpose(0, 1), v[order].transpose(0, 1)
        return [q, k, v, k.reshape(h, s // length, length, d).sum(2) / length]

    def gradient(rows, g, dy):
        size = torch.sqrt((rows * rows).sum(-1, keepdim=True) / d + EPS)
        z = torch.view_as_complex(dy.to(f8).reshape(s, h, d // 2, 2)) * phase.conj()
        u = torch.view_as_real(z).reshape(s, h, d)
        w = u if g is None else u * g.to(f8)
        dx = w / size - rows * (w * rows).sum(-1, keepdim=True) / (d * size ** 3)
        return dx, (u * rows / size).reshape(s * h, d).sum(0)

    def backward(q, k):
        dq, dk, dv = st["grads"]
        (rq, wq), (rk, wk) = gradient(q, st["gq"], dq), gradient(k, st["gk"], dk)
        return [[rq, rk, dv.to(f8)], torch.stack((wq, wk))]

    q, k, v = (p.to(f8) for p in st["parts"])
    if case["kind"] in ("rotate", "partition"):
        return forward(q, k, v)
    if case["kind"] == "backward":
        return backward(q, k)
    first = forward(q, k, v)
    q, k, v = (from8(p, d) for p in (q, k, v))
    return [first, forward(q, k, v), *backward(q, k)]
