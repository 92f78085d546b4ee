"""The atom-wise dense operators: what is measured, and their plain forms.

Two operators and their gradients, on row-major feature matrices (one row per
atom, edge or token):

  norm    s = x + residual,  y = s / sqrt(mean(s^2) + eps) * weight, with y in
          the input's type or in 8 bits (e4m3) with one scale per row;
  linear  y = act(x w^T + bias) + residual, with x and w in one floating type,
          or both in 8 bits with a scale per row of x and per row of w.

A case with `train` is a training step of the operator: the forward pass that
keeps what its backward needs, and the backward pass, returning the gradients.
Otherwise it is the forward pass alone, as when energies are evaluated.

Case keys: op, dtype (f32, f16, bf16, e4m3), rows, train, pad (the row stride
of x exceeds its width by this many elements: a view of wider features);
norm: width, residual, quantize;  linear: inner, outer, act, bias, residual.
"""
import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0
AMAX_FLOOR = 2.0 ** -100  # keeps the reciprocal of an empty row's scale finite
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "silu", "gelu")
# no drawn case costs more than the largest listed one
MOST_FLOPS = 6 * 8192 * 2048 * 8192
MOST_VALUES = 16384 * 4096


def _norm(name, dtype, rows, width, residual=True, quantize=False, train=False, pad=0):
    return dict(name=name, op="norm", dtype=dtype, rows=rows, width=width, residual=residual, quantize=quantize,
                train=train, pad=pad)


def _linear(name, dtype, rows, inner, outer, act, bias=True, residual=True, train=False, pad=0):
    return dict(name=name, op="linear", dtype=dtype, rows=rows, inner=inner, outer=outer, act=act, bias=bias,
                residual=residual, train=train, pad=pad)


def listed():
    return [
        # one row of a wide residual stream: pure launch latency
        _norm("norm_row", "bf16", 1, 4096),
        # the 32,768-atom cell at 128 channels, four invariants a channel, trained in float32
        _norm("norm_atoms_train", "f32", 32768, 512, train=True),
        # rows that leave in 8 bits for a scaled matrix product
        _norm("norm_e4m3", "bf16", 8192, 4096, quantize=True),
        # an odd width: no row but the first is aligned
        _norm("norm_odd", "f16", 5003, 1023, residual=False),
        # a large training batch
        _norm("norm_train", "bf16", 16384, 4096, train=True),
        # one row through a square layer: the weight is read once
        _linear("linear_row", "bf16", 1, 4096, 4096, "silu"),
        # a handful of rows of odd number
        _linear("linear_few", "f16", 17, 2048, 1000, "relu", residual=False),
        # the 4,096-atom cell: l = 0 channels taken as a view of the 16 x 64 message, in float32
        _linear("linear_atoms", "f32", 4096, 64, 256, "silu", residual=False, pad=960),
        # the 32,768-atom cell at 512 invariants, trained in float32
        _linear("linear_atoms_train", "f32", 32768, 512, 512, "silu", train=True),
        # ragged in every direction
        _linear("linear_odd", "bf16", 1531, 1029, 2771, "gelu"),
        # 8-bit activations and weights
        _linear("linear_e4m3", "e4m3", 8192, 4096, 4096, "silu"),
        # the largest: a training step of a wide layer
        _linear("linear_train", "bf16", 8192, 2048, 8192, "silu", train=True),
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], even in its logarithm; half of the larger ones are multiples of 16."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    if n > 64 and rng.random() < 0.5:
        n = min(hi, n // 16 * 16)
    return n - 16 if n == 3072 else n


def draw(rng):
    while True:
        train = rng.random() < 0.4
        pad = rng.choice([0, 0, 0, 8, 13, 128])
        if rng.random() < 0.4:
            dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
            c = _norm("", dtype, _size(rng, 1, 65536), _size(rng, 8, 16384), rng.random() < 0.7,
                      not train and rng.random() < 0.4, train, pad)
            fits = c["rows"] * (c["width"] + pad) <= MOST_VALUES
        else:
            dtype = rng.choice(["f32", "f16", "bf16", "bf16", "e4m3"])
            c = _linear("", dtype, _size(rng, 1, 32768), _size(rng, 16, 8192), _size(rng, 8, 8192),
                        rng.choice(ACTS), rng.random() < 0.7, rng.random() < 0.5, train and dtype != "e4m3", pad)
            fits = work(c)["flops"] <= MOST_FLOPS
        if fits:
            del c["name"]
            return c


def _quantize_rows(x):
    """x (float32 rows) in e4m3 with one scale per row, as a user's program holds it."""
    scale = x.abs().amax(dim=1).clamp_min(AMAX_FLOOR) / E4M3_MAX
    return (x / scale[:, None]).to(torch.float8_e4m3fn), scale


def _view(values, pad):
    """The same values as a column range of a wider matrix."""
    if not pad:
        return values
    wide = torch.zeros(values.shape[0], values.shape[1] + pad, dtype=values.dtype, device=values.device)
    wide[:, : values.shape[1]] = values
    return wide[:, : values.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    rows, eight = case["rows"], case["dtype"] == "e4m3"
    t = torch.bfloat16 if eight else TYPES[case["dtype"]]
    s = dict(case=case, dtype=t)
    if case["op"] == "norm":
        n = case["width"]
        # features differ in size from channel to channel, as a trained network's do
        x = normal(rows, n) * torch.exp(normal(n))
        s["x"] = _view(x.to(t), case["pad"])
        s["weight"] = (1 + 0.1 * normal(n)).to(t)
        s["residual"] = normal(rows, n).to(t) if case["residual"] else None
        if case["train"]:
            s["gy"] = normal(rows, n).to(t)
            # the gradient that arrives along the residual stream
            s["gsum"] = normal(rows, n).to(t) if case["residual"] else None
        return s
    k, n = case["inner"], case["outer"]
    x, w = normal(rows, k), normal(n, k) / k ** 0.5
    s["x_scale"] = s["w_scale"] = None
    if eight:
        x, s["x_scale"] = _quantize_rows(x)
        w, s["w_scale"] = _quantize_rows(w)
        s["x"], s["w"] = _view(x.view(torch.uint8), case["pad"]).view(torch.float8_e4m3fn), w
    else:
        s["x"], s["w"] = _view(x.to(t), case["pad"]), w.to(t)
    s["bias"] = (0.1 * normal(n)).to(t) if case["bias"] else None
    s["residual"] = normal(rows, n).to(t) if case["residual"] else None
    if case["train"]:
        s["gy"] = normal(rows, n).to(t)
    return s


def run(state):
    if state["case"]["op"] == "norm":
        return _own_norm(state) if own else _plain_norm(state)
    return _own_linear(state) if own else _plain_linear(state)


# ------------------------------------------------------------------ the framework's operators


def _own_norm(s):
    from equivariant_edge_convolution_amd import binding as B

    c = s["case"]
    f = B.add_rms_norm(s["x"], s["weight"], residual=s["residual"], eps=EPS, quantize=c["quantize"],
                       save_rstd=c["train"])
    out = dict(y=f["y"])
    if c["residual"]:
        out["sum"] = f["sum"]
    if c["quantize"]:
        out["scale"] = f["scale"]
    if c["train"]:
        b = B.add_rms_norm_backward(s["gy"], f["sum"], s["weight"], f["rstd"], gsum=s["gsum"])
        out.update(gx=b["gx"], gweight=b["gweight"])
    return out


def _own_linear(s):
    from equivariant_edge_convolution_amd import binding as B

    c = s["case"]
    f = B.linear(s["x"], s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], x_scale=s["x_scale"],
                 w_scale=s["w_scale"], out_dtype=s["dtype"], save_preact=c["train"])
    out = dict(y=f["y"])
    if c["train"]:
        b = B.linear_backward(s["gy"], s["x"], s["w"], preact=f["preact"], act=c["act"], bias=c["bias"])
        out.update(gx=b["gx"], gw=b["gw"])
        if c["bias"]:
            out["gbias"] = b["gbias"]
    return out


# ------------------------------------------------------------------ the plain forms, in float32


def _plain_norm(s):
    c, t = s["case"], s["dtype"]
    w = s["weight"].float()
    h = s["x"].float()
    if c["residual"]:
        h = h + s["residual"].float()
    rstd = torch.rsqrt((h * h).mean(dim=1, keepdim=True) + EPS)
    y = h * rstd * w
    out = dict(sum=h.to(t)) if c["residual"] else {}
    if c["quantize"]:
        out["y"], out["scale"] = _quantize_rows(y)
    else:
        out["y"] = y.to(t)
    if c["train"]:
        gy = s["gy"].float()
        xhat = h * rstd
        a = gy * w
        gx = rstd * (a - xhat * (a * xhat).mean(dim=1, keepdim=True))
        if c["residual"]:
            gx = gx + s["gsum"].float()
        out["gx"] = gx.to(t)
        out["gweight"] = (gy * xhat).sum(dim=0).to(t)
    return out


def _act(z, act):
    if act == "relu":
        return torch.clamp_min(z, 0.0)
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * 0.5 ** 0.5))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0.0).float()
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p * (1.0 + z * (1.0 - p))
    return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327


def _plain_linear(s):
    c, t = s["case"], s["dtype"]
    x, w = s["x"].float(), s["w"].float()
    if s["x_scale"] is not None:
        x, w = x * s["x_scale"][:, None], w * s["w_scale"][:, None]
    z = x @ w.t()
    if c["bias"]:
        z = z + s["bias"].float()
    y = _act(z, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    out = dict(y=y.to(t))
    if c["train"]:
        gz = s["gy"].float()
        if c["act"] != "none":
            gz = gz * _act_slope(z, c["act"])
        out["gx"] = (gz @ w).to(t)
        out["gw"] = (gz.t() @ x).to(t)
        if c["bias"]:
            out["gbias"] = gz.sum(dim=0).to(t)
    return out


# ------------------------------------------------------------------ the definitions, in float64


def exact(case, seed):
    """Values in float64, the gradients by differentiating the definition.

    An 8-bit output has the value before its rounding: what the codes stand for."""
    s = prepare(case, seed)
    up = lambda v: None if v is None else v.double()
    if case["op"] == "norm":
        x, w, r = up(s["x"]), up(s["weight"]), up(s["residual"])
        w.requires_grad_(case["train"])
        h = (x if r is None else x + r).requires_grad_(case["train"])
        y = torch.nn.functional.rms_norm(h, (case["width"],), w, EPS)
        out = dict(y=y.detach())
        if r is not None:
            out["sum"] = h.detach()
        if case["quantize"]:
            out["scale"] = y.abs().max(dim=1).values / E4M3_MAX
            out["y"] = y / out["scale"].unsqueeze(1)
        if case["train"]:
            gh, out["gweight"] = torch.autograd.grad(y, (h, w), up(s["gy"]))
            out["gx"] = gh if r is None else gh + up(s["gsum"])
        return out
    x, w = up(s["x"]), up(s["w"])
    if s["x_scale"] is not None:
        x, w = x * up(s["x_scale"]).unsqueeze(1), w * up(s["w_scale"]).unsqueeze(1)
    wanted = [v.requires_grad_(case["train"]) for v in (x, w)]
    b = up(s["bias"])
    if b is not None:
        wanted.append(b.requires_grad_(case["train"]))
    z = torch.nn.functional.linear(x, w, b)
    f = dict(none=lambda v: v, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu)
    a = f[case["act"]](z)
    out = dict(y=a.detach() if s["residual"] is None else a.detach() + up(s["residual"]))
    if case["train"]:
        out.update(zip(("gx", "gw", "gbias"), torch.autograd.grad(a, wanted, up(s["gy"]))))
    return out


def work(case):
    """Each input read once, each output written once; the products' multiplications and additions."""
    rows = case["rows"]
    size = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1}[case["dtype"]]
    if case["op"] == "norm":
        n, res, train = case["width"], int(case["residual"]), int(case["train"])
        # x and, with a residual, residual and sum; y; in training gy, gx and the residual stream's gradient
        moved = 1 + 2 * res + train * (2 + res)
        y = rows * n * (1 if case["quantize"] else size) + (4 * rows if case["quantize"] else 0)
        return dict(bytes=rows * n * size * moved + y + n * size * (1 + train), flops=rows * n * (6 + 10 * train))
    k, n, train = case["inner"], case["outer"], int(case["train"])
    out = 2 if case["dtype"] == "e4m3" else size
    moved = rows * k * size + n * k * size + rows * n * out * (1 + int(case["residual"]) + train)
    moved += n * out * int(case["bias"]) + train * (rows * k + n * k + n * int(case["bias"])) * out
    if case["dtype"] == "e4m3":
        moved += 4 * (rows + n)
    return dict(bytes=moved, flops=2 * rows * k * n * (1 + 2 * train))
