"""A gated layer, products in 8-bit integers, and the update that trains their weights: what is measured, and the plain forms.

Three operators on row-major matrices (one row per atom, edge or token), beside the norm and the dense layer that
perf/operators.py measures:

  gated  z = x w^T + bias, whose first `outer` columns are the gate and the others the value:
         y = act(z_gate) z_value, and its gradients from the z that the forward kept;
  int8   y = act(x w^T + bias) + residual with x and w in 8-bit integers, a scale per row of x (token) and per row
         of w (channel); `dynamic`: x arrives in 16 or 32 bits and its rows are quantised in the pass;
  ortho  an update (a matrix, or several of one shape) brought near the nearest matrix with orthonormal rows or
         columns: X = g / (|g| + eps), then `steps` times X <- a X + (b A + c A^2) X with A = X X^T.

Case keys: op, dtype (f32, f16, bf16; gated and int8: also e4m3, i8);
  gated: rows, inner, outer, act, bias, pad, pass (forward: y;  keep: y and the z that the backward reads;  backward);
  int8:  rows, inner, outer, act, bias, residual, pad, dynamic (dtype: that of x before it is quantised, and of y);
  ortho: batch, rows, cols, steps.
pad: the row stride of x exceeds its width by this many elements (a view of wider features).
"""
import torch

own = False

E4M3_MAX, I8_MAX = 448.0, 127.0
AMAX_FLOOR = 2.0 ** -100  # keeps the reciprocal of an empty row's scale finite
EPS = 1e-7                # beside the norm of an update
QUINTIC = (3.4445, -4.7750, 2.0315)
TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("none", "relu", "silu", "gelu")
# no drawn case costs more than the largest listed one of its kind
MOST_FLOPS = 4 * 8192 * 2048 * 2 * 8192
MOST_ORTHO = 5 * (4 * 2048 * 2048 * 8192 + 2 * 2048 ** 3)


def _gated(name, dtype, rows, inner, outer, act="silu", bias=True, pad=0, pass_="forward"):
    return {"name": name, "op": "gated", "dtype": dtype, "rows": rows, "inner": inner, "outer": outer, "act": act,
            "bias": bias, "pad": pad, "pass": pass_}


def _int8(name, dtype, rows, inner, outer, act="none", bias=True, residual=False, pad=0, dynamic=True):
    return dict(name=name, op="int8", dtype=dtype, rows=rows, inner=inner, outer=outer, act=act, bias=bias,
                residual=residual, pad=pad, dynamic=dynamic)


def _ortho(name, dtype, batch, rows, cols, steps=5):
    return dict(name=name, op="ortho", dtype=dtype, batch=batch, rows=rows, cols=cols, steps=steps)


def listed():
    return [
        # one row through a wide block: both halves of the weight are read once
        _gated("gated_row", "bf16", 1, 2048, 8192, bias=False),
        # the 4,096-atom cell: l = 0 channels taken as a view of the 16 x 64 message, in float32
        _gated("gated_atoms", "f32", 4096, 64, 256, pad=960),
        # ragged in every direction
        _gated("gated_odd", "f16", 1531, 1029, 1387, "gelu"),
        # a large training batch: the forward pass, which keeps what the backward reads ...
        _gated("gated_keep", "bf16", 8192, 2048, 8192, pass_="keep"),
        # ... and its backward pass
        _gated("gated_back", "bf16", 8192, 2048, 8192, pass_="backward"),
        # the 32,768-atom cell at 512 invariants, trained in float32
        _gated("gated_back_atoms", "f32", 32768, 512, 512, pass_="backward"),
        # a handful of rows that are in 8 bits already
        _int8("int8_few", "bf16", 17, 4096, 4096, residual=True, dynamic=False),
        # ragged in every direction, quantised on the way
        _int8("int8_odd", "f16", 1531, 1029, 2771, "gelu"),
        # a large evaluation batch, quantised on the way
        _int8("int8_large", "bf16", 8192, 4096, 4096, "silu", residual=True),
        # the weights of a small head, all in one call
        _ortho("ortho_heads", "f32", 4, 256, 64),
        # one odd matrix in float32
        _ortho("ortho_odd", "f32", 1, 771, 1025),
        # the weight of a wide layer
        _ortho("ortho_wide", "bf16", 1, 8192, 2048),
    ]


def _size(rng, lo, hi):
    """A size in [lo, hi], even in its logarithm; half of the larger ones are multiples of 16."""
    n = int(round(lo * (hi / lo) ** rng.random()))
    return min(hi, n // 16 * 16) if n > 64 and rng.random() < 0.5 else n


def draw(rng):
    while True:
        kind = rng.random()
        pad = rng.choice([0, 0, 0, 8, 13, 128])
        if kind < 0.45:
            c = _gated("", rng.choice(["f32", "f16", "bf16", "bf16", "e4m3", "i8"]), _size(rng, 1, 32768),
                       _size(rng, 16, 8192), _size(rng, 8, 8192), rng.choice(ACTS), rng.random() < 0.7, pad)
            if c["dtype"] in TYPES:
                c["pass"] = rng.choice(["forward", "keep", "backward"])
            most = MOST_FLOPS
        elif kind < 0.7:
            c = _int8("", rng.choice(["f32", "f16", "bf16", "bf16"]), _size(rng, 1, 32768), _size(rng, 16, 8192),
                      _size(rng, 8, 8192), rng.choice(ACTS), rng.random() < 0.7, rng.random() < 0.5, pad,
                      rng.random() < 0.6)
            most = MOST_FLOPS
        else:
            c = _ortho("", rng.choice(["f32", "f16", "bf16", "bf16"]), rng.choice([1, 1, 2, 3, 8]),
                       _size(rng, 16, 8192), _size(rng, 16, 8192), rng.choice([5, 5, 6]))
            most = MOST_ORTHO
        if work(c)["flops"] <= most:
            del c["name"]
            return c


# ------------------------------------------------------------------ inputs


def _quantize(x, most):
    """x (float32 rows) divided by a scale per row, largest magnitude `most`; not yet rounded."""
    scale = x.abs().amax(dim=1).clamp_min(AMAX_FLOOR) / most
    return x / scale[:, None], scale


def _eight_bits(x, i8):
    v, scale = _quantize(x, I8_MAX if i8 else E4M3_MAX)
    return torch.round(v).to(torch.int8) if i8 else v.to(torch.float8_e4m3fn), scale


def _view(values, pad):
    """The same values as a column range of a wider matrix."""
    if not pad:
        return values
    raw = values.view(torch.uint8) if values.dtype == torch.float8_e4m3fn else values
    wide = torch.zeros(raw.shape[0], raw.shape[1] + pad, dtype=raw.dtype, device=raw.device)
    wide[:, : raw.shape[1]] = raw
    return wide[:, : raw.shape[1]].view(values.dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    normal = lambda *shape: torch.randn(*shape, generator=g, device="cuda")
    op, dt = case["op"], case["dtype"]
    t = TYPES.get(dt, torch.bfloat16)
    s = dict(case=case, dtype=t)
    if op == "ortho":
        b, m, n = case["batch"], case["rows"], case["cols"]
        # a gradient: a few strong directions over noise that differs from row to row and from column to column
        r = max(1, min(m, n) // 16)
        u = normal(b, m, n) * torch.exp(0.5 * normal(b, m, 1)) * torch.exp(0.5 * normal(b, 1, n))
        u += (normal(b, m, r) @ normal(b, r, n)) * (4.0 / r ** 0.5)
        s["g"] = (1e-3 * u).to(t)
        return s
    rows, k, n = case["rows"], case["inner"], case["outer"] * (2 if op == "gated" else 1)
    x, w = normal(rows, k), normal(n, k) / k ** 0.5
    if op == "int8":
        # features differ in size from channel to channel, as a trained network's do
        x = x * torch.exp(0.5 * normal(k))
    s["x_scale"] = s["w_scale"] = None
    if dt in ("e4m3", "i8") or (op == "int8" and not case["dynamic"]):
        x, s["x_scale"] = _eight_bits(x, dt != "e4m3")
    else:
        x = x.to(t)
    if dt in ("e4m3", "i8") or op == "int8":
        w, s["w_scale"] = _eight_bits(w, dt != "e4m3")
    else:
        w = w.to(t)
    s["x"], s["w"] = _view(x, case["pad"]), w
    s["bias"] = (0.1 * normal(n)).to(t) if case["bias"] else None
    if op == "int8":
        s["residual"] = normal(rows, n).to(t) if case["residual"] else None
    elif case["pass"] == "backward":
        # z as the forward kept it
        z = s["x"].float() @ w.float().t()
        s["preact"] = (z if s["bias"] is None else z + s["bias"].float()).to(t)
        s["gy"] = normal(rows, case["outer"]).to(t)
    return s


def run(state):
    op = state["case"]["op"]
    if op == "ortho":
        return _own_ortho(state) if own else _plain_ortho(state)
    if op == "int8":
        return _own_int8(state) if own else _plain_int8(state)
    return _own_gated(state) if own else _plain_gated(state)


# ------------------------------------------------------------------ the framework's operators


def _own_gated(s):
    from equivariant_edge_convolution_amd import binding as B

    c = s["case"]
    if c["pass"] == "backward":
        b = B.gated_linear_backward(s["gy"], s["x"], s["w"], s["preact"], act=c["act"], bias=c["bias"])
        return {k: v for k, v in b.items() if v is not None}
    return B.gated_linear(s["x"], s["w"], bias=s["bias"], act=c["act"], x_scale=s["x_scale"], w_scale=s["w_scale"],
                          out_dtype=s["dtype"], save_preact=c["pass"] == "keep")


def _own_int8(s):
    from equivariant_edge_convolution_amd import binding as B

    c, out = s["case"], {}
    x, scale = s["x"], s["x_scale"]
    if c["dynamic"]:
        q = B.quantize_rows(x, torch.int8)
        x, scale = q["y"], q["scale"]
        out.update(q=x, scale=scale)
    f = B.linear(x, s["w"], bias=s["bias"], act=c["act"], residual=s["residual"], x_scale=scale, w_scale=s["w_scale"],
                 out_dtype=s["dtype"])
    return dict(out, y=f["y"])


def _own_ortho(s):
    from equivariant_edge_convolution_amd import binding as B

    return dict(y=B.orthogonalize(s["g"], steps=s["case"]["steps"], coefficients=QUINTIC, eps=EPS))


# ------------------------------------------------------------------ the plain forms, in float32


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
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * 0.5 ** 0.5)) + z * torch.exp(-0.5 * z * z) * 0.3989422804014327
    return torch.ones_like(z)


def _plain_gated(s):
    c, t, n = s["case"], s["dtype"], s["case"]["outer"]
    x, w = s["x"].float(), s["w"].float()
    if c["pass"] == "backward":
        z, gy = s["preact"].float(), s["gy"].float()
        gate, value = z[:, :n], z[:, n:]
        gz = torch.cat([gy * value * _act_slope(gate, c["act"]), gy * _act(gate, c["act"])], dim=1)
        out = dict(gx=(gz @ w).to(t), gw=(gz.t() @ x).to(t))
        if c["bias"]:
            out["gbias"] = gz.sum(dim=0).to(t)
        return out
    if s["x_scale"] is not None:
        x, w = x * s["x_scale"][:, None], w * s["w_scale"][:, None]
    z = x @ w.t()
    if c["bias"]:
        z = z + s["bias"].float()
    out = dict(y=(_act(z[:, :n], c["act"]) * z[:, n:]).to(t))
    if c["pass"] == "keep":
        out["preact"] = z.to(t)
    return out


def _plain_int8(s):
    c, t = s["case"], s["dtype"]
    x, scale, out = s["x"], s["x_scale"], {}
    if c["dynamic"]:
        v, scale = _quantize(x.float(), I8_MAX)
        x = torch.round(v).to(torch.int8)
        out.update(q=x, scale=scale)
    y = (x.float() @ s["w"].float().t()) * scale[:, None] * s["w_scale"]
    if c["bias"]:
        y = y + s["bias"].float()
    y = _act(y, c["act"])
    if c["residual"]:
        y = y + s["residual"].float()
    return dict(out, y=y.to(t))


def _plain_ortho(s):
    a, b, c = QUINTIC
    g = s["g"].float()
    # the norm scales every value: a long sum in 32 bits is off by more than the products after it
    x = g * (1.0 / (g.double().square().sum(dim=(1, 2), keepdim=True).sqrt() + EPS)).float()
    tall = g.shape[1] > g.shape[2]
    if tall:
        x = x.transpose(1, 2).contiguous()
    for _ in range(s["case"]["steps"]):
        gram = x @ x.transpose(1, 2)
        x = a * x + (b * gram + c * (gram @ gram)) @ x
    return dict(y=(x.transpose(1, 2) if tall else x).contiguous().to(s["dtype"]))


# ------------------------------------------------------------------ the definitions, in float64


def exact(case, seed):
    """Values in float64: gradients by differentiating the definition, sums of integers as they are, and the
    orthogonalised update as one polynomial of its first Gram matrix. Codes in 8 bits have none but themselves."""
    s = prepare(case, seed)
    up = lambda v: None if v is None else v.double()
    f = dict(none=lambda v: v, relu=torch.relu, silu=torch.nn.functional.silu, gelu=torch.nn.functional.gelu)
    if case["op"] == "ortho":
        a, b, c = QUINTIC
        g = up(s["g"])
        g = g / (torch.linalg.matrix_norm(g)[:, None, None] + EPS)
        wide = g.shape[1] <= g.shape[2]
        gram = torch.matmul(g, g.mT) if wide else torch.matmul(g.mT, g)
        one = torch.eye(gram.shape[1], dtype=gram.dtype, device=gram.device).expand_as(gram)
        whole = one
        for _ in range(case["steps"]):
            m = a * one + b * gram + c * torch.matmul(gram, gram)
            whole, gram = torch.matmul(m, whole), torch.matmul(torch.matmul(m, gram), m)
        return dict(y=torch.matmul(whole, g) if wide else torch.matmul(g, whole))
    x, w, bias, n = up(s["x"]), up(s["w"]), up(s["bias"]), case["outer"]
    if case["op"] == "int8":
        out, scale = {}, up(s["x_scale"])
        if case["dynamic"]:
            scale = x.abs().max(dim=1).values.clamp(min=AMAX_FLOOR) / I8_MAX
            # a code is the rounded quotient of two float32 numbers, itself a float32 number
            x = torch.round(s["x"].float() / scale.float().unsqueeze(1)).double()
            out.update(q=None, scale=scale)
        z = torch.nn.functional.linear(x, w) * torch.outer(scale, up(s["w_scale"]))
        y = f[case["act"]](z if bias is None else z + bias)
        return dict(out, y=y if s["residual"] is None else y + up(s["residual"]))
    if case["pass"] == "backward":
        z = up(s["preact"]).requires_grad_()
        gate, value = z.chunk(2, dim=1)
        gz, = torch.autograd.grad(f[case["act"]](gate) * value, z, up(s["gy"]))
        out = dict(gx=torch.mm(gz, w), gw=torch.mm(gz.mT, x))
        return dict(out, gbias=gz.sum(0)) if case["bias"] else out
    if s["x_scale"] is not None:
        x, w = x * up(s["x_scale"]).unsqueeze(1), w * up(s["w_scale"]).unsqueeze(1)
    z = torch.nn.functional.linear(x, w, bias)
    gate, value = z.chunk(2, dim=1)
    out = dict(y=f[case["act"]](gate) * value)
    return dict(out, preact=z) if case["pass"] == "keep" else out


def work(case):
    """Each input read once, each output written once; the products' multiplications and additions."""
    size = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "i8": 1}[case["dtype"]]
    if case["op"] == "ortho":
        m, n = sorted((case["rows"], case["cols"]))
        # the smaller side's Gram matrix, its square, and their product with X, as the formula has them
        return dict(bytes=2 * case["batch"] * m * n * size,
                    flops=case["batch"] * case["steps"] * (4 * m * m * n + 2 * m ** 3))
    rows, k, n = case["rows"], case["inner"], case["outer"]
    if case["op"] == "int8":
        x = rows * k * (size + 1 if case["dynamic"] else 1) + 4 * rows
        y = rows * n * size * (1 + int(case["residual"])) + n * size * int(case["bias"])
        return dict(bytes=x + n * k + 4 * n + y, flops=2 * rows * k * n)
    out = max(size, 2)
    moved = rows * k * size + 2 * n * k * size + (4 * (rows + 2 * n) if size == 1 else 0)
    bias = 2 * n * out * int(case["bias"])
    if case["pass"] == "backward":
        # gy and z in; the gradients of x, w and bias out
        return dict(bytes=2 * moved + 3 * rows * n * out + bias, flops=8 * rows * k * n)
    y = rows * n * out * (3 if case["pass"] == "keep" else 1)
    return dict(bytes=moved + bias + y, flops=4 * rows * k * n)
