"""Cases that time and check the layer operators: the RMS norm with the residual's addition, the matrix
product with bias, activation and residual in its epilogue, and their gradients.

listed() gives the cases, draw(rng) one more of the same ranges, prepare(case, seed) the inputs on the GPU, and
run(state) one pass: in elementary torch operations in 32 bits where `own` is false, through
persistent_tiled_gemm_amd where it is true. work(case) is what a pass has to move and compute; exact(case, seed)
is what run returns for these inputs, computed in 64 bits from the definitions:

  norm           s = x + residual;  r = 1 / sqrt(mean_j s^2 + eps);  y = s r weight;
                 e4m3 outputs: scale_m = max_j |y_mj| / 448 (1 where a row is all zeros), codes y / scale
  norm_backward  for a given s, with h = s r and g = dy weight:  dx = r (g - h mean_j(g h)) + dsum,
                 dweight_j = sum_m dy h
  linear         z = x_scale_m w_scale_n sum_k x_mk w_nk + bias_n (scales: e4m3 operands);
                 out = act(z) + residual; pre = z, kept for the gradient
  act_backward   dpre = dout act'(pre);  dbias_n = sum_m dpre (before its rounding)
  linear_backward  dx = dpre w;  dw = dpre^T x (dpre as it is stored, in bf16)
"""

import math

import torch

own = False

EPS = 1e-6
E4M3_MAX = 448.0


def listed():
    return [
        # one token of a decode step on its way into an e4m3 product: latency
        dict(name="norm_token_e4m3", kind="norm", m=1, n=8192, type="bf16", out="e4m3", residual=True, pad=0),
        # a long prefill's residual stream, normed and quantised for the products that follow
        dict(name="norm_prefill_e4m3", kind="norm", m=16384, n=8192, type="bf16", out="e4m3", residual=True, pad=0),
        # a small training batch of ragged size, residual stream in fp32
        dict(name="norm_backward_ragged", kind="norm_backward", m=1111, n=2056, type="f32", out="bf16", residual=True, pad=0),
        # a training step's norm: the stream's own gradient joins here
        dict(name="norm_backward_large", kind="norm_backward", m=8192, n=8192, type="bf16", out="bf16", residual=True, pad=0),
        # one token through a projection with its activation: every weight is read for one row
        dict(name="linear_token", kind="linear", m=1, n=8192, k=8192, type="bf16", out="bf16", act="silu", bias=True,
             residual=False, pre=False, pad=0),
        # a decode batch through an e4m3 projection back onto the residual stream
        dict(name="linear_batch_e4m3", kind="linear", m=24, n=8192, k=8192, type="e4m3", out="bf16", act="none", bias=False,
             residual=True, pre=False, pad=0),
        # a ragged training chunk: every edge lies inside a tile; x is a slice of a wider buffer
        dict(name="linear_ragged", kind="linear", m=1000, n=4104, k=2056, type="bf16", out="bf16", act="gelu", bias=True,
             residual=True, pre=True, pad=64),
        # the 8192^3 product of the benchmark as a training layer's forward pass
        dict(name="linear_square", kind="linear", m=8192, n=8192, k=8192, type="bf16", out="bf16", act="gelu_tanh", bias=True,
             residual=False, pre=True, pad=0),
        # the same size in e4m3 with row scales: prefill
        dict(name="linear_square_e4m3", kind="linear", m=8192, n=8192, k=8192, type="e4m3", out="bf16", act="none", bias=False,
             residual=True, pre=False, pad=0),
        # the activation's and the bias's gradient of a training layer (rows not a multiple of anything)
        dict(name="act_backward", kind="act_backward", m=8191, n=8192, act="gelu_tanh"),
        # both products of a layer's gradient: a ragged small batch, and the benchmark's size
        dict(name="linear_backward_ragged", kind="linear_backward", m=777, n=2056, k=1032),
        dict(name="linear_backward_large", kind="linear_backward", m=8192, n=8192, k=8192),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["norm", "norm_backward", "linear", "linear", "linear", "act_backward", "linear_backward"])
    if kind in ("norm", "norm_backward"):
        m, n = _log(rng, 1, 16384), _log(rng, 512, 16384, 8)
        m = min(m, 16384 * 8192 // n if kind == "norm" else 8192 * 8192 // n)
        return dict(kind=kind, m=m, n=n, type=rng.choice(["bf16", "bf16", "f32"]),
                    out=rng.choice(["e4m3", "e4m3", "bf16", "f32"]) if kind == "norm" else rng.choice(["bf16", "f32"]),
                    residual=rng.random() < 0.75, pad=rng.choice([0, 0, 64]))
    if kind == "act_backward":
        n = _log(rng, 512, 16384, 8)
        return dict(kind=kind, m=min(_log(rng, 1, 16384), 8191 * 8192 // n), n=n,
                    act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]))
    m = _log(rng, 1, 16384)
    if kind == "linear_backward":
        n, k = _log(rng, 256, 16384, 8), _log(rng, 256, 16384, 8)
        return dict(kind=kind, m=max(1, min(m, 8192 ** 3 // (n * k))), n=n, k=k)
    type_ = rng.choice(["bf16", "bf16", "e4m3"])
    step = 16 if type_ == "e4m3" else 8
    n, k = _log(rng, 256, 16384, 8), _log(rng, 256, 16384, step)
    return dict(kind=kind, m=max(1, min(m, 8192 ** 3 // (n * k))), n=n, k=k, type=type_, out=rng.choice(["bf16", "bf16", "f32"]),
                act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.6,
                residual=rng.random() < 0.5, pre=type_ == "bf16" and rng.random() < 0.4, pad=rng.choice([0, 0, 64]))


TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}
SIZES = {"f32": 4, "bf16": 2, "e4m3": 1}


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def padded(t):
        # the row slice of a wider buffer, as a fused projection's part is
        if not case["pad"]:
            return t
        wide = torch.zeros(t.shape[0], t.shape[1] + case["pad"], dtype=t.dtype, device="cuda")
        wide[:, : t.shape[1]] = t
        return wide[:, : t.shape[1]]

    def quantised(t):
        # per-row scales, as the norm writes them for activations and a loader for weights
        scale = t.abs().amax(dim=1) / E4M3_MAX
        return (t / scale[:, None]).to(torch.float8_e4m3fn), scale

    kind, m, n = case["kind"], case["m"], case["n"]
    s = {"case": case}
    if kind in ("norm", "norm_backward"):
        t = TYPES[case["type"]]
        # a residual stream: most channels of order one, a few far larger
        x = normal(m, n)
        x[:, :: 509] *= 20.0
        s["x"] = padded(x.to(t))
        s["weight"] = (1.0 + 0.1 * normal(n)).to(torch.bfloat16)
        if kind == "norm":
            s["residual"] = normal(m, n).to(t) if case["residual"] else None
        else:
            s["dy"] = normal(m, n).to(TYPES[case["out"]])
            s["dsum"] = normal(m, n).to(t) if case["residual"] else None
    elif kind == "act_backward":
        s["dout"] = normal(m, n).to(torch.bfloat16)
        s["pre"] = normal(m, n).to(torch.bfloat16)
    elif kind == "linear_backward":
        k = case["k"]
        s["dpre"] = (0.1 * normal(m, n)).to(torch.bfloat16)
        s["x"] = normal(m, k).to(torch.bfloat16)
        s["w"] = (normal(n, k) / math.sqrt(k)).to(torch.bfloat16)
    else:
        k = case["k"]
        x, w = normal(m, k), normal(n, k) / math.sqrt(k)
        s["x_scale"] = s["w_scale"] = None
        if case["type"] == "e4m3":
            x, s["x_scale"] = quantised(x)
            s["w"], s["w_scale"] = quantised(w)
            s["x"] = padded(x)
        else:
            s["x"], s["w"] = padded(x.to(torch.bfloat16)), w.to(torch.bfloat16)
        s["bias"] = (0.5 * normal(n)).to(torch.bfloat16) if case["bias"] else None
        s["residual"] = normal(m, n).to(torch.bfloat16) if case["residual"] else None
    if own:
        import persistent_tiled_gemm_amd as ptg

        s["ptg"], s["plan"] = ptg, _plan(ptg)

        def empty(t, *shape):
            return torch.empty(*shape, dtype=t, device="cuda")

        if kind == "norm":
            s["sum"] = empty(t, m, n) if case["residual"] else None
            s["out"] = empty(TYPES[case["out"]], m, n)
            s["scale"] = empty(torch.float32, m) if case["out"] == "e4m3" else None
        elif kind == "norm_backward":
            s["dx"], s["dweight"] = empty(t, m, n), empty(torch.float32, n)
        elif kind == "act_backward":
            s["grad"], s["dbias"] = empty(torch.bfloat16, m, n), empty(torch.float32, n)
        elif kind == "linear_backward":
            s["dx"], s["dw"] = empty(torch.bfloat16, m, k), empty(torch.float32, n, k)
        else:
            s["out"] = empty(TYPES[case["out"]], m, n)
            s["z"] = empty(torch.bfloat16, m, n) if case["pre"] else None
    return s


_kept = []


def _plan(ptg):
    """The plan that a program makes once and keeps."""
    if not _kept:
        _kept.append(ptg.layer_create())
    return _kept[0]


def run(state):
    s, case = state, state["case"]
    if own:
        return _run_own(s, case)
    kind = case["kind"]
    if kind == "norm":
        x = s["x"].float()
        if s["residual"] is not None:
            x = x + s["residual"].float()
        r = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
        y = x * r * s["weight"].float()
        out = {}
        if s["residual"] is not None:
            out["sum"] = x.to(s["x"].dtype)
        if case["out"] == "e4m3":
            amax = y.abs().amax(dim=1)
            scale = torch.where(amax == 0, torch.ones_like(amax), amax / E4M3_MAX)
            out["out"], out["scale"] = (y / scale[:, None]).to(torch.float8_e4m3fn), scale
        else:
            out["out"] = y.to(TYPES[case["out"]])
        return out
    if kind == "norm_backward":
        x, dy = s["x"].float(), s["dy"].float()
        r = torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS)
        h, g = x * r, dy * s["weight"].float()
        dx = r * (g - h * (g * h).mean(dim=1, keepdim=True))
        if s["dsum"] is not None:
            dx = dx + s["dsum"].float()
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * h).sum(dim=0)}
    if kind == "act_backward":
        d = s["dout"].float() * _plain_grad(s["pre"].float(), case["act"])
        return {"dpre": d.to(torch.bfloat16), "dbias": d.sum(dim=0)}
    if kind == "linear_backward":
        d = s["dpre"].float()
        return {"dx": torch.matmul(d, s["w"].float()).to(torch.bfloat16), "dw": torch.matmul(d.t(), s["x"].float())}
    z = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["x_scale"] is not None:
        z = z * s["x_scale"][:, None] * s["w_scale"][None, :]
    if s["bias"] is not None:
        z = z + s["bias"].float()
    y = _plain_act(z, case["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    out = {"out": y.to(TYPES[case["out"]])}
    if case["pre"]:
        out["pre"] = z.to(torch.bfloat16)
    return out


def _plain_act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return z / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _plain_grad(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        c = math.sqrt(2.0 / math.pi)
        p = 1.0 / (1.0 + torch.exp(-2.0 * c * (z + 0.044715 * z * z * z)))
        return p + 2.0 * c * z * (1.0 + 3 * 0.044715 * z * z) * p * (1.0 - p)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-z))
        return p + z * p * (1.0 - p)
    return torch.ones_like(z)


def _run_own(s, case):
    ptg, plan, kind = s["ptg"], s["plan"], case["kind"]
    if kind == "norm":
        ptg.layer_rmsnorm(s["x"], s["weight"], s["out"], residual=s["residual"], sum_out=s["sum"], scale=s["scale"], eps=EPS)
        out = {"out": s["out"]}
        if s["sum"] is not None:
            out["sum"] = s["sum"]
        if s["scale"] is not None:
            out["scale"] = s["scale"]
        return out
    if kind == "norm_backward":
        ptg.layer_rmsnorm_backward(s["dy"], s["x"], s["weight"], s["dx"], s["dweight"], plan, dsum=s["dsum"], eps=EPS)
        return {"dx": s["dx"], "dweight": s["dweight"]}
    if kind == "act_backward":
        ptg.layer_activation_backward(s["dout"], s["pre"], s["grad"], plan, activation=case["act"], dbias=s["dbias"])
        return {"dpre": s["grad"], "dbias": s["dbias"]}
    if kind == "linear_backward":
        ptg.layer_linear_backward(s["dpre"], s["x"], s["w"], plan, dx=s["dx"], dw=s["dw"])
        return {"dx": s["dx"], "dw": s["dw"]}
    ptg.layer_linear(s["x"], s["w"], s["out"], plan, bias=s["bias"], activation=case["act"], residual=s["residual"], pre=s["z"],
                     x_scale=s["x_scale"], w_scale=s["w_scale"])
    return {"out": s["out"], "pre": s["z"]} if case["pre"] else {"out": s["out"]}


def work(case):
    kind, m, n = case["kind"], case["m"], case["n"]
    if kind == "norm":
        moved = m * n * (SIZES[case["type"]] * (3 if case["residual"] else 1) + SIZES[case["out"]])
        return {"bytes": moved + 2 * n + (4 * m if case["out"] == "e4m3" else 0), "flops": 5 * m * n}
    if kind == "norm_backward":
        return {"bytes": m * n * (SIZES[case["type"]] * (3 if case["residual"] else 2) + SIZES[case["out"]]) + 6 * n,
                "flops": 10 * m * n}
    if kind == "act_backward":
        return {"bytes": 6 * m * n + 4 * n, "flops": 10 * m * n}
    k = case["k"]
    if kind == "linear_backward":
        return {"bytes": 2 * m * n + 2 * m * k + 2 * n * k + 2 * m * k + 4 * n * k, "flops": 4 * m * n * k}
    size = SIZES[case["type"]]
    moved = size * (m * k + n * k) + m * n * (SIZES[case["out"]] + (2 if case["residual"] else 0) + (2 if case["pre"] else 0))
    return {"bytes": moved + (2 * n if case["bias"] else 0) + (4 * (m + n) if size == 1 else 0), "flops": 2 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]

    def d(name):
        return None if s[name] is None else s[name].to(torch.float64)

    if kind == "norm":
        v = d("x") if s["residual"] is None else d("x") + d("residual")
        y = v / (v.square().sum(dim=1, keepdim=True) / case["n"] + EPS).sqrt() * d("weight")
        out = {} if s["residual"] is None else {"sum": v}
        if case["out"] != "e4m3":
            return {**out, "out": y}
        top = y.abs().max(dim=1).values
        top[top == 0] = E4M3_MAX
        return {**out, "out": y * E4M3_MAX / top[:, None], "scale": top / E4M3_MAX}
    if kind == "norm_backward":
        x, dy, w = d("x"), d("dy"), d("weight")
        ms = x.square().sum(dim=1, keepdim=True) / case["n"] + EPS
        # d/dx of x / sqrt(ms), row by row: the quotient rule
        dx = dy * w / ms.sqrt() - x * (dy * w * x).sum(dim=1, keepdim=True) / (case["n"] * ms * ms.sqrt())
        return {"dx": dx if s["dsum"] is None else dx + d("dsum"), "dweight": (dy * x / ms.sqrt()).sum(dim=0)}
    if kind == "act_backward":
        z = d("pre").requires_grad_(True)
        _exact_act(z, case["act"]).backward(d("dout"))
        return {"dpre": z.grad, "dbias": z.grad.sum(dim=0)}
    if kind == "linear_backward":
        return {"dx": d("dpre") @ d("w"), "dw": d("dpre").t().contiguous() @ d("x")}
    z = d("x") @ d("w").t()
    if s["x_scale"] is not None:
        z = z * torch.outer(d("x_scale"), d("w_scale"))
    if s["bias"] is not None:
        z = z + d("bias")
    y = _exact_act(z, case["act"])
    out = {"out": y if s["residual"] is None else y + d("residual")}
    return {**out, "pre": z} if case["pre"] else out


def _exact_act(z, act):
    if act == "relu":
        return z.clamp(min=0)
    if act == "gelu":
        return z * torch.special.erfc(-z / math.sqrt(2.0)) / 2
    if act == "gelu_tanh":
        return z / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)))
    if act == "silu":
        return z * torch.sigmoid(z)
    return z * 1
