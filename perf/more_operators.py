"""Cases that time and check the operators at a layer stack's two ends: 8-bit integer rows and the product of them, with which
a trained layer is served, and the softmax cross entropy of an output head and its gradient, with which it is trained, without
the logits ever being kept.

listed() gives the cases, draw(rng) one more of the same ranges, prepare(case, seed) the inputs on the GPU, and run(state) one
pass: in elementary torch operations in 32 bits where `own` is false, through persistent_tiled_gemm_amd where it is true.
work(case) is what a pass has to move and compute; exact(case, seed) is what run returns for these inputs, computed in 64 bits
from the definitions:

  quantize       scale_m = max_j |x_mj| / top (1 where a row is all zeros), top = 127 for int8 and 448 for e4m3, the fp32
                 quotient; codes x / scale, the fp32 quotient rounded to nearest, ties to even
  linear         z = x_scale_m w_scale_n sum_k x_mk w_nk + bias_n with x and w in int8;  out = act(z) + residual;
                 pre = z, kept for the gradient
  loss           z = x w^T (a row for each token, a column for each of the vocabulary's n entries);  lse_m = log sum_v exp z_mv;
                 loss_m = lse_m - z_m,label, 0 where the label is negative
  loss_backward  of dloss sum_m weight_m loss_m at a given lse:  dz_mv = dloss weight_m (exp(z_mv - lse_m) - [v = label_m]), 0
                 where the label is negative;  dx = dz w;  dw = dz^T x
"""

import math

import torch

own = False

TOP = {"i8": 127.0, "e4m3": 448.0}


def listed():
    return [
        # one token's activations on their way into an int8 product: latency
        dict(name="quantize_token", kind="quantize", m=1, n=8192, type="bf16", out="i8", pad=0),
        # a ragged chunk's activations from fp32, a column slice of a wider buffer, into e4m3 rows
        dict(name="quantize_ragged_e4m3", kind="quantize", m=1111, n=10248, type="f32", out="e4m3", pad=64),
        # a long prefill's activations
        dict(name="quantize_prefill", kind="quantize", m=16384, n=8192, type="bf16", out="i8", pad=0),
        # one token through a projection with its activation: every weight is read for one row
        dict(name="linear_token", kind="linear", m=1, n=8192, k=8192, out="bf16", act="silu", bias=True, residual=False, pre=False,
             pad=0),
        # a decode batch through a projection back onto the residual stream
        dict(name="linear_batch", kind="linear", m=24, n=8192, k=8192, out="bf16", act="none", bias=False, residual=True, pre=False,
             pad=0),
        # a ragged chunk: every edge lies inside a tile; x is a slice of a wider buffer
        dict(name="linear_ragged", kind="linear", m=1000, n=4104, k=2064, out="bf16", act="gelu", bias=True, residual=True, pre=True,
             pad=64),
        # the benchmark's 8192^3 product as prefill
        dict(name="linear_square", kind="linear", m=8192, n=8192, k=8192, out="bf16", act="none", bias=False, residual=True,
             pre=False, pad=0),
        # four tokens' log-probabilities: every row of the head is read for them
        dict(name="loss_tokens", kind="loss", m=4, n=32768, k=4096),
        # an evaluation chunk of ragged size
        dict(name="loss_ragged", kind="loss", m=1000, n=50264, k=2056),
        # a training step's loss over a large vocabulary
        dict(name="loss_large", kind="loss", m=4096, n=131072, k=4096),
        # the gradient of a ragged small batch, every row with a weight of its own
        dict(name="loss_backward_ragged", kind="loss_backward", m=777, n=20008, k=1032, weight=True),
        # a training step's gradient over a large vocabulary
        dict(name="loss_backward_large", kind="loss_backward", m=4096, n=131072, k=4096, weight=False),
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of `step` between lo and hi, spread evenly over its logarithm."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(v / step)) * step))


def draw(rng):
    kind = rng.choice(["quantize", "linear", "linear", "loss", "loss_backward"])
    if kind == "quantize":
        m, n = _log(rng, 1, 16384), _log(rng, 512, 65536, 8)
        type_ = rng.choice(["bf16", "bf16", "f32"])
        return dict(kind=kind, m=max(1, min(m, 16384 * 8192 // n // (2 if type_ == "f32" else 1))), n=n, type=type_,
                    out=rng.choice(["i8", "i8", "e4m3"]), pad=rng.choice([0, 0, 64]))
    if kind == "linear":
        m, n, k = _log(rng, 1, 16384), _log(rng, 256, 16384, 8), _log(rng, 256, 16384, 16)
        return dict(kind=kind, m=max(1, min(m, 8192 ** 3 // (n * k))), n=n, k=k, out=rng.choice(["bf16", "bf16", "f32"]),
                    act=rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]), bias=rng.random() < 0.6,
                    residual=rng.random() < 0.5, pre=rng.random() < 0.3, pad=rng.choice([0, 0, 64]))
    n, k = _log(rng, 2048, 131072, 8), _log(rng, 512, 8192, 8)
    m = min(_log(rng, 1 if kind == "loss" else 128, 16384), 4096 * 4096 * 131072 // (n * k))
    if kind == "loss":
        return dict(kind=kind, m=m, n=n, k=k)
    return dict(kind=kind, m=m, n=n, k=k, weight=rng.random() < 0.4)


TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "i8": torch.int8}
SIZES = {"f32": 4, "bf16": 2, "e4m3": 1, "i8": 1}


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

    def whole(t):
        # integer rows with their scales
        scale = t.abs().amax(dim=1) / 127
        return (t / scale[:, None]).round().clamp(-127, 127).to(torch.int8), scale

    kind, m, n = case["kind"], case["m"], case["n"]
    s = {"case": case}
    if kind == "quantize":
        # activations: most channels of order one, a few far larger
        x = normal(m, n)
        x[:, :: 509] *= 20.0
        s["x"] = padded(x.to(TYPES[case["type"]]))
    elif kind == "linear":
        k = case["k"]
        x, s["x_scale"] = whole(normal(m, k))
        s["x"] = padded(x)
        s["w"], s["w_scale"] = whole(normal(n, k) / math.sqrt(k))
        s["bias"] = (0.5 * normal(n)).to(torch.bfloat16) if case["bias"] else None
        s["residual"] = normal(m, n).to(torch.bfloat16) if case["residual"] else None
    else:
        # logits of standard deviation 2, and labels between unpredictable (their logit like any other) and sure (14 above)
        k = case["k"]
        w = (2.0 / math.sqrt(k)) * normal(n, k)
        label = torch.randint(0, n, (m,), generator=g, device="cuda")
        lift = 14.0 * torch.rand(m, generator=g, device="cuda")
        s["x"] = (normal(m, k) + (lift / 4.0)[:, None] * w[label]).to(torch.bfloat16)
        s["w"] = w.to(torch.bfloat16)
        # a tenth of the rows is not counted: a prompt's, or padding
        label[torch.rand(m, generator=g, device="cuda") < 0.1] = -100
        s["label"] = label
        if kind == "loss_backward":
            s["lse"] = torch.cat([torch.logsumexp(torch.matmul(r.float(), s["w"].float().t()), dim=1) for r in s["x"].split(1024)])
            s["weight"] = 0.5 + torch.rand(m, generator=g, device="cuda") if case["weight"] else None
            # the mean over the counted rows
            s["dloss"] = 1.0 / (label >= 0).sum().clamp(min=1).float()
    if own:
        import persistent_tiled_gemm_amd as ptg

        s["ptg"], s["plan"] = ptg, _plan(ptg)

        def empty(t, *shape):
            return torch.empty(*shape, dtype=t, device="cuda")

        if kind == "quantize":
            s["out"], s["scale"] = empty(TYPES[case["out"]], m, n), empty(torch.float32, m)
        elif kind == "linear":
            s["out"] = empty(TYPES[case["out"]], m, n)
            s["z"] = empty(torch.bfloat16, m, n) if case["pre"] else None
        elif kind == "loss":
            s["loss"], s["lse"] = empty(torch.float32, m), empty(torch.float32, m)
        else:
            s["dx"], s["dw"] = empty(torch.bfloat16, m, k), empty(torch.bfloat16, n, k)
            s["scratch"] = empty(torch.uint8, ptg.layer_cross_entropy_scratch(m, n, k, pieces=-(-n // 16384)))
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
    if kind == "quantize":
        x = s["x"].float()
        amax = x.abs().amax(dim=1)
        # (a tensor as the divisor: by a number, torch multiplies with its reciprocal, a step of fp32 off now and then)
        scale = torch.where(amax == 0, torch.ones_like(amax), amax / torch.full_like(amax, TOP[case["out"]]))
        q = x / scale[:, None]
        return {"out": q.round().to(torch.int8) if case["out"] == "i8" else q.to(torch.float8_e4m3fn), "scale": scale}
    if kind == "linear":
        z = torch.matmul(s["x"].float(), s["w"].float().t()) * s["x_scale"][:, None] * s["w_scale"][None, :]
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _plain_act(z, case["act"])
        if s["residual"] is not None:
            y = y + s["residual"].float()
        out = {"out": y.to(TYPES[case["out"]])}
        if case["pre"]:
            out["pre"] = z.to(torch.bfloat16)
        return out
    counted = s["label"] >= 0
    at = torch.where(counted, s["label"], torch.zeros_like(s["label"]))[:, None]
    z = torch.matmul(s["x"].float(), s["w"].float().t())
    if kind == "loss":
        top = z.amax(dim=1)
        lse = top + torch.log(torch.exp(z - top[:, None]).sum(dim=1))
        return {"loss": torch.where(counted, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse)), "lse": lse}
    g = s["dloss"] * (counted.float() if s["weight"] is None else torch.where(counted, s["weight"], torch.zeros_like(s["weight"])))
    dz = torch.exp(z - s["lse"][:, None])
    dz.scatter_add_(1, at, -torch.ones_like(dz[:, :1]))
    dz = dz * g[:, None]
    return {"dx": torch.matmul(dz, s["w"].float()).to(torch.bfloat16), "dw": torch.matmul(dz.t(), s["x"].float()).to(torch.bfloat16)}


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


def _run_own(s, case):
    ptg, plan, kind = s["ptg"], s["plan"], case["kind"]
    if kind == "quantize":
        ptg.layer_quantize(s["x"], s["out"], s["scale"])
        return {"out": s["out"], "scale": s["scale"]}
    if kind == "linear":
        ptg.layer_linear(s["x"], s["w"], s["out"], plan, bias=s["bias"], activation=case["act"], residual=s["residual"], pre=s["z"],
                         x_scale=s["x_scale"], w_scale=s["w_scale"])
        return {"out": s["out"], "pre": s["z"]} if case["pre"] else {"out": s["out"]}
    if kind == "loss":
        ptg.layer_cross_entropy(s["x"], s["w"], s["label"], s["lse"], plan, loss=s["loss"])
        return {"loss": s["loss"], "lse": s["lse"]}
    ptg.layer_cross_entropy_backward(s["x"], s["w"], s["label"], s["lse"], s["scratch"], plan, dx=s["dx"], dw=s["dw"],
                                     weight=s["weight"], dloss=s["dloss"])
    return {"dx": s["dx"], "dw": s["dw"]}


def work(case):
    kind, m, n = case["kind"], case["m"], case["n"]
    if kind == "quantize":
        return {"bytes": m * n * (SIZES[case["type"]] + 1) + 4 * m, "flops": 2 * m * n}
    k = case["k"]
    if kind == "linear":
        moved = m * k + n * k + m * n * (SIZES[case["out"]] + (2 if case["residual"] else 0) + (2 if case["pre"] else 0))
        return {"bytes": moved + (2 * n if case["bias"] else 0) + 4 * (m + n), "flops": 2 * m * n * k}
    if kind == "loss":
        return {"bytes": 2 * k * (m + n) + 16 * m, "flops": 2 * m * n * k}
    # the logits are computed again, and both products
    return {"bytes": 4 * k * (m + n) + (16 if case["weight"] else 12) * m + 4, "flops": 6 * m * n * k}


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]

    def d(name):
        return None if s[name] is None else s[name].to(torch.float64)

    if kind == "quantize":
        # the codes are defined by the fp32 quotient
        top = d("x").abs().max(dim=1).values
        top[top == 0] = TOP[case["out"]]
        scale = top / TOP[case["out"]]
        return {"out": None if case["out"] == "i8" else d("x") / scale[:, None], "scale": scale}
    if kind == "linear":
        z = (d("x") @ d("w").t()) * torch.outer(d("x_scale"), d("w_scale"))
        if s["bias"] is not None:
            z = z + d("bias")
        y = _exact_act(z, case["act"])
        out = {"out": y if s["residual"] is None else y + d("residual")}
        return {**out, "pre": z} if case["pre"] else out
    # rows in pieces: 64-bit logits of the largest case would take 8 bytes for each of its 2^29
    w, count = d("w"), (s["label"] >= 0)
    if kind == "loss":
        lse, loss = [], []
        for x, label in zip(d("x").split(1024), s["label"].split(1024)):
            z = x @ w.t()
            lse.append(z.logsumexp(dim=1))
            loss.append(lse[-1] - z[torch.arange(len(label), device=z.device), label.clamp(min=0)])
        return {"loss": torch.cat(loss) * count, "lse": torch.cat(lse)}
    g = d("dloss") * count * (1.0 if s["weight"] is None else d("weight"))
    dx, dw = [], torch.zeros_like(w)
    for x, label, lse, r in zip(d("x").split(1024), s["label"].split(1024), d("lse").split(1024), g.split(1024)):
        p = (x @ w.t() - lse[:, None]).exp()
        p[torch.arange(len(label), device=p.device), label.clamp(min=0)] -= 1
        p *= r[:, None]
        dx.append(p @ w)
        dw += p.t().contiguous() @ x
    return {"dx": torch.cat(dx), "dw": dw}


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
