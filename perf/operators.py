"""Cases of the 8-bit activation operators: the 8-bit form itself (pack and
unpack), layer norm forward and backward (from the input or from its 8-bit
form), the linear layer's product in 8-bit integers and its weight gradient
from the 8-bit form.

A case is a dict of plain values: ``op`` picks the operator, ``rows`` x
``cols`` is the activation matrix (tokens x features), ``out`` the linear
layer's output features, ``group`` the columns that share a step (0: the
row), ``dtype`` the activations' type.  ``run`` computes the operators in
plain torch operations, or calls the library's entry points where ``own`` is
true; ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
EPS = 1e-5
MOST_FLOPS = 2.0 * 16384 * 4096 * 4096      # the largest listed product
MOST_ELEMENTS = 16384 * 4096                # the largest listed activation


def listed():
    return [
        # the 8-bit form of a few tokens, kept between steps: latency
        dict(name="round_trip_few_tokens", op="round_trip", rows=16, cols=1024,
             group=128, dtype="bf16"),
        # a layer's activations checkpointed in 8 bits and expanded again
        dict(name="round_trip_batch", op="round_trip", rows=16384, cols=4096,
             group=128, dtype="bf16"),
        # inference on one sequence of a few tokens
        dict(name="norm_few_tokens", op="norm", rows=16, cols=1024, group=0,
             dtype="bf16"),
        # fp16 training on a ragged batch, odd width, input kept as it is
        dict(name="norm_step_odd", op="norm_step", rows=1531, cols=1001,
             group=0, dtype="f16", packed=False),
        # fp32 training, input kept as it is
        dict(name="norm_step_f32", op="norm_step", rows=4096, cols=2048,
             group=0, dtype="f32", packed=False),
        # a training step's norm whose input is kept in 8 bits only
        dict(name="norm_step_packed", op="norm_step", rows=16384, cols=4096,
             group=128, dtype="bf16", packed=True),
        # weight gradient of a narrow layer: few output tiles, long sums
        dict(name="wgrad_narrow", op="wgrad", rows=8192, cols=1024, out=1024,
             group=128, dtype="bf16"),
        # weight gradient of a wide layer over a long batch
        dict(name="wgrad_wide", op="wgrad", rows=16384, cols=4096, out=4096,
             group=0, dtype="bf16"),
        # fp16 gradient, ragged token count, odd features
        dict(name="wgrad_odd", op="wgrad", rows=2027, cols=1001, out=1531,
             group=64, dtype="f16"),
        # one token through a wide layer: serving
        dict(name="linear_one_token", op="linear", rows=1, cols=4096, out=4096,
             group=0, dtype="bf16"),
        # a ragged serving batch through odd features
        dict(name="linear_ragged", op="linear", rows=203, cols=4100, out=2050,
             group=0, dtype="f16"),
        # a training batch through a wide layer
        dict(name="linear_batch", op="linear", rows=8192, cols=4096, out=8192,
             group=0, dtype="bf16"),
    ]


def draw(rng):
    def spread(lo, hi):
        v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
        form = rng.random()
        if form < 0.35 and v >= 128:
            v = v // 64 * 64
        elif form < 0.7:
            v |= 1
        return max(lo, min(hi, v))

    while True:
        op = rng.choice(("round_trip", "norm", "norm_step", "wgrad", "linear"))
        c = dict(op=op, rows=spread(1, 16384), cols=spread(64, 8192), group=0,
                 dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
        if op in ("round_trip", "wgrad") or (op == "norm_step" and rng.random() < 0.7):
            c["group"] = rng.choice((0, 32, 64, 128, 256, 512, 1024))
        if op == "norm_step":
            c["packed"] = rng.random() < 0.6
        if op in ("wgrad", "linear"):
            c["out"] = spread(64, 8192)
        if (c["rows"] * c["cols"] <= MOST_ELEMENTS
                and 2.0 * c["rows"] * c["cols"] * c.get("out", 0) <= MOST_FLOPS
                and work(c)["bytes"] <= work(listed()[5])["bytes"]):
            return c


def work(case):
    r, c, e = case["rows"], case["cols"], SIZE[case["dtype"]]
    o, groups = case.get("out", 0), -(-c // (case["group"] or c))
    form = r * c + 4 * r * groups               # an 8-bit form: codes, steps
    if case["op"] == "round_trip":              # x in, form out; form in, x^ out
        return {"bytes": 2 * e * r * c + 2 * form, "flops": 4 * r * c}
    if case["op"] == "norm":
        return {"bytes": 2 * e * r * c + 8 * (c + r), "flops": 8 * r * c}
    if case["op"] == "norm_step":
        # x in, y out, dy in, dx out; the kept input out and in, or in again
        kept = 2 * form if case["packed"] else e * r * c
        return {"bytes": 4 * e * r * c + kept + 16 * r + 20 * c, "flops": 22 * r * c}
    if case["op"] == "wgrad":
        return {"bytes": e * r * o + form + 4 * o * (c + 1), "flops": 2.0 * r * c * o}
    return {"bytes": e * r * (c + o) + o * c + 8 * o, "flops": 2.0 * r * c * o}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r, c, t = case["rows"], case["cols"], DTYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    # activations: features of very different size, as in trained networks
    x = (normal(r, c) * torch.exp(normal(c)) + 0.1 * normal(c)).to(t)
    s = dict(case=case, x=x)
    if case["op"] in ("norm", "norm_step"):
        s["weight"] = 1.0 + 0.2 * normal(c)
        s["bias"] = 0.2 * normal(c)
    if case["op"] == "norm_step":
        s["dy"] = (normal(r, c) * 1e-2).to(t)
    if case["op"] == "wgrad":
        s["dy"] = (normal(r, case["out"]) * 1e-2).to(t)
        # the 8-bit form that the forward pass kept: codes in rows of
        # 16-byte pitch, zero behind the last column
        s["codes"], s["steps"] = _form(x, case["group"])
        del s["x"]
    if case["op"] == "linear":
        o = case["out"]
        s["w_codes"], s["w_steps"] = _form(normal(o, c) / math.sqrt(c), 0)
        s["bias"] = 0.1 * normal(o)
    return s


# ------------------------------------------------------------ plain form ----
def _steps(x, group):
    """Power-of-two step of each group: [rows, groups] in 32 bits."""
    r, c = x.shape
    g = group or c
    n = -(-c // g)
    a = torch.zeros(r, n * g, device=x.device)
    a[:, :c] = x.abs()
    m = a.view(r, n, g).amax(-1)
    frac, e = torch.frexp(m)                    # m = frac 2^e, frac in [1/2, 1)
    e = torch.where(frac <= 127 / 128, e - 7, e - 6).clamp(min=-126)
    step = ((e + 127) << 23).view(torch.float32)    # 2^e, exact
    return torch.where(m > 0, step, 0.0)


def _spread(steps, c, group):
    return steps.repeat_interleave(group or c, dim=1)[:, :c]


def _codes(x, steps, group):
    """round(x / step), ties to even, as fp32."""
    s = _spread(steps, x.shape[1], group)
    return torch.where(s > 0, torch.round(x / torch.where(s > 0, s, 1.0)), 0.0)


def _form(x, group):
    x = x.float()
    steps = _steps(x, group)
    r, c = x.shape
    codes = torch.zeros(r, -(-c // 16) * 16, dtype=torch.int8, device=x.device)
    codes[:, :c] = _codes(x, steps, group).to(torch.int8)
    return codes, steps


def _norm(x, weight, bias):
    mean = x.mean(1, keepdim=True)
    d = x - mean
    rstd = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
    return d * rstd * weight + bias, mean, rstd


def _norm_backward(dy, x, mean, rstd, weight):
    xh = (x - mean) * rstd
    a = dy * weight
    dx = rstd * (a - a.mean(1, keepdim=True) - xh * (a * xh).mean(1, keepdim=True))
    return dx, (dy * xh).sum(0), dy.sum(0)


def _plain(s):
    case = s["case"]
    op, group, t = case["op"], case["group"], DTYPES[case["dtype"]]
    if op == "round_trip":
        x = s["x"].float()
        steps = _steps(x, group)
        back = _codes(x, steps, group) * _spread(steps, x.shape[1], group)
        return {"x": back.to(t), "steps": steps}
    if op == "norm":
        return {"y": _norm(s["x"].float(), s["weight"], s["bias"])[0].to(t)}
    if op == "norm_step":
        x = s["x"].float()
        y, mean, rstd = _norm(x, s["weight"], s["bias"])
        if case["packed"]:
            steps = _steps(x, group)
            x = _codes(x, steps, group) * _spread(steps, x.shape[1], group)
        dx, dw, db = _norm_backward(s["dy"].float(), x, mean, rstd, s["weight"])
        return {"y": y.to(t), "mean": mean[:, 0], "rstd": rstd[:, 0],
                "dx": dx.to(t), "dweight": dw, "dbias": db}
    if op == "wgrad":
        c = case["cols"]
        x = s["codes"][:, :c].float() * _spread(s["steps"], c, group)
        dy = s["dy"].float()
        return {"dweight": dy.t().contiguous() @ x, "dbias": dy.sum(0)}
    x = s["x"].float()
    steps = _steps(x, 0)
    acc = _codes(x, steps, 0) @ s["w_codes"][:, :case["cols"]].float().t()
    return {"y": (acc * steps * s["w_steps"].view(1, -1) + s["bias"]).to(t)}


# ------------------------------------------------------- the library's calls ----
def _own(s):
    from communication_efficient_gradient_amd import gq

    case = s["case"]
    op = case["op"]
    r, c, o, t = case["rows"], case["cols"], case.get("out", 0), DTYPES[case["dtype"]]
    if "keep" not in s:     # the buffers a program holds from step to step
        k = s["keep"] = {"act": gq.act(r, c, t, case["group"])}

        def new(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        if op in ("round_trip", "linear") or (op == "norm_step" and case["packed"]):
            k["codes"], k["steps"] = gq.alloc_act(k["act"])
        if op == "round_trip":
            k["back"] = new(r, c, dtype=t)
        if op in ("norm", "norm_step"):
            k["y"] = new(r, c, dtype=t)
        if op == "norm_step":
            k["dx"] = new(r, c, dtype=t)
            k["mean"], k["rstd"], k["dw"], k["db"] = new(r), new(r), new(c), new(c)
            k["ws"] = gq.alloc_workspace(gq.gq_layer_norm_workspace(k["act"]))
        if op == "wgrad":
            k["dw"], k["db"] = new(o, c), new(o)
            k["ws"] = gq.alloc_workspace(gq.gq_act_wgrad_workspace(k["act"], o))
        if op == "linear":
            k["y"] = new(r, o, dtype=t)
            k["ws"] = gq.alloc_workspace(gq.gq_act_linear_workspace(k["act"], o))
    k = s["keep"]
    a = k["act"]
    if op == "round_trip":
        gq.gq_act_pack(a, s["x"], k["codes"], k["steps"])
        gq.gq_act_unpack(a, k["codes"], k["steps"], k["back"])
        return {"x": k["back"], "steps": k["steps"]}
    if op == "norm":
        gq.gq_layer_norm(a, s["x"], s["weight"], s["bias"], EPS, k["y"])
        return {"y": k["y"]}
    if op == "norm_step":
        x_form = (k["codes"], k["steps"]) if case["packed"] else None
        gq.gq_layer_norm(a, s["x"], s["weight"], s["bias"], EPS, k["y"],
                         mean=k["mean"], rstd=k["rstd"], x_form=x_form)
        gq.gq_layer_norm_backward(
            a, s["dy"], x_form if case["packed"] else s["x"], k["mean"], k["rstd"],
            s["weight"], k["dx"], k["dw"], k["db"], workspace=k["ws"])
        return {"y": k["y"], "mean": k["mean"], "rstd": k["rstd"],
                "dx": k["dx"], "dweight": k["dw"], "dbias": k["db"]}
    if op == "wgrad":
        gq.gq_act_wgrad(a, s["dy"], s["codes"], s["steps"], k["dw"], k["db"],
                        workspace=k["ws"])
        return {"dweight": k["dw"], "dbias": k["db"]}
    gq.gq_act_pack(a, s["x"], k["codes"], k["steps"])
    gq.gq_act_linear(a, k["codes"], k["steps"], s["w_codes"], s["w_steps"],
                     s["bias"], k["y"], workspace=k["ws"])
    return {"y": k["y"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- 64 bits ----
def _power64(e):
    """2^e, exact (a library's pow may be off by its last bit)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _form64(x, group):
    """x^ of the 8-bit form in 64 bits, by halving and doubling trial steps
    from an estimate: 127 step >= max|x| > 127 step / 2."""
    r, c = x.shape
    back, steps = torch.empty_like(x), []
    for lo in range(0, c, group or c):
        part = x[:, lo:lo + (group or c)]
        m = part.abs().max(1).values
        e = torch.floor(torch.log2(torch.where(m > 0, m, 1.0) / 127.0))
        for _ in range(3):
            e = torch.where(127.0 * _power64(e) < m, e + 1, e)
            e = torch.where(127.0 * _power64(e - 1) >= m, e - 1, e)
        step = torch.where(m > 0, _power64(e.clamp(min=-126)), 0.0)
        q = part / torch.where(m > 0, step, 1.0)[:, None]
        low = torch.floor(q)
        rest = q - low
        up = (rest > 0.5) | ((rest == 0.5) & (low % 2 != 0))
        back[:, lo:lo + (group or c)] = (low + up) * step[:, None]
        steps.append(step)
    return back, torch.stack(steps, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op, group, c = case["op"], case["group"], case["cols"]
    x = s["x"].double() if "x" in s else None
    if op == "round_trip":
        back, steps = _form64(x, group)
        return {"x": back, "steps": steps}
    if op in ("norm", "norm_step"):
        w, b = s["weight"].double(), s["bias"].double()
        var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
        rstd = 1.0 / torch.sqrt(var + EPS)
        y = torch.addcmul(b, (x - mean) / torch.sqrt(var + EPS), w)
        if op == "norm":
            return {"y": y}
        if case["packed"]:
            x = _form64(x, group)[0]
        # the gradient through y = w xh + b with mean and rstd as they were
        # kept: sums over the row by products with the all-ones vector
        xh, dy = (x - mean) * rstd, s["dy"].double()
        one = torch.ones(c, 1, dtype=torch.float64, device=x.device)
        a = dy * w
        dx = (c * a - a @ one - xh * ((xh * a) @ one)) * (rstd / c)
        return {"y": y, "mean": mean[:, 0], "rstd": rstd[:, 0], "dx": dx,
                "dweight": (xh * dy).sum(0), "dbias": dy.sum(0)}
    if op == "wgrad":
        x = s["codes"][:, :c].double()
        for k, lo in enumerate(range(0, c, group or c)):
            x[:, lo:lo + (group or c)] *= s["steps"][:, k:k + 1].double()
        dy = s["dy"].double()
        return {"dweight": torch.mm(dy.t().contiguous(), x), "dbias": dy.sum(0)}
    back = _form64(x, 0)[0]
    w = s["w_codes"][:, :c].double() * s["w_steps"].double()
    return {"y": torch.addmm(s["bias"].double(), back, w.t().contiguous())}
