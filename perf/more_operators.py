"""Cases of the operators of a training step in 8-bit floating point: the
weight's form (e4m3 codes with a step per block of 128 x 128, as it lies and
transposed), the linear layer's product from forms with a step per 128 columns,
alone and grouped by expert over ragged numbers of tokens, its weight gradient
by expert, and the AdamW step over all tensors with states in 32 or 8 bits.

A case is a dict of plain values: ``op`` picks the operator, ``rows`` x
``cols`` is the activation matrix (tokens x features), ``out`` the layer's
output features, ``experts`` the weights that share the tokens, ``dtype`` the
activations' type; ``n`` the parameters in ``layers`` tensors, ``bits`` those
of a state, ``clip`` whether the gradient is clipped to a norm first.  ``run``
computes the operators in plain torch operations, or calls the library's entry
points where ``own`` is true; ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 128             # columns (and rows of a weight) that share a step
STATES = 256            # values of an 8-bit state that share a step
LR, BETA1, BETA2, EPS, DECAY, STEP = 1e-4, 0.9, 0.999, 1e-8, 0.1, 7
MAX_NORM = 1.0
MOST_FLOPS = 2.0 * 8192 * 4096 * 8192       # the largest listed product
MOST_VALUES = 64_000_000                    # the largest listed update


def listed():
    return [
        # a layer's weights for the next step, both directions
        dict(name="weight_layer", op="weight", experts=1, out=4096, cols=1024,
             dtype="f32"),
        # all experts' weights of a layer, odd features, from a 16-bit model
        dict(name="weight_experts_odd", op="weight", experts=8, out=1001, cols=2050,
             dtype="bf16"),
        # one token through a wide layer: serving
        dict(name="linear_one_token", op="linear", rows=1, cols=4096, out=4096,
             experts=1, dtype="bf16"),
        # a ragged serving batch through odd features
        dict(name="linear_ragged", op="linear", rows=203, cols=4100, out=2050,
             experts=1, dtype="f16"),
        # a training batch through a wide layer
        dict(name="linear_batch", op="linear", rows=8192, cols=4096, out=8192,
             experts=1, dtype="bf16"),
        # serving: a few tokens' choices among experts, some without any
        dict(name="experts_few_tokens", op="linear", rows=32, cols=2048, out=1024,
             experts=16, dtype="bf16"),
        # a training batch over experts of very different load
        dict(name="experts_batch", op="linear", rows=16384, cols=2048, out=2048,
             experts=32, dtype="bf16"),
        # the experts' weight gradients of a training batch
        dict(name="wgrad_experts", op="wgrad", rows=16384, cols=2048, out=2048,
             experts=8, dtype="bf16"),
        # fp16 gradients, few tokens to an expert, odd features
        dict(name="wgrad_experts_odd", op="wgrad", rows=1531, cols=1001, out=770,
             experts=12, dtype="f16"),
        # a small model's update: latency
        dict(name="adamw_small", op="adamw", n=65_536, layers=6, bits=32, clip=False),
        # a vision model's size, clipped, 160 tensors, states in 32 bits
        dict(name="adamw_clipped", op="adamw", n=25_600_000, layers=160, bits=32,
             clip=True),
        # states in 8 bits, for what they leave free
        dict(name="adamw_states8", op="adamw", n=64_000_000, layers=291, bits=8,
             clip=False),
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
        op = rng.choice(("weight", "linear", "linear", "linear", "wgrad", "adamw"))
        if op == "adamw":
            n = spread(1000, MOST_VALUES)
            return dict(op=op, n=n, layers=rng.randint(1, min(300, n // 100)),
                        bits=rng.choice((8, 32)), clip=rng.random() < 0.5)
        c = dict(op=op, cols=spread(64, 8192), out=spread(64, 8192),
                 experts=1 if rng.random() < 0.3 else spread(2, 64),
                 dtype=rng.choice(("bf16", "bf16", "f16", "f32")))
        if op != "weight":
            c["rows"] = spread(1, 16384)
        if (c["experts"] * c["out"] * c["cols"] <= 32 * 2048 * 2048
                and work(c)["flops"] <= MOST_FLOPS):
            return c


def work(case):
    if case["op"] == "adamw":
        n = case["n"]
        state = 8 * n if case["bits"] == 32 else 2 * n + 8 * -(-n // STATES)
        # gradient and parameters in, states in and out, parameters out
        return {"bytes": 12 * n + 2 * state + 8 * case["layers"],
                "flops": (16 if case["clip"] else 14) * n}
    k, c, o, s = case["experts"], case["cols"], case["out"], SIZE[case["dtype"]]
    blocks = -(-c // BLOCK) * -(-o // BLOCK)
    if case["op"] == "weight":                  # both directions
        return {"bytes": k * (c * o * (s + 2) + 8 * blocks), "flops": 3.0 * k * c * o}
    r = case["rows"]
    used = min(k, r)                            # experts that have tokens, at most
    if case["op"] == "linear":
        return {"bytes": s * r * (c + o) + used * (c * o + 4 * blocks + 4 * o),
                "flops": 2.0 * r * c * o}
    return {"bytes": s * r * o + r * (c + 4 * -(-c // BLOCK)) + 4 * k * o * (c + 1),
            "flops": 2.0 * r * c * o}


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "adamw":
        return _prepare_update(case, normal, g)
    k, c, o, t = case["experts"], case["cols"], case["out"], DTYPES[case["dtype"]]
    s = dict(case=case)
    if case["op"] == "weight":
        s["w"] = (normal(k, o, c) / math.sqrt(c)).to(t)
        return s
    r = case["rows"]
    # tokens sorted by expert: loads of very different size, some of none
    load = torch.softmax(1.5 * normal(k), 0)
    load = torch.where(load < 0.3 / k, 0.0, load)
    first = torch.zeros(k + 1, dtype=torch.int64, device="cuda")
    first[1:] = torch.round(torch.cumsum(load / load.sum(), 0) * r).long().clamp(max=r)
    first[-1] = r
    s["offsets"], s["first"] = first, first.tolist()
    # activations: features of very different size, as in trained networks
    x = (normal(r, c) * torch.exp(normal(c)) + 0.1 * normal(c)).to(t)
    if case["op"] == "linear":
        s["x"] = x
        s["w_codes"], s["w_steps"] = _weight_form(normal(k, o, c) / math.sqrt(c))
        s["bias"] = 0.1 * normal(k, o)
    else:
        # the form that the forward pass kept: rows of codes padded with zeros
        # to 16, and the gradient of the layer's output
        s["codes"], s["steps"] = _form(x)
        s["dy"] = (normal(r, o) * 1e-2).to(t)
    return s


def _prepare_update(case, normal, g):
    n, layers = case["n"], case["layers"]
    cut = torch.exp(2.0 * normal(layers))
    first = torch.zeros(layers + 1, dtype=torch.int64, device="cuda")
    first[1:] = torch.round(torch.cumsum(cut / cut.sum(), 0) * n).long().clamp(max=n)
    first[-1] = n
    # gradients of layers, and of values within one, of very different size
    size = torch.exp(normal(layers)).repeat_interleave(first.diff(), output_size=n)
    s = dict(case=case, offsets=first, g=normal(n) * torch.exp(normal(n)) * size * 1e-4,
             p=0.05 * normal(n), rate=torch.exp(0.3 * normal(layers)),
             decay=torch.where(normal(layers) > 0, DECAY, 0.0), seed=int(first[1]) + n)
    m = s["g"] * (0.5 + 0.3 * normal(n))
    v = s["g"].square() * torch.exp(0.5 * normal(n)) + 1e-16
    if case["bits"] == 32:
        return dict(s, m=m, v=v)
    half = torch.full((n,), 1 << 15, dtype=torch.int64, device="cuda")
    s["m"], s["m_steps"] = _state_codes(m, half, E4M3)
    s["v"], s["v_steps"] = _state_codes(v, half, E5M2)
    return s


# ------------------------------------------------------------ plain form ----
def _power(e):
    """2^e for -126 <= e <= 127, exact."""
    return ((e + 127) << 23).view(torch.float32)


def _steps(m, most, cap):
    """The smallest power of two with most * step >= m, from 2^-126 to 2^cap."""
    top = math.frexp(most)                      # most = top[0] 2^top[1]
    frac, e = torch.frexp(m)                    # m = frac 2^e, frac in [1/2, 1)
    e = torch.where(frac <= top[0], e - top[1], e - top[1] + 1).clamp(-126, cap)
    return torch.where(m > 0, _power(e), 0.0)


def _form(x):
    """Codes [rows, cols up to 16] and steps [rows, groups] of 128 columns."""
    r, c = x.shape
    cap = 7 if x.dtype == torch.float16 else 119
    n = -(-c // BLOCK)
    a = torch.zeros(r, n * BLOCK, device=x.device)
    a[:, :c] = x
    steps = _steps(a.view(r, n, BLOCK).abs().amax(-1), 448.0, cap)
    s = steps.repeat_interleave(BLOCK, dim=1)
    q = torch.where(s > 0, a / torch.where(s > 0, s, 1.0), 0.0).clamp(-448, 448)
    return q[:, :-(-c // 16) * 16].to(torch.float8_e4m3fn).contiguous(), steps


def _weight_form(w):
    """Codes [experts, out, cols up to 16] and steps [experts, blocks of out,
    blocks of cols] of blocks of 128 x 128."""
    k, o, c = w.shape
    cap = 7 if w.dtype == torch.float16 else 119
    no, nc = -(-o // BLOCK), -(-c // BLOCK)
    a = torch.zeros(k, no * BLOCK, nc * BLOCK, device=w.device)
    a[:, :o, :c] = w
    steps = _steps(a.view(k, no, BLOCK, nc, BLOCK).abs().amax((2, 4)), 448.0, cap)
    s = steps.repeat_interleave(BLOCK, dim=1).repeat_interleave(BLOCK, dim=2)
    q = torch.where(s > 0, a / torch.where(s > 0, s, 1.0), 0.0).clamp(-448, 448)
    return q[:, :o, :-(-c // 16) * 16].to(torch.float8_e4m3fn).contiguous(), steps


def _values(codes, steps, c):
    return codes[:, :c].float() * steps.repeat_interleave(BLOCK, dim=1)[:, :c]


def _weight_values(codes, steps, c):
    s = steps.repeat_interleave(BLOCK, dim=0)[:codes.shape[0]]
    return _values(codes, s, c)


# Two 8-bit floats: mantissa bits, exponent bias, largest value, type.
E4M3 = (3, 7, 448.0, torch.float8_e4m3fn)
E5M2 = (2, 15, 57344.0, torch.float8_e5m2)


def _random(n, seed, step, device):
    """Sixteen random bits twice for each value: word i mod 4 of Philox4x32-10
    with the key `seed` at the counter (i / 4, step), its upper and lower half."""
    i = torch.arange(-(-n // 4), dtype=torch.int64, device=device)
    low = 0xffffffff
    c = [i & low, i >> 32, torch.full_like(i, step), torch.zeros_like(i)]
    k0, k1 = seed & low, seed >> 32 & low
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57     # 64 bits, wrapped
        c = [(b >> 32 & low) ^ c[1] ^ k0, b & low, (a >> 32 & low) ^ c[3] ^ k1, a & low]
        k0, k1 = k0 + 0x9E3779B9 & low, k1 + 0xBB67AE85 & low
    w = torch.stack(c, 1).view(-1)[:n]
    return w >> 16, w & 0xffff


def _state_codes(x, r16, form):
    """Codes and steps of 256 values each; up where the place between two
    codes, in units of 2^-16, and `r16` together reach one.  v stays over 0."""
    bits, bias, most, kind = form
    n = x.numel()
    a = torch.zeros(-(-n // STATES) * STATES, device=x.device)
    a[:n] = x
    steps = _steps(a.view(-1, STATES).abs().amax(1), most, 119)
    s = steps.repeat_interleave(STATES)[:n]
    y = torch.where(s > 0, x.abs() / torch.where(s > 0, s, 1.0), 0.0)
    # as a float whose upper bits are the code's
    z = (y * 2.0 ** (bias - 127)).view(torch.int32).to(torch.int64)
    code = z + (r16 << 7 - bits) >> 23 - bits
    if form is E5M2:
        code = torch.where(x > 0, code.clamp(min=1), code)
    code = code | torch.where(x < 0, 128, 0)
    return code.to(torch.uint8).view(kind), steps


def _state_values(codes, steps):
    return codes.float() * steps.repeat_interleave(STATES)[:codes.numel()]


def _plain_update(s):
    case, n = s["case"], s["case"]["n"]
    g = s["g"]
    out = {}
    if case["clip"]:
        norm = g.double().square().sum().sqrt()
        out["norm"] = norm.float()
        g = g * torch.where(norm > MAX_NORM, MAX_NORM / norm, 1.0).float()
    m, v = s["m"], s["v"]
    if case["bits"] == 8:
        m, v = _state_values(m, s["m_steps"]), _state_values(v, s["v_steps"])
    m = m * BETA1 + g * (1 - BETA1)
    v = v * BETA2 + g * (1 - BETA2) * g
    counts = s["offsets"].diff()
    lr = s["rate"] * LR
    size = (lr / (1 - BETA1 ** STEP)).repeat_interleave(counts, output_size=n)
    decay = (lr * s["decay"]).repeat_interleave(counts, output_size=n)
    root = torch.sqrt(v) * (1 / math.sqrt(1 - BETA2 ** STEP)) + EPS
    s["p"] = s["p"] - (size * m / root + decay * s["p"])
    if case["bits"] == 32:
        s["m"], s["v"] = m, v
        return dict(out, p=s["p"], m=m, v=v)
    up, low = _random(n, s["seed"], STEP, g.device)
    s["m"], s["m_steps"] = _state_codes(m, up, E4M3)
    s["v"], s["v_steps"] = _state_codes(v, low, E5M2)
    return dict(out, p=s["p"], m=s["m"], m_steps=s["m_steps"], v=s["v"],
                v_steps=s["v_steps"])


def _plain(s):
    case = s["case"]
    if case["op"] == "adamw":
        return _plain_update(s)
    if case["op"] == "weight":
        codes, steps = _weight_form(s["w"])
        t_codes, t_steps = _weight_form(s["w"].transpose(1, 2))
        return {"codes": codes, "steps": steps, "t_codes": t_codes, "t_steps": t_steps}
    r, c, o, first = case["rows"], case["cols"], case["out"], s["first"]
    if case["op"] == "linear":
        x = _values(*_form(s["x"]), c)
        y = torch.empty(r, o, device=x.device)
        for k in range(case["experts"]):
            if first[k] < first[k + 1]:
                w = _weight_values(s["w_codes"][k], s["w_steps"][k], c)
                y[first[k]:first[k + 1]] = x[first[k]:first[k + 1]] @ w.t() + s["bias"][k]
        return {"y": y.to(s["x"].dtype)}
    x, dy = _values(s["codes"], s["steps"], c), s["dy"].float()
    dw = torch.empty(case["experts"], o, c, device=x.device)
    db = torch.empty(case["experts"], o, device=x.device)
    for k in range(case["experts"]):
        part = dy[first[k]:first[k + 1]]
        dw[k] = part.t().contiguous() @ x[first[k]:first[k + 1]]
        db[k] = part.sum(0)
    return {"dweight": dw, "dbias": db}


# ------------------------------------------------------- the library's calls ----
def _own_update(s, gq):
    case, n = s["case"], s["case"]["n"]
    k = s.get("keep")
    if k is None:           # what a program holds from step to step
        k = s["keep"] = {"adamw": gq.adamw(LR, BETA1, BETA2, EPS, DECAY, case["bits"])}
        if case["clip"]:
            k["norm"], k["scale"] = (torch.empty(1, device="cuda") for _ in range(2))
            k["ws"] = gq.alloc_workspace(gq.gq_grad_norm_workspace(n))
    out, scale = {}, None
    if case["clip"]:
        gq.gq_grad_norm(s["g"], MAX_NORM, k["norm"], k["scale"], workspace=k["ws"])
        out["norm"], scale = k["norm"][0], k["scale"]
    m, v = s["m"], s["v"]
    if case["bits"] == 8:
        m, v = (m, s["m_steps"]), (v, s["v_steps"])
    gq.gq_adamw(k["adamw"], s["g"], s["p"], m, v, STEP, s["offsets"], s["rate"],
                s["decay"], grad_scale=scale, seed=s["seed"])
    out.update(p=s["p"], m=s["m"], v=s["v"])
    if case["bits"] == 8:
        out.update(m_steps=s["m_steps"], v_steps=s["v_steps"])
    return out


def _own(s):
    from communication_efficient_gradient_amd import gq

    case = s["case"]
    op = case["op"]
    if op == "adamw":
        return _own_update(s, gq)
    e, c, o, t = case["experts"], case["cols"], case["out"], DTYPES[case["dtype"]]
    k = s.get("keep")
    if k is None:           # what a program holds from step to step
        k = s["keep"] = {}

        def new(*shape, dtype=torch.float32):
            return torch.empty(*shape, dtype=dtype, device="cuda")

        if op == "weight":
            k["act"] = gq.act(o, c, t, BLOCK)
            k["form"] = gq.alloc_block_weight(k["act"], e)
            k["t_form"] = gq.alloc_block_weight(k["act"], e, transposed=True)
        else:
            r = case["rows"]
            k["act"] = gq.act(r, c, t, BLOCK)
            k["offsets"] = s["offsets"] if e > 1 else None
        if op == "linear":
            k["form"], k["y"] = gq.alloc_block(k["act"]), new(r, o, dtype=t)
            k["ws"] = gq.alloc_workspace(gq.gq_block_linear_workspace(k["act"], o, e))
        if op == "wgrad":
            k["dw"], k["db"] = new(e, o, c), new(e, o)
            k["ws"] = gq.alloc_workspace(gq.gq_block_wgrad_workspace(k["act"], o, e))
    a = k["act"]
    if op == "weight":
        gq.gq_block_pack_weight(a, s["w"], k["form"], k["t_form"])
        return {"codes": k["form"][0], "steps": k["form"][1],
                "t_codes": k["t_form"][0], "t_steps": k["t_form"][1]}
    if op == "linear":
        gq.gq_block_pack(a, s["x"], *k["form"])
        gq.gq_block_linear(a, *k["form"], s["w_codes"], s["w_steps"], s["bias"], k["y"],
                         offsets=k["offsets"], workspace=k["ws"])
        return {"y": k["y"]}
    gq.gq_block_wgrad(a, s["dy"], s["codes"], s["steps"], k["dw"], k["db"],
                    offsets=k["offsets"], workspace=k["ws"])
    return {"dweight": k["dw"], "dbias": k["db"]}


def run(state):
    return _own(state) if own else _plain(state)


# ------------------------------------------------------------- 64 bits ----
def _power64(e):
    """2^e, exact (a library's pow may be off by its last bit)."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _steps64(m, most, cap):
    """By halving and doubling trial steps from an estimate."""
    e = torch.floor(torch.log2(torch.where(m > 0, m, 1.0) / most))
    for _ in range(3):
        e = torch.where(most * _power64(e) < m, e + 1, e)
        e = torch.where(most * _power64(e - 1) >= m, e - 1, e)
    return torch.where(m > 0, _power64(e.clamp(-126, cap)), 0.0)


def _grid64(y, bits, lowest):
    """Spacing of the 8-bit floats around |y|: `bits` of mantissa, exponents
    from `lowest` up."""
    e = torch.frexp(y.abs())[1] - 1
    return _power64(e.clamp(min=lowest) - bits)


def _nearest64(y):
    """y as the nearest e4m3 value, ties to even."""
    u = _grid64(y, 3, -6)
    q = y.abs() / u
    low = torch.floor(q)
    rest = q - low
    up = (rest > 0.5) | ((rest == 0.5) & (low % 2 != 0))
    return torch.copysign(((low + up) * u).clamp(max=448), y)


def _weight64(w, cap):
    """Codes and steps, padded to 16 columns, block by block."""
    k, o, c = w.shape
    codes = torch.zeros(k, o, -(-c // 16) * 16, dtype=torch.float64, device=w.device)
    steps = torch.zeros(k, -(-o // BLOCK), -(-c // BLOCK), dtype=torch.float64,
                        device=w.device)
    for i, a in enumerate(range(0, o, BLOCK)):
        for j, b in enumerate(range(0, c, BLOCK)):
            part = w[:, a:a + BLOCK, b:b + BLOCK]
            s = _steps64(part.abs().amax((1, 2)), 448.0, cap)
            y = part / torch.where(s > 0, s, 1.0)[:, None, None]
            codes[:, a:a + BLOCK, b:b + part.shape[2]] = _nearest64(y)
            steps[:, i, j] = s
    return codes, steps


def _state64(x, r16, bits, lowest, most):
    """Codes and steps of a state's 256-value blocks, random rounding."""
    codes = torch.zeros_like(x)
    pad = torch.nn.functional.pad(x.abs(), (0, -x.numel() % STATES))
    steps = _steps64(pad.view(-1, STATES).max(1).values, most, 119)
    at = torch.arange(x.numel(), device=x.device) // STATES
    s = steps[at]
    y = x.abs() / torch.where(s > 0, s, 1.0)
    u = _grid64(y, bits, lowest)
    low = torch.floor(y / u)
    up = (y / u - low) + r16.double() * 2.0 ** -16 >= 1.0
    q = (low + up) * u
    if lowest < -6:                             # v: over 0 stays over 0
        q = torch.where((x > 0) & (q == 0), u, q)
    codes = torch.copysign(q, x)
    return codes, steps


def _exact_update(s):
    case, n = s["case"], s["case"]["n"]
    g, p, m, v = (s[k].double() for k in ("g", "p", "m", "v"))
    out = {}
    if case["bits"] == 8:
        at = torch.arange(n, device=g.device) // STATES
        m, v = m * s["m_steps"].double()[at], v * s["v_steps"].double()[at]
    if case["clip"]:
        out["norm"] = torch.linalg.vector_norm(g)
        g = g * min(1.0, MAX_NORM / float(out["norm"]))
    m = torch.lerp(g, m, BETA1)
    v = torch.lerp(g * g, v, BETA2)
    layer = torch.searchsorted(s["offsets"][1:], torch.arange(n, device=g.device), right=True)
    lr = LR * s["rate"].double()[layer]
    p = p - lr * s["decay"].double()[layer] * p - lr * (m / (1 - BETA1 ** STEP)) / (
        torch.sqrt(v / (1 - BETA2 ** STEP)) + EPS)
    if case["bits"] == 32:
        return dict(out, p=p, m=m, v=v)
    up, low = _random(n, s["seed"], STEP, g.device)
    mc, ms = _state64(m, up, 3, -6, 448.0)
    vc, vs = _state64(v, low, 2, -14, 57344.0)
    return dict(out, p=p, m=mc, m_steps=ms, v=vc, v_steps=vs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "adamw":
        return _exact_update(s)
    cap = 7 if case["dtype"] == "f16" else 119
    if case["op"] == "weight":
        w = s["w"].double()
        codes, steps = _weight64(w, cap)
        t_codes, t_steps = _weight64(w.transpose(1, 2).contiguous(), cap)
        return {"codes": codes, "steps": steps, "t_codes": t_codes, "t_steps": t_steps}
    r, c, o = case["rows"], case["cols"], case["out"]
    groups = range(0, c, BLOCK)
    if case["op"] == "linear":
        x = s["x"].double()
        for lo in groups:
            part = x[:, lo:lo + BLOCK]
            step = _steps64(part.abs().amax(1), 448.0, cap)[:, None]
            x[:, lo:lo + BLOCK] = _nearest64(part / torch.where(step > 0, step, 1.0)) * step
        y = torch.zeros(r, o, dtype=torch.float64, device=x.device)
        of = torch.arange(o, device=x.device) // BLOCK
        for k in range(case["experts"]):
            mine = slice(s["first"][k], s["first"][k + 1])
            w = s["w_codes"][k][:, :c].double()
            for j, lo in enumerate(groups):
                w[:, lo:lo + BLOCK] *= s["w_steps"][k][of, j].double()[:, None]
            y[mine] = torch.addmm(s["bias"][k].double(), x[mine], w.t().contiguous())
        return {"y": y}
    x, dy = s["codes"][:, :c].double(), s["dy"].double()
    for j, lo in enumerate(groups):
        x[:, lo:lo + BLOCK] *= s["steps"][:, j:j + 1].double()
    dw, db = [], []
    for k in range(case["experts"]):
        mine = slice(s["first"][k], s["first"][k + 1])
        one = torch.ones(1, mine.stop - mine.start, dtype=torch.float64, device=x.device)
        dw.append(torch.mm(dy[mine].t().contiguous(), x[mine]))
        db.append(torch.mm(one, dy[mine])[0])
    return {"dweight": torch.stack(dw), "dbias": torch.stack(db)}
