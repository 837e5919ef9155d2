"""The 8-bit floating point products and the optimizer's step together: the
example's experts against fp32 gradients, a graph of the calls against the eager
calls, two streams at once, and arrays whose offsets pass 32 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import step as S
from tests.act_util import rounding

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


@pytest.fixture(scope="module")
def example(gq):
    spec = importlib.util.spec_from_file_location(
        "experts_step", os.path.join(ROOT, "examples", "experts_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def reference(p, x, offsets, dy):
    """(y, dx, gradients) in fp32 on the CPU."""
    p = {k: v.cpu().clone().requires_grad_() for k, v in p.items()}
    x = x.float().cpu().requires_grad_()
    parts = []
    for e, (lo, hi) in enumerate(zip(offsets, offsets[1:])):
        u = x[lo:hi] @ p["w1"][e].T + p["b1"][e]
        parts.append(torch.nn.functional.gelu(u) @ p["w2"][e].T + p["b2"][e])
    y = x + torch.cat(parts)
    y.backward(dy.float().cpu())
    return y.detach(), x.grad, {k: v.grad for k, v in p.items()}


def test_experts_against_fp32_gradients(example):
    """A value's e4m3 form is off by at most 2^-4 of it, evenly spread, so by
    0.036 of its size in the mean square.  A gradient sees four such operands at
    most one after the other (x or v, dy, du, a weight), and gelu's slope at a u
    that is off by two: 0.2 covers their sum however they add up."""
    t, f, h, k = 300, 200, 330, 4
    b = example.Experts(t, f, h, k)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(t, f, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(t, f, generator=gen, device="cuda").bfloat16()
    b.p["b1"].normal_(0.0, 0.2, generator=gen)
    offsets = [0, 100, 100, 170, 300]
    y = b.forward(x, torch.tensor(offsets, device="cuda"))
    dx = b.backward(dy)
    wy, wdx, wg = reference(b.p, x, offsets, dy)

    def off(got, want):
        return float((got.float().cpu() - want).norm() / want.norm())

    assert off(y, wy) < 0.2
    assert off(dx, wdx) < 0.2
    for name, g in b.g.items():
        assert off(g, wg[name]) < 0.2, name
        assert not g[1].any()                   # an expert without tokens
    # accumulated: twice the gradient, exactly where no product is in between
    first = b.grad.clone()
    b.backward(dy, beta=1.0)
    assert torch.equal(b.g["b2"].flatten(), 2 * first[-k * f:])
    assert off(b.grad, 2 * first.cpu()) < 1e-5


def test_example_runs_and_updates(example):
    """Every call of a step: parameters move by what AdamW makes of the gradient
    that arrived, and the packed weights follow."""
    b = example.Experts(200, 130, 270, 3)
    tr = example.Trainer(b, lr=1e-2, max_norm=0.5)
    gen = torch.Generator(device="cuda").manual_seed(4)
    offsets = torch.tensor([0, 50, 120, 200], device="cuda")
    n = b.flat.numel()
    m = v = np.zeros(n, np.float32)
    ends = b.layers.cpu().numpy()
    decay = b.decay.cpu().numpy()[np.searchsorted(ends[1:], np.arange(n), side="right")]
    for step in (1, 2):
        x = torch.randn(200, 130, generator=gen, device="cuda").bfloat16()
        b.forward(x, offsets)
        b.backward(x)
        before = b.flat.cpu().numpy()
        tr.update()
        g = tr.mean.cpu().numpy()
        norm = np.sqrt((g.astype(np.float64) ** 2).sum())
        assert abs(float(b.norm) - norm) <= 2.0 ** -23 * norm
        scale = float(b.scale)
        assert abs(scale - min(1.0, 0.5 / norm)) <= 2.0 ** -23
        p, m, v = S.adamw(before, m, v, g, step, np.float32(1e-2), 0.9, 0.999, 1e-8, decay,
                          scale, np.float32)
        assert np.array_equal(b.flat.cpu().numpy(), p)
        w = S.philox(0, step, n)
        mc, ms = S.state_codes(m.astype(np.float64), w >> np.uint64(16), S.E4M3, 448.0)
        vc, vs = S.state_codes(v.astype(np.float64), w & np.uint64(0xffff), S.E5M2, 57344.0)
        assert np.array_equal(tr.m[0].view(torch.uint8).cpu().numpy(), mc)
        assert np.array_equal(tr.v[0].view(torch.uint8).cpu().numpy(), vc)
        m = S.state_values(mc, ms, S.E4M3).astype(np.float32)
        v = S.state_values(vc, vs, S.E5M2).astype(np.float32)
    codes, steps = S.pack_weight(b.p["w2"].double().cpu().numpy())
    assert np.array_equal(b.w2[0].view(torch.uint8).cpu().numpy(), codes)
    assert np.array_equal(b.w2[1].cpu().numpy(), steps)
    losses = example.train(256, 128, 128, 2, 3, say=lambda *_: None)
    assert len(losses) == 3 and all(np.isfinite(losses))


def tensors(o):
    return [t for v in o.values() for t in (v if isinstance(v, tuple) else (v,))]


def same(p, q):
    return torch.equal(p.view(torch.uint8), q.view(torch.uint8))


class Step:
    """All calls of a step on buffers of its own."""

    def __init__(self, gq, rows, cols, out, experts, dtype, bits, ws, seed=3):
        self.gq, self.rows, self.cols, self.out, self.k = gq, rows, cols, out, experts
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.a = gq.act(rows, cols, dtype, 128)
        self.d = gq.act(rows, out, dtype, 128)
        self.aw = gq.act(out, cols, torch.float32, 128)
        self.x, self.dy = self.normal(rows, cols).to(dtype), self.normal(rows, out).to(dtype)
        self.bias = self.normal(experts, out)
        self.n = experts * out * (cols + 1)
        self.adamw = gq.adamw(1e-3, bits=bits, weight_decay=0.1)
        self.schedule = torch.empty(4, device="cuda")
        self.offsets = torch.linspace(0, rows, experts + 1, device="cuda").long()
        self.layers = torch.tensor([0, experts * out * cols, self.n], device="cuda")
        self.p0 = self.normal(self.n)
        self.need = max(gq.gq_block_linear_workspace(self.a, out, experts),
                        gq.gq_block_linear_workspace(self.d, cols, experts),
                        gq.gq_block_wgrad_workspace(self.a, out, experts),
                        gq.gq_grad_norm_workspace(self.n))
        self.ws = gq.alloc_workspace(self.need) if ws is None else ws

    def normal(self, *s):
        return torch.randn(*s, generator=self.gen, device="cuda")

    def outputs(self):
        gq, k = self.gq, self.k
        m, v = gq.alloc_adamw(self.adamw, self.n)
        return dict(x8=gq.alloc_block(self.a), dy8=gq.alloc_block(self.d),
                    w=gq.alloc_block_weight(self.aw, k),
                    wt=gq.alloc_block_weight(self.aw, k, transposed=True),
                    y=torch.empty_like(self.dy), dx=torch.empty_like(self.x),
                    back=torch.empty_like(self.x), grad=torch.zeros(self.n, device="cuda"),
                    norm=torch.empty(1, device="cuda"), scale=torch.empty(1, device="cuda"),
                    p=self.p0.clone(), m=m, v=v,
                    p16=torch.zeros(self.n, dtype=torch.bfloat16, device="cuda"))

    def run(self, o):
        gq, at = self.gq, dict(offsets=self.offsets, workspace=self.ws)
        nw = self.k * self.out * self.cols
        gq.gq_block_pack_weight(self.aw, o["p"][:nw].view(self.k, self.out, self.cols), o["w"],
                                o["wt"])
        gq.gq_block_pack(self.a, self.x, *o["x8"])
        gq.gq_block_unpack(self.a, *o["x8"], o["back"])
        gq.gq_block_linear(self.a, *o["x8"], *o["w"], self.bias, o["y"], **at)
        gq.gq_block_wgrad(self.a, self.dy, *o["x8"], o["grad"][:nw], o["grad"][nw:], **at)
        gq.gq_block_pack(self.d, self.dy, *o["dy8"])
        gq.gq_block_linear(self.d, *o["dy8"], *o["wt"], None, o["dx"], **at)
        gq.gq_grad_norm(o["grad"], 1.0, o["norm"], o["scale"], workspace=self.ws)
        gq.gq_adamw(self.adamw, o["grad"], o["p"], o["m"], o["v"], 1, self.layers,
                    grad_scale=o["scale"], schedule=self.schedule, p16=o["p16"], seed=7)


CASES = [(96, 200, 130, 3, torch.bfloat16, 8), (700, 256, 256, 2, torch.float32, 32),
         (5, 64, 1000, 4, torch.float16, 8), (600, 4100, 136, 1, torch.bfloat16, 32)]


@pytest.mark.parametrize("rows,cols,out,experts,dtype,bits", CASES)
def test_graph_replays(gq, rows, cols, out, experts, dtype, bits):
    """A step in one graph, replayed with eager work between; inputs, the table
    and the schedule change from replay to replay."""
    s = Step(gq, rows, cols, out, experts, dtype, bits, None)
    eager, held = s.outputs(), s.outputs()
    s.schedule.copy_(gq.adamw_schedule(s.adamw, 1))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        s.run(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.run(held)
    for k in ("p", "m", "v"):           # both sides from the same states
        for a, b in zip(*((o[k] if isinstance(o[k], tuple) else (o[k],)) for o in (held, eager))):
            a.view(torch.uint8).copy_(b.view(torch.uint8))
    for turn in range(4):
        s.x.copy_(s.normal(rows, cols))
        s.dy.copy_(s.normal(rows, out))
        cut = torch.randint(0, rows + 1, (experts - 1,), generator=s.gen, device="cuda")
        s.offsets[1:-1] = cut.sort()[0]
        s.schedule.copy_(gq.adamw_schedule(s.adamw, turn + 1, lr=1e-3 / (turn + 1)))
        s.run(eager)
        torch.cuda.synchronize()
        for name in ("y", "dx", "grad", "norm", "scale", "back"):
            held[name].fill_(3)
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(tensors(eager), tensors(held)):
            assert same(p, q), turn


def test_two_graphs_share_a_workspace(gq):
    """One after the other, in both orders."""
    shapes = [(300, 4100, 136, 1, torch.bfloat16, 8), (3000, 130, 96, 3, torch.bfloat16, 8)]
    need = max(Step(gq, *c, None).need for c in shapes)
    ws = gq.alloc_workspace(need)
    steps, held, want, graphs = [], [], [], []
    for c in shapes:
        s = Step(gq, *c, ws)
        s.schedule.copy_(gq.adamw_schedule(s.adamw, 1))
        o, w = s.outputs(), s.outputs()
        s.run(w)
        with torch.cuda.stream(torch.cuda.Stream()):
            torch.cuda.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                s.run(o)
        steps.append(s), held.append(o), want.append(w), graphs.append(graph)
    torch.cuda.synchronize()
    fresh = [{k: [t.clone() for t in (v if isinstance(v, tuple) else (v,))] for k, v in o.items()}
             for o in (s.outputs() for s in steps)]
    for order in ((0, 1), (1, 0), (0, 1)):
        for i in order:
            for k in ("p", "m", "v", "grad"):
                v = held[i][k]
                for a, b in zip(v if isinstance(v, tuple) else (v,), fresh[i][k]):
                    a.view(torch.uint8).copy_(b.view(torch.uint8))
            ws.fill_(0xff)
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            for p, q in zip(tensors(want[i]), tensors(held[i])):
                assert same(p, q)


def test_two_streams_at_once(gq):
    """Calls on streams of their own, with workspaces of their own, leave each
    other alone and repeat bit for bit."""
    c = (900, 4100, 200, 2, torch.bfloat16, 8)
    steps = [Step(gq, *c, None, seed=s) for s in (1, 2)]
    want = []
    for s in steps:
        s.schedule.copy_(gq.adamw_schedule(s.adamw, 1))
        o = s.outputs()
        s.run(o)
        want.append(o)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in steps]
    for _ in range(3):
        got = [s.outputs() for s in steps]
        torch.cuda.synchronize()
        for s, st, o in zip(steps, streams, got):
            with torch.cuda.stream(st):
                s.run(o)
        torch.cuda.synchronize()
        for w, o in zip(want, got):
            for p, q in zip(tensors(w), tensors(o)):
                assert same(p, q)


def test_stream_argument(gq):
    """Work goes to the stream that is given."""
    st = torch.cuda.Stream()
    a = gq.act(64, 128, torch.bfloat16, 128)
    x = torch.randn(64, 128, device="cuda").bfloat16()
    f, want = gq.alloc_block(a), gq.alloc_block(a)
    gq.gq_block_pack(a, x, *want)
    torch.cuda.synchronize()
    gq.gq_block_pack(a, x, *f, stream=st)
    st.synchronize()
    assert same(f[0], want[0]) and torch.equal(f[1], want[1])


def test_offsets_past_32_bits(gq):
    """More than 2^32 bytes of activations and 2^31 codes: the last rows."""
    rows, cols, tail, out = 540_000, 4100, 3, 40
    a = gq.act(rows, cols, torch.bfloat16, 128)
    assert rows * a.pitch > 2 ** 31
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    x[-tail:] = torch.randn(tail, cols, generator=gen, device="cuda").bfloat16()
    x[0] = 1.0
    codes, steps = gq.alloc_block(a)
    gq.gq_block_pack(a, x, codes, steps)
    wc, wsteps = S.pack(x[-tail:].double().cpu().numpy(), "bf16")
    raw = codes.view(torch.uint8)
    assert np.array_equal(raw[-tail:].cpu().numpy(), wc)
    assert np.array_equal(steps[-tail:].cpu().numpy(), wsteps)
    assert bool((raw[1:1000] == 0).all())
    back = torch.full((rows, cols), 5.0, dtype=torch.bfloat16, device="cuda")
    gq.gq_block_unpack(a, codes, steps, back)
    xr = S.unpack(wc, wsteps, cols)
    assert np.array_equal(back[-tail:].double().cpu().numpy(), xr)
    assert bool((back[0] == 1).all()) and bool((back[1:1000] == 0).all())
    del back, x

    # the weight gradient: dy is 0 but in the first and the last rows
    off = torch.tensor([0, rows - 5, rows], device="cuda")
    dy = torch.zeros(rows, out, dtype=torch.bfloat16, device="cuda")
    dy[0] = 2.0
    dy[-tail:] = torch.arange(tail * out, device="cuda").view(tail, out) % 7 - 3
    dw, db = torch.empty(2, out, cols, device="cuda"), torch.empty(2, out, device="cuda")
    gq.gq_block_wgrad(a, dy, codes, steps, dw, db, offsets=off,
                      workspace=gq.alloc_workspace(gq.gq_block_wgrad_workspace(a, out, 2)))
    d = dy[-tail:].double().cpu().numpy()
    assert bool((dw[0] == 2.0).all()) and bool((db[0] == 2.0).all())
    mag = np.abs(d).T @ np.abs(xr)
    assert (np.abs(dw[1].double().cpu().numpy() - d.T @ xr) <= 2 * 12 * 2.0 ** -24 * mag).all()
    assert np.array_equal(db[1].double().cpu().numpy(), d.sum(0))
    del dy

    # the product: the weight is 1 for one expert, -1 for the other
    w = torch.empty(2, out, codes.shape[1], dtype=torch.uint8, device="cuda")
    w[0], w[1] = 0x38, 0xb8
    w[:, :, cols:] = 0
    one = torch.ones(2, 1, a.groups, device="cuda")
    y = torch.full((rows, out), 9.0, dtype=torch.bfloat16, device="cuda")
    gq.gq_block_linear(a, codes, steps, w.view(E4M3), one, None, y, offsets=off,
                       workspace=gq.alloc_workspace(gq.gq_block_linear_workspace(a, out, 2)))
    want = -np.repeat(xr.sum(1)[:, None], out, 1)
    tol = ((cols + 2) * 2.0 ** -23 + 2.0 ** -10) * np.abs(xr).sum(1)[:, None]
    got = y[-tail:].double().cpu().numpy()
    assert (np.abs(got - want) <= tol + rounding(np.abs(want) + tol, "bf16")).all()
    assert bool((y[0] == float(torch.tensor(4100.0).bfloat16())).all())
    assert bool((y[1:-tail] == 0).all())


def test_few_tokens_through_a_weight_past_32_bits(gq):
    out, cols = 270_000, 8200
    a = gq.act(3, cols, torch.float32, 128)
    assert out * a.pitch > 2 ** 31
    w = torch.full((1, out, a.pitch), 0x38, dtype=torch.uint8, device="cuda")
    w[..., cols:] = 0
    w[0, -1, :cols] = 0x44                          # 3
    v = torch.ones(1, -(-out // 128), a.groups, device="cuda")
    x = torch.full((3, a.pitch), 0x40, dtype=torch.uint8, device="cuda")    # 2
    x[:, cols:] = 0
    s = torch.ones(3, a.groups, device="cuda")
    y = torch.zeros(3, out, device="cuda")
    gq.gq_block_linear(a, x.view(E4M3), s, w.view(E4M3), v, None, y)
    assert bool((y[:, :-1] == 2 * cols).all()) and bool((y[:, -1] == 6 * cols).all())


@pytest.mark.parametrize("bits", [8, 32])
def test_update_past_32_bits(gq, bits):
    """More values than 2^22 workgroups of the smallest size take: the first and
    the last of them."""
    n = (2 ** 33 if bits == 8 else 2 ** 32) + 1003
    d = gq.adamw(1e-2, bits=bits, weight_decay=0.1)
    g, p = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    tail = 1003 + 256
    gen = torch.Generator(device="cuda").manual_seed(5)
    for t in (g, p):
        t[-tail:] = torch.randn(tail, generator=gen, device="cuda")
    g[0] = 1.0
    m, v = gq.alloc_adamw(d, n)
    ends = torch.tensor([0, n - 700, n], device="cuda")
    scale = torch.tensor([1.0, 0.5], device="cuda")
    gl, pl = (t[-tail:].cpu().numpy() for t in (g, p))
    gq.gq_adamw(d, g, p, m, v, 1, ends, lr_scale=scale, seed=11)
    lr = np.where(np.arange(tail) < tail - 700, np.float32(1e-2), np.float32(1e-2) * np.float32(0.5))
    zero = np.zeros(tail, np.float32)
    wp, wm, wv = S.adamw(pl, zero, zero, gl, 1, lr, 0.9, 0.999, 1e-8, np.float32(0.1),
                         kind=np.float32)
    assert np.array_equal(p[-tail:].cpu().numpy(), wp)
    assert float(p[0]) < 0 and not bool(p[1:100000].any())
    if bits == 32:
        assert np.array_equal(m[-tail:].cpu().numpy(), wm)
        assert np.array_equal(v[-tail:].cpu().numpy(), wv)
    else:
        w = S.philox(11, 1, tail, first=n - tail)
        mc, ms = S.state_codes(wm.astype(np.float64), w >> np.uint64(16), S.E4M3, 448.0)
        vc, vs = S.state_codes(wv.astype(np.float64), w & np.uint64(0xffff), S.E5M2, 57344.0)
        assert np.array_equal(m[0].view(torch.uint8)[-tail:].cpu().numpy(), mc)
        assert np.array_equal(v[0].view(torch.uint8)[-tail:].cpu().numpy(), vc)
        assert np.array_equal(m[1][-5:].cpu().numpy(), ms)
    norm = torch.empty(1, device="cuda")
    gq.gq_grad_norm(g, 1.0, norm, workspace=gq.alloc_workspace(gq.gq_grad_norm_workspace(n)))
    want = np.sqrt(1.0 + (gl.astype(np.float64) ** 2).sum())
    assert abs(float(norm) - want) <= 2.0 ** -23 * want
