"""The 8-bit activation operators together: the example's block against a
block in fp32 with torch's own gradients, a graph of the calls against the
eager calls, and matrices whose offsets pass 32 bits."""
import importlib.util
import os

import numpy as np
import pytest
import torch

from oracle import activations as A

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


@pytest.fixture(scope="module")
def example(gq):
    spec = importlib.util.spec_from_file_location(
        "mlp_step", os.path.join(ROOT, "examples", "mlp_step.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_block_against_fp32_gradients(example):
    """An 8-bit operand with steps of at most 2 * max / 127 and max near 4
    sigma is off by at most 0.063 / sqrt(12) = 0.018 sigma; a gradient sees
    five such operands at most (x, norm, u, v, a weight), so 0.1 covers their
    sum however they add up."""
    b = example.Block(300, 200, 330)
    gen = torch.Generator(device="cuda").manual_seed(2)
    x = torch.randn(300, 200, generator=gen, device="cuda").bfloat16()
    dy = torch.randn(300, 200, generator=gen, device="cuda").bfloat16()
    b.p["norm.weight"].normal_(1.0, 0.2, generator=gen)
    b.p["b1"].normal_(0.0, 0.2, generator=gen)
    y = b.forward(x)
    dx = b.backward(dy)
    flat = b.flat.cpu().requires_grad_()
    xr = x.float().cpu().requires_grad_()
    p, at = {}, 0
    for name, v in b.p.items():
        p[name] = flat[at:at + v.numel()].view(v.shape)
        at += v.numel()
    n = torch.nn.functional.layer_norm(xr, (200,), p["norm.weight"], p["norm.bias"], 1e-5)
    v = torch.nn.functional.gelu(n @ p["w1"].T + p["b1"], approximate="tanh")
    yr = xr + v @ p["w2"].T + p["b2"]
    yr.backward(dy.float().cpu())

    def off(got, want):
        return float((got.float().cpu() - want).norm() / want.norm())

    assert off(y, yr.detach()) < 0.1
    assert off(dx, xr.grad) < 0.1
    at = 0
    for name, g in b.g.items():
        want = flat.grad[at:at + g.numel()].view(g.shape)
        at += g.numel()
        assert off(g, want) < 0.1, name
    # accumulated: twice the gradient, exactly where no product is in between
    first = b.grad.clone()
    b.backward(dy, beta=1.0)
    assert torch.equal(b.g["b2"], 2 * first[-200:])
    assert off(b.grad, 2 * first.cpu()) < 1e-5


def test_training_lowers_the_loss(example):
    """Every step lowers the loss, and all of them together lower it as much
    as the same descent in fp32 does, but for a gradient that is off by at
    most 0.1 of its length (the bound above): 0.1 of the way."""
    t, f, h, steps = 512, 256, 512, 12
    losses = example.train(t, f, h, steps, say=lambda *_: None)
    assert all(np.diff(losses) < 0)

    b = example.Block(t, f, h)              # the same start and data
    p = {k: v.cpu().clone().requires_grad_() for k, v in b.p.items()}
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(t, f, generator=gen, device="cuda").to(b.dtype)
    mix = torch.randn(f, f, generator=gen, device="cuda") * f ** -0.5
    target = (x + torch.tanh(x.float() @ mix).to(b.dtype)).float().cpu()
    x = x.float().cpu()
    want = []
    for _ in range(steps):
        n = torch.nn.functional.layer_norm(x, (f,), p["norm.weight"], p["norm.bias"], 1e-5)
        v = torch.nn.functional.gelu(n @ p["w1"].T + p["b1"], approximate="tanh")
        diff = x + v @ p["w2"].T + p["b2"] - target
        want.append(float(diff.detach().square().mean()))
        grads = torch.autograd.grad(diff.square().sum() / t, list(p.values()))
        with torch.no_grad():
            for q, g in zip(p.values(), grads):
                q -= 0.5 / h * g
    fell, way = losses[0] - losses[-1], want[0] - want[-1]
    assert abs(fell - way) < 0.1 * way


@pytest.mark.parametrize("rows,cols,out", [(96, 200, 130), (2048, 256, 256), (5, 64, 1000)])
def test_graph_replays(gq, rows, cols, out):
    """All calls of a step in one graph, replayed with eager work between."""
    gen = torch.Generator(device="cuda").manual_seed(3)

    def normal(*s):
        return torch.randn(*s, generator=gen, device="cuda")

    a = gq.act(rows, cols, torch.bfloat16)
    x, dy, du = (normal(rows, c).bfloat16() for c in (cols, out, cols))
    w, b, bias = normal(cols), normal(cols), normal(out)
    aw = gq.act(out, cols, torch.float32)
    w8 = gq.alloc_act(aw)
    gq.gq_act_pack(aw, normal(out, cols), *w8)
    ws = gq.alloc_workspace(max(gq.gq_layer_norm_workspace(a), gq.gq_act_wgrad_workspace(a, out),
                                gq.gq_act_linear_workspace(a, out)))

    def outputs():
        return dict(x8=gq.alloc_act(a), n8=gq.alloc_act(a), n=torch.empty_like(x),
                    z=torch.empty(rows, out, dtype=x.dtype, device="cuda"),
                    back=torch.empty_like(x), dx=torch.empty_like(x),
                    stats=torch.empty(2, rows, device="cuda"),
                    dn=torch.empty(2, cols, device="cuda"),
                    dw=torch.empty(out, cols, device="cuda"), db=torch.empty(out, device="cuda"))

    def step(o):
        gq.gq_layer_norm(a, x, w, b, 1e-5, o["n"], mean=o["stats"][0], rstd=o["stats"][1],
                         x_form=o["x8"], y_form=o["n8"])
        gq.gq_act_linear(a, *o["n8"], *w8, bias, o["z"], workspace=ws)
        gq.gq_act_wgrad(a, dy, *o["n8"], o["dw"], o["db"], workspace=ws)
        gq.gq_act_unpack(a, *o["x8"], o["back"])
        gq.gq_layer_norm_backward(a, du, o["x8"], *o["stats"], w, o["dx"], *o["dn"],
                                  workspace=ws)

    def tensors(o):
        return [t for v in o.values() for t in (v if isinstance(v, tuple) else (v,))]

    eager, held = outputs(), outputs()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(held)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(held)
    for turn in range(4):
        x.copy_(normal(rows, cols))
        dy.copy_(normal(rows, out))
        for t in tensors(held):
            t.fill_(3)
        step(eager)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for p, q in zip(tensors(eager), tensors(held)):
            assert torch.equal(p, q), turn


def test_offsets_past_32_bits(gq):
    """More than 2^32 bytes of activations and 2^31 codes: the last rows."""
    rows, cols, tail = 540_000, 4100, 3
    a = gq.act(rows, cols, torch.bfloat16, 128)
    assert rows * a.pitch > 2 ** 31
    x = torch.zeros(rows, cols, dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    x[-tail:] = torch.randn(tail, cols, generator=gen, device="cuda").bfloat16()
    x[0] = 1.0
    codes, steps = gq.alloc_act(a)
    gq.gq_act_pack(a, x, codes, steps)
    wc, wsteps = A.pack(x[-tail:].double().cpu().numpy(), 128)
    assert np.array_equal(codes[-tail:].cpu().numpy(), wc)
    assert np.array_equal(steps[-tail:].cpu().numpy(), wsteps)
    assert (codes[0, :cols] == 64).all() and (codes[1:1000] == 0).all()
    back = torch.full((rows, cols), 5.0, dtype=torch.bfloat16, device="cuda")
    gq.gq_act_unpack(a, codes, steps, back)
    xr = A.unpack(wc, wsteps, cols, 128)
    assert np.array_equal(back[-tail:].double().cpu().numpy(), xr)
    assert (back[0] == 1).all() and (back[1:1000] == 0).all()

    # the weight gradient: dy is 0 but in the first and the last rows
    out = 40
    dy = torch.zeros(rows, out, dtype=torch.bfloat16, device="cuda")
    dy[0] = 2.0
    dy[-tail:] = torch.arange(tail * out, device="cuda").view(tail, out) % 7 - 3
    dw, db = torch.empty(out, cols, device="cuda"), torch.empty(out, device="cuda")
    work = gq.alloc_workspace(gq.gq_act_wgrad_workspace(a, out))
    gq.gq_act_wgrad(a, dy, codes, steps, dw, db, workspace=work)
    d = dy[-tail:].double().cpu().numpy()
    want = d.T @ xr + 2.0
    mag = np.abs(d).T @ np.abs(xr) + 2.0
    assert (np.abs(dw.double().cpu().numpy() - want) <= 2 * 12 * 2.0 ** -24 * mag).all()
    assert np.array_equal(db.double().cpu().numpy(), d.sum(0) + 2.0)
    del dy, work

    # layer norm and its backward pass in place of x and of its output
    x[-tail:] += 1.0
    xl = x[-tail:].double().cpu().numpy()
    mean, rstd = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
    gq.gq_layer_norm(a, x, None, None, 1e-5, back, mean=mean, rstd=rstd)
    wy, wm, wr = A.layer_norm(xl, None, None, 1e-5)
    np.testing.assert_allclose(back[-tail:].double().cpu().numpy(), wy, rtol=2 ** -8, atol=1e-5)
    np.testing.assert_allclose(mean[-tail:].double().cpu().numpy(), wm, rtol=0, atol=1e-5)
    gq.gq_layer_norm_backward(a, back, x, mean, rstd, None, back)
    m, r = (t[-tail:].double().cpu().numpy() for t in (mean, rstd))
    dyl = torch.as_tensor(wy).bfloat16().double().numpy()
    wd, _, _ = A.layer_norm_backward(dyl, xl, m, r, None)
    # dx of dy = xh is 0 but for dy's roundings (2^-8 of a value up to 4.5)
    np.testing.assert_allclose(back[-tail:].double().cpu().numpy(), wd, rtol=0,
                               atol=4.5 * 2 ** -8 * 2)


@pytest.mark.parametrize("rows,cols,out", [(270_000, 8192, 24), (270_000, 8200, 24),
                                           (600_000, 8200, 70)])
def test_integer_product_past_32_bits(gq, rows, cols, out):
    """Also with a last k-tile that is short: what lies behind its end is not
    the codes two gigabytes further."""
    a = gq.act(rows, cols, torch.bfloat16)
    assert rows * a.pitch > 2 ** 31
    codes, steps = gq.alloc_act(a)
    codes.fill_(1)
    codes[:, cols:] = 0
    steps.fill_(0.5)
    rng = np.random.default_rng(11)
    last = rng.integers(-127, 128, (2, a.pitch)).astype(np.int8)
    last[:, cols:] = 0
    codes[-2:] = torch.as_tensor(last).cuda()
    w = rng.integers(-127, 128, (out, a.pitch)).astype(np.int8)
    w[:, cols:] = 0
    y = torch.full((rows, out), 9.0, dtype=torch.bfloat16, device="cuda")
    work = gq.alloc_workspace(gq.gq_act_linear_workspace(a, out))
    gq.gq_act_linear(a, codes, steps, torch.as_tensor(w).cuda(), torch.ones(out, device="cuda"),
                     None, y, workspace=work)
    half, one = np.full((2, 1), 0.5, np.float32), np.ones(out, np.float32)
    want = A.linear(last, half, w, one, None, cols)
    got = y[-2:].double().cpu().numpy()
    assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want)).all()
    rest = A.linear(np.ones((1, cols), np.int8), half[:1], w, one, None, cols)
    assert torch.equal(y[:-2], torch.as_tensor(rest).bfloat16().cuda().expand(rows - 2, out))


def test_few_tokens_through_a_weight_past_32_bits(gq):
    out, cols = 270_000, 8200
    a, aw = gq.act(3, cols, torch.float32), gq.act(out, cols, torch.float32)
    w, v = gq.alloc_act(aw)
    assert w.numel() > 2 ** 31
    w.fill_(1)
    w[:, cols:] = 0
    v.fill_(1.0)
    x, s = gq.alloc_act(a)
    x.fill_(2)
    x[:, cols:] = 0
    s.fill_(1.0)
    w[-1, :cols] = 3
    y = torch.zeros(3, out, device="cuda")
    gq.gq_act_linear(a, x, s, w, v.view(-1), None, y)
    assert (y[:, :-1] == 2 * cols).all() and (y[:, -1] == 6 * cols).all()
