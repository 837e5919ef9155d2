"""Refusals and sizes of the 8-bit activation operators' C entry points: every
argument error is found on the host before any launch (no GPU needed)."""
import ctypes as C

import pytest

M = 1 << 24                    # fake addresses, aligned and far apart


@pytest.fixture(scope="module")
def gq():
    from communication_efficient_gradient_amd import gq as mod
    return mod


def act(gq, rows=10, cols=100, dtype=1, group=0):
    return gq.gq_act(rows, cols, dtype, group)


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), -1), (dict(cols=0), -1), (dict(cols=(1 << 20) + 1), -1),
    (dict(rows=1 << 38), -1), (dict(dtype=3), -2), (dict(dtype=-1), -2),
    (dict(group=16), -1), (dict(group=48), -1), (dict(group=65536), -1),
    (dict(group=-32), -1)])
def test_bad_descriptors(gq, kw, status):
    L, a, b = gq.lib(), act(gq, **kw), C.c_int64()
    assert L.gq_act_size(C.byref(a), C.byref(b), None) == status
    assert L.gq_act_pack(C.byref(a), M, 1 << 21, 2 * M, 3 * M, None) == status
    assert L.gq_layer_norm_workspace(C.byref(a), C.byref(b)) == status
    assert L.gq_act_linear_workspace(C.byref(a), 5, C.byref(b)) == status
    assert L.gq_act_wgrad_workspace(C.byref(a), 5, C.byref(b)) == status
    assert L.gq_act_size(None, None, None) == -1


def test_sizes(gq):
    for rows, cols, group, want in [
            (10, 100, 0, (1120, 10)), (10, 100, 32, (1120, 40)),
            (0, 5, 0, (0, 0)), (3, 16, 64, (48, 3)), (3, 129, 128, (432, 6)),
            (1 << 18, 1 << 20, 32768, (1 << 38, 1 << 23))]:
        a = act(gq, rows, cols, 0, group)
        assert gq.gq_act_size(a) == want
    import torch
    a = gq.act(10, 100, torch.float16, 32)
    assert (a.pitch, a.groups, a.dtype) == (112, 4, gq.GQ_F16)
    with pytest.raises(TypeError):
        gq.act(10, 100, torch.float64)
    with pytest.raises(gq.GQError) as ex:
        gq.act(10, 100, torch.float16, 33)
    assert ex.value.status == gq.GQ_EINVAL


def test_pack_unpack_refusals(gq):
    L, a = gq.lib(), act(gq)
    for f, order in ((L.gq_act_pack, (0, 1, 2, 3)), (L.gq_act_unpack, (2, 3, 0, 1))):
        def call(x=M, ld=100, codes=2 * M, steps=3 * M, desc=a):
            v = [x, ld, codes, steps]
            return f(C.byref(desc), *[v[i] for i in order], None)
        assert call(x=None) == -1
        assert call(x=M + 1) == -1                     # bf16: 2-byte alignment
        assert call(ld=99) == -1
        assert call(ld=1 << 42) == -1
        assert call(codes=None) == -1
        assert call(codes=2 * M + 8) == -1
        assert call(steps=None) == -1
        assert call(steps=3 * M + 2) == -1
        assert call(codes=M + 992) == -1               # inside x
        if f is L.gq_act_pack:
            assert call(steps=2 * M + 16) == -1        # inside codes, both written
        assert call(x=2 * M + 1118) == -1              # codes' last bytes
        # no rows: nothing to point to
        assert call(x=None, codes=None, steps=None, desc=act(gq, rows=0)) == 0


def test_linear_refusals(gq):
    L = gq.lib()

    def call(out=50, codes=M, steps=2 * M, wc=3 * M, ws=4 * M, bias=5 * M, y=6 * M,
             ld=50, work=7 * M, nb=None, desc=act(gq)):
        need = C.c_int64()
        if nb is None:
            L.gq_act_linear_workspace(C.byref(desc), out, C.byref(need))
            nb = need.value
        return L.gq_act_linear(C.byref(desc), out, codes, steps, wc, ws, bias, y, ld,
                               work, nb, None)

    assert call(out=0) == -1
    assert call(desc=act(gq, group=32)) == -2          # one step per row only
    assert call(desc=act(gq, cols=131072)) == -2       # the sum would not fit 32 bits
    assert call(desc=act(gq, rows=1 << 31, cols=1), out=64, nb=1 << 40) == -2  # too many tiles
    assert call(codes=None) == -1
    assert call(steps=None) == -1
    assert call(wc=None) == -1
    assert call(wc=3 * M + 4) == -1
    assert call(ws=None) == -1
    assert call(bias=5 * M + 1) == -1
    assert call(y=None) == -1
    assert call(ld=49) == -1
    assert call(y=3 * M) == -1                         # over the weight
    assert call(y=5 * M + 196) == -1                   # over the bias's last value
    big = dict(desc=act(gq, rows=1100, cols=60000), out=1000, ld=1000, codes=M, steps=8 * M,
               wc=9 * M, ws=14 * M, bias=15 * M, y=16 * M, work=17 * M)
    need = C.c_int64()
    assert L.gq_act_linear_workspace(C.byref(big["desc"]), 1000, C.byref(need)) == 0
    assert need.value > 0
    assert call(**big, nb=need.value - 1) == -1
    assert call(**{**big, "work": None}) == -1
    assert call(**{**big, "work": 17 * M + 8}) == -1
    assert call(**{**big, "work": M}) == -1            # over the codes
    assert call(desc=act(gq, rows=0), codes=None, steps=None, y=None) == 0


def test_wgrad_refusals(gq):
    L = gq.lib()

    def call(out=50, dy=M, ld=50, codes=2 * M, steps=3 * M, beta=0.0, dw=4 * M,
             db=5 * M, work=6 * M, nb=None, desc=act(gq)):
        need = C.c_int64()
        if nb is None:
            L.gq_act_wgrad_workspace(C.byref(desc), out, C.byref(need))
            nb = need.value
        return L.gq_act_wgrad(C.byref(desc), out, dy, ld, codes, steps, beta, dw, db,
                              work, nb, None)

    assert call(out=0) == -1
    assert call(dy=None) == -1
    assert call(dy=M + 1) == -1
    assert call(ld=49) == -1
    assert call(codes=2 * M + 8) == -1
    assert call(steps=None) == -1
    assert call(beta=float("nan")) == -1
    assert call(beta=float("inf")) == -1
    assert call(dw=None) == -1
    assert call(dw=4 * M + 2) == -1
    assert call(db=5 * M + 2) == -1
    assert call(dw=M + 64) == -1                       # over dy
    assert call(db=4 * M + 4 * 4999) == -1             # over dweight's last value
    long = act(gq, rows=100000)
    need = C.c_int64()
    assert L.gq_act_wgrad_workspace(C.byref(long), 50, C.byref(need)) == 0
    assert need.value > 0
    assert call(desc=long, nb=need.value - 1) == -1
    assert call(desc=long, work=None) == -1
    assert call(desc=long, work=2 * M) == -1


def test_layer_norm_refusals(gq):
    L = gq.lib()

    def fwd(x=M, ldx=100, w=2 * M, b=3 * M, eps=1e-5, y=4 * M, ldy=100, mean=5 * M,
            rstd=6 * M, xc=7 * M, xs=8 * M, yc=9 * M, ys=10 * M, desc=act(gq)):
        return L.gq_layer_norm(C.byref(desc), x, ldx, w, b, eps, y, ldy, mean, rstd,
                               xc, xs, yc, ys, None)

    assert fwd(x=None) == -1
    assert fwd(ldx=99) == -1
    assert fwd(eps=-1e-6) == -1
    assert fwd(eps=float("nan")) == -1
    assert fwd(w=2 * M + 1) == -1
    assert fwd(xs=None) == -1                          # half a form
    assert fwd(yc=None) == -1
    assert fwd(y=None, yc=None, ys=None) == -1         # no output at all
    assert fwd(y=None, desc=act(gq, cols=20000), ldx=20000) == -2
    assert fwd(y=None, desc=act(gq, cols=5000, group=1024), ldx=5000) == -2
    assert fwd(y=M + 200) == -1                        # over x, not the same matrix
    assert fwd(y=M, ldy=101) == -1
    assert fwd(mean=M + 4) == -1
    assert fwd(y=M, xc=M + 64) == -1                   # y in place, the form is not
    assert fwd(mean=5 * M, rstd=5 * M) == -1
    assert fwd(x=None, y=None, mean=None, rstd=None, xc=None, xs=None, yc=None,
               ys=None, desc=act(gq, rows=0)) == 0

    def bwd(dy=M, ldd=100, x=2 * M, ldx=100, c=None, s=None, mean=3 * M, rstd=4 * M,
            w=5 * M, dx=6 * M, ldo=100, beta=0.0, dw=7 * M, db=8 * M, work=9 * M,
            nb=None, desc=act(gq)):
        need = C.c_int64()
        if nb is None:
            L.gq_layer_norm_workspace(C.byref(desc), C.byref(need))
            nb = need.value
        return L.gq_layer_norm_backward(C.byref(desc), dy, ldd, x, ldx, c, s, mean, rstd,
                                        w, dx, ldo, beta, dw, db, work, nb, None)

    assert bwd(dy=None) == -1
    assert bwd(x=None) == -1                           # neither x nor its form
    assert bwd(c=10 * M, s=11 * M) == -1               # both
    assert bwd(x=None, c=10 * M) == -1                 # half a form
    assert bwd(mean=None) == -1
    assert bwd(rstd=None) == -1
    assert bwd(beta=float("inf")) == -1
    assert bwd(dx=None) == -1
    assert bwd(dx=M + 100) == -1
    assert bwd(dw=M) == -1                             # over dy
    assert bwd(dx=M, dw=M) == -1                       # dx in place of dy, dweight too
    assert bwd(work=None) == -1
    assert bwd(nb=16) == -1
    assert bwd(work=2 * M) == -1


def test_binding_checks(gq):
    import torch
    a = gq.act(4, 6, torch.bfloat16)
    host = torch.zeros(4, 6, dtype=torch.bfloat16)
    codes = torch.zeros(4, 16, dtype=torch.int8)
    steps = torch.zeros(4, 1)
    with pytest.raises(ValueError, match="device tensor"):
        gq.gq_act_pack(a, host, codes, steps)
    with pytest.raises(TypeError):
        gq.gq_act_pack(a, None, codes, steps)
    with pytest.raises(ValueError, match="device tensor"):
        gq.gq_layer_norm(a, host, None, None, 1e-5, host)
    with pytest.raises(ValueError, match="matrix"):
        gq.gq_act_wgrad(a, host[0], codes, steps, torch.zeros(6))
    with pytest.raises(gq.GQError) as ex:
        gq.gq_act_linear_workspace(gq.act(4, 64, torch.float32, 32), 8)
    assert ex.value.status == gq.GQ_EUNSUPPORTED
    assert gq.alloc_workspace(0) is None
