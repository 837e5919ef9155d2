"""The binding's descriptor of activations: built directly or changed, it says
and checks what the one from act() does (no GPU needed)."""
import copy

import pytest
import torch


@pytest.fixture(scope="module")
def gq():
    from communication_efficient_gradient_amd import gq as mod
    return mod


def facts(a):
    return a.rows, a.cols, a.torch_dtype, a.pitch, a.groups


@pytest.mark.parametrize("rows,cols,dtype,group", [
    (4, 6, torch.float32, 0), (10, 100, torch.bfloat16, 32), (0, 129, torch.float16, 128)])
def test_built_directly(gq, rows, cols, dtype, group):
    want = gq.act(rows, cols, dtype, group)
    a = gq.gq_act(rows, cols, gq.DTYPES[dtype], group)
    assert facts(a) == facts(want)
    assert gq.gq_act_size(a) == gq.gq_act_size(want)
    assert gq.gq_layer_norm_workspace(a) == gq.gq_layer_norm_workspace(want)
    assert gq.gq_act_wgrad_workspace(a, 8) == gq.gq_act_wgrad_workspace(want, 8)
    codes, steps = gq.alloc_act(a, device="cpu")
    assert codes.shape == (rows, want.pitch) and steps.shape == (rows, want.groups)
    assert gq.gq_act(rows=3, cols=5, dtype=gq.GQ_F16).pitch == 16


def test_changed(gq):
    a = gq.act(4, 100, torch.bfloat16, 32)
    assert facts(a) == (4, 100, torch.bfloat16, 112, 4)
    a.rows, a.cols, a.dtype, a.group = 9, 250, gq.GQ_F32, 64
    assert facts(a) == (9, 250, torch.float32, 256, 4)
    a.group = 0
    assert a.groups == 1
    assert gq.alloc_act(a, device="cpu")[0].shape == (9, 256)
    b = copy.copy(a)
    b.cols = 17
    assert facts(a)[3] == 256 and facts(b)[3] == 32


def test_what_the_library_refuses(gq):
    for bad, status in ((gq.gq_act(4, 6, 3, 0), gq.GQ_EUNSUPPORTED),
                        (gq.gq_act(4, 0, 0, 0), gq.GQ_EINVAL),
                        (gq.gq_act(4, 6, 0, 33), gq.GQ_EINVAL)):
        with pytest.raises(gq.GQError) as ex:
            bad.pitch
        assert ex.value.status == status
        with pytest.raises(gq.GQError):
            gq.gq_act_pack(bad, torch.zeros(4, 6), torch.zeros(4, 16, dtype=torch.int8),
                           torch.zeros(4, 1))
    a = gq.act(4, 6)
    a.cols = -1
    with pytest.raises(gq.GQError):
        a.groups
    with pytest.raises(AttributeError):
        a.nothing


def test_calls_check_the_type_of_a_direct_descriptor(gq):
    a = gq.gq_act(4, 6, gq.GQ_BF16, 0)
    host = torch.zeros(4, 6, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="device tensor"):
        gq.gq_act_pack(a, host, torch.zeros(4, 16, dtype=torch.int8), torch.zeros(4, 1))


@pytest.mark.parametrize("rows", [1, 8, 9, 16, 17, 33, 64])
def test_few_tokens_need_no_workspace(gq, rows):
    for out in (1, 64, 4097, 8193, 40000, 1 << 18):
        for cols in (1, 1000, 16384, 131071):
            assert gq.gq_act_linear_workspace(gq.act(rows, cols, torch.bfloat16), out) == 0
