"""GPU pack and unpack of matrices that need more workgroups than one launch
holds (2^24 of 256 threads)."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def gq():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from communication_efficient_gradient_amd import gq
    return gq


@pytest.fixture(autouse=True)
def memory_back():
    yield
    if torch.cuda.is_available():
        torch.cuda.empty_cache()


def need(gib):
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < gib * 2 ** 30:
        pytest.skip(f"needs {gib} GiB of device memory")


def parts(rows, n=1 << 26):
    return [slice(lo, min(rows, lo + n)) for lo in range(0, rows, n)]


@pytest.mark.parametrize("group", [32, 512])
def test_pack_of_very_many_short_rows(gq, group):
    """64 rows of one column per workgroup; any group that holds the row."""
    need(40)
    rows = (1 << 30) + 1000
    x = torch.empty(rows, 1, dtype=torch.bfloat16, device="cuda")
    for p in parts(rows):
        x[p, 0] = (torch.arange(p.start, p.stop, device="cuda") * 40503 % 255 - 127).bfloat16()
    a = gq.act(rows, 1, torch.bfloat16, group)
    codes, steps = gq.alloc_act(a)
    for p in parts(rows):
        codes[p].fill_(55)
    steps.fill_(5.0)
    gq.gq_act_pack(a, x, codes, steps)
    for p in parts(rows):
        c, v = codes[p, 0].float(), x[p, 0].float()
        assert (c * steps[p, 0] == v).all()          # 7 bits: nothing is rounded
        assert ((c.abs() >= 64) | (v == 0)).all()    # and the smallest step is taken
        assert (codes[p, 1:].view(torch.uint8).amax(1) == 0).all()
    back = torch.full_like(x, 3)
    gq.gq_act_unpack(a, codes, steps, back)
    assert all(torch.equal(back[p], x[p]) for p in parts(rows))


def test_unpack_of_very_many_rows(gq):
    """Two units of one row per workgroup, and two units to a row."""
    need(120)
    rows, cols = (1 << 24) + 100, 2056
    a = gq.act(rows, cols, torch.bfloat16)
    codes, steps = gq.alloc_act(a)
    for p in parts(rows, 1 << 21):
        r = torch.arange(p.start, p.stop, device="cuda")[:, None]
        codes[p] = ((r + torch.arange(a.pitch, device="cuda")) % 255 - 127).to(torch.int8)
        steps[p] = torch.exp2((r % 5).float())
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    gq.gq_act_unpack(a, codes, steps, x)
    for p in parts(rows, 1 << 21):
        assert torch.equal(x[p], codes[p, :cols].bfloat16() * steps[p].bfloat16())
