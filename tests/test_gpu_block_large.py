"""The operators at a layer's ends where offsets pass 32 bits (needs an MI355X
and some 40 GB): reads through strides of gigabytes, and outputs of more than
2^31 elements.  A row's result depends on that row alone, so the last rows are
held bit for bit against a small call on them; weights' gradients, which sum
over all rows, are held where one row has a gradient."""
import pytest
import torch

import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
BF = torch.bfloat16
D, ROWS, TAIL = 16384, 131072 + 64, 8      # rows * D passes 2^31


@pytest.fixture(autouse=True)
def free():
    yield
    torch.cuda.empty_cache()


def far(rows=1100, width=512, stride=1 << 21, dtype=BF, seed=0):
    """(rows one stride apart, the last past 2^31 elements; the same packed)."""
    g = torch.Generator().manual_seed(seed)
    store = torch.zeros(rows * stride, dtype=dtype, device="cuda")
    x = store.view(rows, stride)[:, :width]
    if dtype is torch.int8:
        x.copy_(torch.randint(-128, 128, (rows, width), generator=g, dtype=dtype))
    else:
        x.copy_(torch.randn(rows, width, generator=g))
    assert x.stride(0) * (rows - 1) > 1 << 31
    return x, x.contiguous()


def test_reads_through_wide_strides():
    x, xc = far()
    w = torch.randn(512, generator=torch.Generator().manual_seed(1)).to(BF).cuda()
    for a, b in zip(gdr.quantize_rows(x), gdr.quantize_rows(xc)):
        assert torch.equal(a, b)
    for how in (dict(norm_group=0), dict(norm_group=128, norm_before_gate=False), dict(norm_group=256)):
        v = w[:how["norm_group"]] if how["norm_group"] else w
        for a, b in zip(gdr.gated_rms_norm_fwd(x, x, v, **how), gdr.gated_rms_norm_fwd(xc, xc, v, **how)):
            assert torch.equal(a, b)
    res = torch.randn(x.shape, generator=torch.Generator().manual_seed(2)).cuda()
    for a, b in zip(gdr.sandwich_rms_norm_fwd(x, res, w, w, gate=x), gdr.sandwich_rms_norm_fwd(xc, res, w, w, gate=xc)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("width", [512, 517])
def test_product_of_far_rows(width):
    x, xc = far(width=width, dtype=torch.int8)
    g = torch.Generator().manual_seed(3)
    w = torch.randint(-128, 128, (80, width), generator=g, dtype=torch.int8).cuda()
    xs, ws = torch.rand(1100, generator=g).cuda(), torch.rand(80, generator=g).cuda()
    assert torch.equal(gdr.int8_matmul(x, xs, w, ws), gdr.int8_matmul(xc, xs, w, ws))
    assert torch.equal(gdr.int8_matmul(x[-9:], xs[-9:], w, ws), gdr.int8_matmul(xc[-9:], xs[-9:], w, ws))


def wide(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(ROWS, D, generator=g, device="cuda", dtype=BF)


@pytest.mark.parametrize("group", [128, 16384, 2048])
def test_gated_norm_past_32_bits(group):
    x, z = wide(0), wide(1)
    w = torch.randn(group, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    y, rstd = gdr.gated_rms_norm_fwd(x, z, w, norm_group=group)
    ys, rs = gdr.gated_rms_norm_fwd(x[-TAIL:], z[-TAIL:], w, norm_group=group)
    assert torch.equal(y[-TAIL:], ys) and torch.equal(rstd[-TAIL:], rs)
    del y
    q, scale = gdr.gated_rms_norm_quant(x, z, w, norm_group=group, format="int8", group_size=128)
    qs, ss = gdr.gated_rms_norm_quant(x[-TAIL:], z[-TAIL:], w, norm_group=group, format="int8", group_size=128)
    assert torch.equal(q[-TAIL:], qs) and torch.equal(scale[-TAIL:], ss)
    del q
    dy = torch.zeros_like(x)
    dy[-1] = x[0]
    dx, dz, dw = gdr.gated_rms_norm_bwd(dy, x, z, w, rstd, norm_group=group)
    ex, ez, ew = gdr.gated_rms_norm_bwd(dy[-TAIL:], x[-TAIL:], z[-TAIL:], w, rstd[-TAIL:], norm_group=group)
    assert torch.equal(dx[-TAIL:], ex) and torch.equal(dz[-TAIL:], ez)
    # the walkers add zeros to one row's terms, which rounds nothing; its groups'
    # terms may be added in another order: 16384 / group - 1 additions of 2^-24 of
    # the terms' magnitudes on either side, and two roundings to bf16 of 2^-8
    u = x[-1].double() * rstd[-1].double().repeat_interleave(group)
    act = z[-1].double() * torch.sigmoid(z[-1].double())
    size = (dy[-1].double() * u * act).abs().view(-1, group).sum(0)
    tol = 2 * (D // group) * 2.0 ** -24 * size + 2 * 2.0 ** -8 * ew.abs().double()
    assert ((dw.double() - ew.double()).abs() <= tol).all()


def test_sandwich_norm_past_32_bits():
    x, res = wide(0), wide(1)
    w = torch.randn(D, generator=torch.Generator().manual_seed(2)).to(BF).cuda()
    y, h, rx, rh = gdr.sandwich_rms_norm_fwd(x, res, w, w)
    small = gdr.sandwich_rms_norm_fwd(x[-TAIL:], res[-TAIL:], w, w)
    for a, b in zip((y, h, rx, rh), small):
        assert torch.equal(a[-TAIL:], b)
    dy = torch.zeros_like(x)
    dy[-1] = x[0]
    got = gdr.sandwich_rms_norm_bwd(dy, None, x, h, w, w, rx, rh)
    want = gdr.sandwich_rms_norm_bwd(dy[-TAIL:], None, x[-TAIL:], h[-TAIL:], w, w, rx[-TAIL:], rh[-TAIL:])
    assert torch.equal(got[0][-TAIL:], want[0]) and torch.equal(got[1][-TAIL:], want[1])
    for i in (2, 3):  # sums of one row's terms and of zeros
        assert torch.equal(got[i], want[i])


def test_product_past_32_bits():
    g = torch.Generator().manual_seed(0)
    M, N, K = ROWS, D, 64
    x = torch.randint(-128, 128, (M, K), generator=g, dtype=torch.int8).cuda()
    w = torch.randint(-128, 128, (N, K), generator=g, dtype=torch.int8).cuda()
    xs, ws = torch.rand(M, generator=g).cuda(), torch.rand(N, generator=g).cuda()
    y = gdr.int8_matmul(x, xs, w, ws)
    assert torch.equal(y[-300:], gdr.int8_matmul(x[-300:], xs[-300:], w, ws))
    q, scale = gdr.quantize_rows(y)
    qs, ss = gdr.quantize_rows(y[-TAIL:])
    assert torch.equal(q[-TAIL:], qs) and torch.equal(scale[-TAIL:], ss)
