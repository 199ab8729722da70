"""Rows in 8 bits and the product of 8-bit integers on the GPU against plain
64-bit forms (needs an MI355X).

The product's sums are exact.  What is rounded: the sum's conversion to fp32
(2^-24), two products with scales (2^-24 each, the second inside the addition of
the bias, which rounds once more) and the output: 2^-21 of the terms'
magnitudes and half a step.  A row's scale is one fp32 division, a value the
rounded quotient: 2^-22."""
import ctypes

import pytest
import torch

import _block_ref as bref
import _layer_ref as ref
import gated_delta_rule_66_amd as gdr
from gated_delta_rule_66_amd import _lib

pytestmark = pytest.mark.gpu
SLACK = 2.0 ** -21
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def make(M, N, K, bias=True, bdt=F32, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randint(-128, 128, s, generator=g, dtype=torch.int8)  # noqa: E731
    return dict(x=r(M, K), xs=torch.rand(M, generator=g) / 64 + 1e-4, w=r(N, K),
                ws=torch.rand(N, generator=g) / 64 + 1e-4,
                bias=torch.randn(N, generator=g).to(bdt) if bias else None)


def run(t, out=BF, **kw):
    g = {**{k: (None if v is None else v.cuda()) for k, v in t.items()}, **kw}
    return gdr.int8_matmul(g["x"], g["xs"], g["w"], g["ws"], g["bias"], out_dtype=out)


def held(t, y, out):
    want, mag = bref.product(t["x"], t["xs"], t["w"], t["ws"], t["bias"])
    ref.held("y", y, want, mag, out, SLACK)


@pytest.mark.parametrize("K", [1, 3, 15, 16, 17, 63, 64, 65, 127, 128, 130, 144, 250, 256, 511, 1000])
def test_lengths_of_the_sum(K):
    for M, N in ((1, 5), (19, 33), (70, 100)):
        t = make(M, N, K, seed=K)
        for out in (BF, HF, F32):
            held(t, run(t, out), out)


@pytest.mark.parametrize("M,N,K", [
    (1, 1, 1), (1, 4096, 4096), (7, 1000, 96), (16, 16, 64), (17, 17, 640), (32, 200, 80), (33, 12288, 256),
    (64, 31, 4096), (65, 4099, 48), (100, 257, 2505), (256, 4096, 512), (129, 16384, 128),
    (1000, 2500, 192), (1000, 2500, 177), (2049, 1025, 176), (2049, 1025, 175), (4097, 4098, 80), (4097, 4098, 16),
    (4097, 4098, 79), (5000, 4000, 272), (300, 60000, 64), (60000, 300, 64), (16641, 1024, 128),
    (200001, 90, 32), (3, 300001, 32),
    # rows that are padded for few tokens, or read where they lie
    (64, 12288, 1025), (33, 4100, 2049), (16, 12288, 513), (1, 12288, 514), (20, 9000, 4100)])
def test_sizes(M, N, K):
    t = make(M, N, K, seed=M)
    for out, bdt in ((BF, BF), (HF, F32)) if M * N > 1 << 22 else ((BF, BF), (HF, F32), (F32, F32)):
        t["bias"] = t["bias"].to(bdt)
        held(t, run(t, out), out)
    t["bias"] = None
    held(t, run(t, BF), BF)


def test_workspaces():
    """None where rows are multiples of 16 bytes; for few tokens, too, elsewhere."""
    size = lambda M, N, K, stride: _lib.lib.gdr_int8_matmul_workspace_size(  # noqa: E731
        ctypes.byref(_lib.Int8MatmulProblem(M, N, K, 0, 0, stride)))
    for M in (1, 20, 64, 65, 300, 3000, 20000):
        for N in (1, 70, 4096, 12288):
            assert size(M, N, 4096, 4096) == size(M, N, 16, 4096) == 0
    assert size(64, 12288, 4097, 4097) >= (64 + 12288) * 4112
    assert size(3000, 4096, 4096, 4097) >= 3000 * 4096
    assert size(3000, 4096, 4096, 4097) < 4096 * 4096


def test_largest_sums_are_exact():
    """65,536 products of 2^14: sums of 2^30, which fp32 holds exactly; and odd
    ones that only integers hold, seen through their remainder."""
    for M, N in ((3, 5), (300, 5000), (3000, 6000)):
        x = torch.full((M, 65536), -128, dtype=torch.int8, device="cuda")
        w = torch.full((N, 65536), -128, dtype=torch.int8, device="cuda")
        one, ones = torch.ones(M, device="cuda"), torch.ones(N, device="cuda")
        assert (gdr.int8_matmul(x, one, w, ones, out_dtype=F32) == 2.0 ** 30).all()
        # the first half's sum is cancelled but for one product of each
        x[:, 32768:] = 127
        w[:, 0] = 3
        y = gdr.int8_matmul(x, one, w, ones, out_dtype=F32)
        exact = 32767 * 2 ** 14 - 384 - 32768 * 127 * 128
        assert (y == float(torch.tensor(exact).float())).all() and abs(exact) < 2 ** 24


def test_scales_that_are_no_numbers():
    for M, N in ((20, 40), (4200, 4300)):
        t = make(M, N, 64)
        clean = run(t, BF)
        t["xs"][3], t["ws"][5], t["bias"][7] = float("nan"), float("inf"), float("nan")
        y = run(t, BF)
        rows, cols = torch.arange(M) != 3, torch.ones(N, dtype=torch.bool)
        cols[[5, 7]] = False
        assert torch.equal(y[rows][:, cols], clean[rows][:, cols])
        assert y[3].isnan().all() and y[:, 7].isnan().all() and not y[:, 5].isfinite().any()


def test_slices_shapes_and_addresses():
    """Slices of a wider tensor, leading dimensions, rows that begin at any
    byte; scales with a last dimension of one."""
    g = torch.Generator().manual_seed(1)
    for M, N, K in ((6, 50, 48), (90, 300, 128), (4200, 4200, 64)):
        t = make(M, N, K)
        base = run(t)
        wide = torch.randint(-128, 128, (M, K + 77), generator=g, dtype=torch.int8).cuda()
        for at in (0, 1, 16):
            wide[:, at:at + K] = t["x"].cuda()
            assert torch.equal(run(t, x=wide[:, at:at + K]), base)
        flat = torch.empty(N * K + 3, dtype=torch.int8, device="cuda")
        w = flat[3:].view(N, K)
        w.copy_(t["w"])
        assert torch.equal(run(t, w=w), base)
        assert torch.equal(run(t, w=t["w"].t().contiguous().t().cuda()), base)
        three = run(t, x=t["x"].cuda().view(2, M // 2, K), xs=t["xs"].cuda().view(2, M // 2, 1),
                    ws=t["ws"].cuda()[:, None])
        assert three.shape == (2, M // 2, N) and torch.equal(three.view(M, N), base)
        swapped = run(t, x=t["x"].cuda().view(2, M // 2, K).transpose(0, 1),
                      xs=t["xs"].cuda().view(2, M // 2).t())
        assert torch.equal(swapped.transpose(0, 1).reshape(M, N), base)
    one = run(t, x=t["x"].cuda()[5], xs=t["xs"].cuda()[5])
    assert one.shape == (4200,) and torch.equal(one, base[5])


def test_a_row_does_not_depend_on_the_others():
    """The same token alone, in a small and in a large batch: the same bits."""
    t = make(5000, 4100, 2048)
    y = run(t)
    for n in (1, 16, 17, 32, 33, 64, 65, 500, 1500):
        assert torch.equal(run({**t, "x": t["x"][:n], "xs": t["xs"][:n]}), y[:n]), n


def test_outputs_stay_inside():
    """What lies around y is left as it was."""
    for M, N, K in ((5, 33, 40), (130, 257, 144), (4100, 4111, 32), (4100, 4111, 31)):
        t = make(M, N, K, bias=False)
        g = {k: v.cuda() for k, v in t.items() if v is not None}
        buf = torch.full((M * N + 1024,), 7.0, device="cuda", dtype=BF)
        p = ctypes.byref(_lib.Int8MatmulProblem(M, N, K, 0, 0, K))
        n = _lib.lib.gdr_int8_matmul_workspace_size(p)
        ws = torch.full((n + 1024,), 7, device="cuda", dtype=torch.uint8)
        _lib.check(_lib.lib.gdr_int8_matmul(p, g["x"].data_ptr(), g["xs"].data_ptr(), g["w"].data_ptr(),
                                            g["ws"].data_ptr(), None, buf[512:].data_ptr(),
                                            ws[512:].data_ptr(), n, torch.cuda.current_stream().cuda_stream))
        torch.cuda.synchronize()
        assert (ws[:512] == 7).all() and (ws[512 + n:] == 7).all()
        assert (buf[:512] == 7).all() and (buf[512 + M * N:] == 7).all()
        assert torch.equal(buf[512:512 + M * N].view(M, N), run(t))


def test_products_past_two_to_the_31():
    """More than 2^31 outputs, and inputs of more than 2^31 bytes: rows at the
    end equal their own run."""
    t = {k: (None if v is None else v.cuda()) for k, v in make(1, 2100, 32).items()}
    M = (1 << 20) + 5000
    x = torch.randint(-128, 128, (M, 32), dtype=torch.int8, device="cuda")
    xs = torch.rand(M, device="cuda")
    y = gdr.int8_matmul(x, xs, t["w"], t["ws"], t["bias"])
    end = slice(M - 700, M)
    assert torch.equal(y[end], gdr.int8_matmul(x[end], xs[end], t["w"], t["ws"], t["bias"]))
    del y
    for M, N in ((33000, 40), (33000, 600), (40, 33000)):
        x = torch.randint(-128, 128, (max(M, 1), 65536), dtype=torch.int8, device="cuda")
        w = torch.randint(-128, 128, (N, 65536), dtype=torch.int8, device="cuda")
        xs, ws = torch.rand(M, device="cuda"), torch.rand(N, device="cuda")
        y = gdr.int8_matmul(x, xs, w, ws)
        assert torch.equal(y[-9:], gdr.int8_matmul(x[-9:], xs[-9:], w, ws))
        assert torch.equal(y[:, -9:], gdr.int8_matmul(x, xs, w[-9:], ws[-9:]))


# ---- rows -------------------------------------------------------------------------

@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("rows,D,dtype", [(1, 1, BF), (5, 7, F32), (130, 128, HF), (9, 1000, BF),
                                          (3, 5003, HF), (2, 4096, F32), (6, 16384, BF), (2, 20001, HF),
                                          (2, 40000, F32), (2, 65536, BF)])
def test_rows_in_eight_bits(rows, D, dtype, fmt, group):
    g = torch.Generator().manual_seed(0)
    x = torch.randn(rows, D, generator=g).to(dtype)
    if rows > 1:
        x[0] = 0
    q, scale = gdr.quantize_rows(x.cuda(), fmt, group)
    qv = bref.quantised(x, q, scale, fmt, group, 2.0 ** -22)
    if rows > 1:
        assert qv[0].abs().max() == 0
    top = qv.abs().amax()
    assert top == (448 if fmt == "fp8" else 127)
    wide = torch.zeros(rows, D + 13, dtype=dtype, device="cuda")
    wide[:, 5:5 + D] = x.cuda()
    q2, scale2 = gdr.quantize_rows(wide[:, 5:5 + D], fmt, group)
    assert torch.equal(q2.view(torch.uint8), q.view(torch.uint8)) and torch.equal(scale2, scale)


def test_rows_with_infinities_and_nans():
    x = torch.randn(5, 300).cuda()
    clean_q, clean_s = gdr.quantize_rows(x)
    x[1, 4], x[3, 200] = float("inf"), float("nan")
    q, s = gdr.quantize_rows(x)
    assert torch.equal(q[[0, 2, 4]], clean_q[[0, 2, 4]]) and torch.equal(s[[0, 2, 4]], clean_s[[0, 2, 4]])
    assert s[1, 0] == float("inf") and s[3, 0].isnan() and (q[[1, 3]] == 0).all()
    q, s = gdr.quantize_rows(x, group_size=128)
    assert s[3, :1].isfinite() and s[3, 1].isnan() and s[1, 1:].isfinite().all()
    assert torch.equal(q[1, 128:], gdr.quantize_rows(x[1:2, 128:], group_size=128)[0][0])


def test_a_quantised_projection():
    """Weights and tokens by quantize_rows, then the product: what the two hold
    in 8 bits, exactly; and within the two quantisations of the product of
    what they were made from (half a step of each row's largest, 1 / 254, on
    either operand: at most sum |x| |w| / 254 per row's largest, as a bound)."""
    g = torch.Generator().manual_seed(3)
    x, w = torch.randn(50, 700, generator=g), torch.randn(90, 700, generator=g) / 26
    (xq, xs), (wq, ws) = gdr.quantize_rows(x.to(BF).cuda()), gdr.quantize_rows(w.to(BF).cuda())
    y = gdr.int8_matmul(xq, xs, wq, ws, out_dtype=F32)
    held(dict(x=xq, xs=xs, w=wq, ws=ws, bias=None), y, F32)
    a, b = x.to(BF).double(), w.to(BF).double()
    ex, ew = a.abs().amax(1, keepdim=True) / 254, b.abs().amax(1, keepdim=True) / 254
    bar = ex * b.abs().sum(1) + (a.abs() + ex).sum(1, keepdim=True) * ew.t()
    assert ((ref.d(y) - a @ b.t()).abs() <= bar * (1 + 2.0 ** -10)).all()
