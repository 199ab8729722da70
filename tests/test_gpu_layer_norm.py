"""The RMS norm with the residual's addition on the GPU against a plain 64-bit
form (needs an MI355X).

Tolerances: an output is one rounding to its type plus fp32 arithmetic.  The
mean of squares of D values summed by at most 64 + 10 + 16 additions in a row
is off by 90 2^-24 relative, its root by half of that, the products by a few
2^-24: 2^-17 of the magnitudes covers them, for the row's mean in the gradient
too.  The weight gradient adds rows / blocks + blocks / 4 values in a row, at
most 8 + 256 here: 2^-15.  A value in 8 bits is within half a step of y /
scale, and within a whole step where fp32 rounding moves it over a border."""
import pytest
import torch

import _layer_ref as ref
import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
SLACK, SUM_SLACK = 2.0 ** -17, 2.0 ** -15
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def make(rows, D, dtype, rdt=None, wdt=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=r(rows, D).to(dtype), w=(1 + r(D) / 4).to(wdt or dtype),
                res=None if rdt is None else (2 * r(rows, D)).to(rdt), dy=r(rows, D).to(dtype),
                dh=None if rdt is None else r(rows, D).to(rdt))


def dev(t):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in t.items()}


CASES = {
    "one_value": (1, 1, F32, None, None),
    "one_row": (1, 4096, BF, BF, None),
    "narrow_odd": (7, 45, HF, F32, F32),
    "wave": (130, 512, BF, F32, None),
    "wave2": (33, 1000, F32, F32, None),
    "two_per_thread": (9, 4096, BF, BF, F32),
    "odd": (5, 5003, HF, HF, None),
    "no_residual": (65, 2049, BF, None, F32),
    "wide": (3, 16384, BF, F32, None),
    "wider": (2, 20001, HF, HF, None),
    "widest": (2, 65536, BF, BF, None),
    "many_rows": (5000, 72, BF, BF, None),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_gradients(name):
    rows, D, dtype, rdt, wdt = CASES[name]
    t = make(rows, D, dtype, rdt, wdt)
    g = dev(t)
    leaves = [g[k].requires_grad_(True) for k in ("x", "w", "res") if g[k] is not None]
    out = gdr.rms_norm(g["x"], g["w"], EPS, residual=g["res"])
    outs, go = ([out], [g["dy"]]) if rdt is None else (list(out), [g["dy"], g["dh"]])
    grads = torch.autograd.grad(outs, leaves, go)
    torch.cuda.synchronize()
    r = ref.norm(t["x"], t["w"], EPS, t["res"], t["dy"], t["dh"])
    ref.held("y", outs[0], r["y"], r["y"].abs(), dtype, SLACK)
    if rdt is not None:
        assert torch.equal(outs[1].cpu().double(), r["h"])
    ref.held("dx", grads[0], r["dx"], r["dxm"], dtype, SLACK)
    ref.held("dw", grads[1], r["dw"], r["dwm"], grads[1].dtype, SUM_SLACK)
    if rdt is not None:
        ref.held("dres", grads[2], r["dx"], r["dxm"], rdt, SLACK)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("rows,D,dtype,rdt", [(1, 4096, BF, BF), (5, 45, HF, F32), (6, 1000, F32, None),
                                              (3, 5003, BF, F32), (130, 128, HF, HF),
                                              (2, 20000, BF, None), (3, 129, BF, BF)])
def test_eight_bits(rows, D, dtype, rdt, fmt, group):
    t = make(rows, D, dtype, rdt)
    t["x"][0] = 0
    if t["res"] is not None:
        t["res"][0] = 0                      # a row of zeros stays zeros
    g = dev(t)
    q, scale, h = gdr.rms_norm_quant(g["x"], g["w"], EPS, g["res"], format=fmt, group_size=group)
    r = ref.norm(t["x"], t["w"], EPS, t["res"])
    top = 448.0 if fmt == "fp8" else 127.0
    width = group or D
    y = torch.nn.functional.pad(r["y"], (0, (-D) % width)).unflatten(1, (-1, width))
    want = (y.abs().amax(-1) / top).clamp_min(2.0 ** -126)
    got = scale.cpu().double().reshape(want.shape)
    assert ((got - want).abs() <= SLACK * want).all()
    v = (y / got[..., None]).flatten(1)[:, :D]
    qv = q.cpu().double() if fmt == "int8" else q.cpu().float().double()
    # e4m3: half a step is 2^-4 relative, 2^-10 below its normal range; int8: 1/2
    bar = (v.abs() * 2.0 ** -4).clamp_min(2.0 ** -10) if fmt == "fp8" else torch.full_like(v, 0.5)
    assert ((qv - v).abs() <= bar * (1 + SLACK) + v.abs() * SLACK * 2).all()
    assert qv[0].abs().max() == 0
    assert (h is None) == (rdt is None)
    if h is not None:
        assert torch.equal(h.cpu().double(), r["h"])


def test_nans_and_infinities_stay_in_their_row():
    t = dev(make(4, 300, BF, BF))
    clean = gdr.rms_norm(t["x"], t["w"], EPS, t["res"])[0]
    x = t["x"].clone()
    x[1, 7] = float("nan")
    x[2, 9] = float("inf")
    y = gdr.rms_norm(x, t["w"], EPS, t["res"])[0]
    assert torch.equal(y[[0, 3]], clean[[0, 3]])
    assert y[1].isnan().all() and y[2, 9].isnan()
    for fmt in ("fp8", "int8"):
        q, scale, _ = gdr.rms_norm_quant(x, t["w"], EPS, t["res"], format=fmt)
        assert scale[1:3, 0].isnan().all() and scale[[0, 3]].isfinite().all()
    q, scale, _ = gdr.rms_norm_quant(x, t["w"], EPS, t["res"], format="int8", group_size=128)
    assert (q[1] == 0).all() and scale[1].isnan().all()


def test_rows_of_a_wider_tensor_and_leading_dimensions():
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(3, 7, 100, generator=g).to(BF).cuda()
    w = torch.ones(33, dtype=BF, device="cuda")
    x = wide[:, :, 3:36]
    dy = torch.randn(3, 7, 33, generator=g).to(BF).cuda()
    a = x.detach().requires_grad_(True)
    b = x.detach().contiguous().requires_grad_(True)
    ya, yb = gdr.rms_norm(a, w), gdr.rms_norm(b, w)
    assert ya.shape == (3, 7, 33) and torch.equal(ya, yb)
    assert torch.equal(torch.autograd.grad(ya, a, dy)[0], torch.autograd.grad(yb, b, dy)[0])
    assert torch.equal(gdr.rms_norm(x.transpose(0, 1), w), yb.transpose(0, 1))
    assert torch.equal(gdr.rms_norm(x[0, 0], w), yb[0, 0])
    four = wide.reshape(3, 7, 4, 25)
    assert torch.equal(gdr.rms_norm(four, w[:25]), gdr.rms_norm(four.reshape(84, 25), w[:25]).reshape(3, 7, 4, 25))


def test_gradient_against_differences():
    """fp32, random directions; with step 2^-7 the central difference is off
    by about h^2 and 2^-23 / h of the outputs, under 1e-3 of the root of the
    summed squares."""
    t = dev(make(6, 200, F32, F32, seed=4))
    out = gdr.rms_norm_fwd(t["x"], t["w"], EPS, t["res"])
    dx, dres, dw = gdr.rms_norm_bwd(t["dy"], out[1], t["w"], out[2], t["dh"], has_residual=True)
    gen = torch.Generator().manual_seed(2)
    h = 2.0 ** -7
    for k, g in (("x", dx), ("res", dres), ("w", dw)):
        v = torch.randn(t[k].shape, generator=gen).cuda()

        def value(s):
            q = dict(t)
            q[k] = t[k] + s * v
            y, hh, _ = gdr.rms_norm_fwd(q["x"], q["w"], EPS, q["res"])
            return (y.double() * t["dy"]).sum() + (hh.double() * t["dh"]).sum()

        diff = (value(h) - value(-h)) / (2 * h)
        want = (g.double() * v).sum()
        scale = (g.double() * v).square().sum().sqrt()
        assert abs(diff - want) <= 1e-3 * scale, (k, float(diff), float(want))


def test_captured_and_replayed():
    t = dev(make(70, 1500, BF, F32))

    def step():
        y, h, rstd = gdr.rms_norm_fwd(t["x"], t["w"], EPS, t["res"])
        g = gdr.rms_norm_bwd(t["dy"], h, t["w"], rstd, t["dh"], has_residual=True)
        q, s, _ = gdr.rms_norm_quant(t["x"], t["w"], EPS, t["res"], group_size=128)
        return (y, h, rstd) + g + (q.view(torch.uint8), s)

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for _ in range(3):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        step()


def test_python_refusals():
    t = dev(make(4, 32, BF, BF))
    x, w = t["x"], t["w"]
    for call, name in [
        (lambda: gdr.rms_norm(x, w[:16]), "GDR_ERR_SHAPE"),
        (lambda: gdr.rms_norm(x, w.half()), "GDR_ERR_DTYPE"),
        (lambda: gdr.rms_norm(x, w, residual=t["res"][:2]), "GDR_ERR_SHAPE"),
        (lambda: gdr.rms_norm(x, w, residual=t["res"].half()), "GDR_ERR_DTYPE"),
        (lambda: gdr.rms_norm(x, w, eps=-1.0), "GDR_ERR_ARG"),
        (lambda: gdr.rms_norm(x.double(), w), "GDR_ERR_DTYPE"),
        (lambda: gdr.rms_norm(x, w.cpu()), "GDR_ERR_DEVICE"),
        (lambda: gdr.rms_norm(x[:0], w), "GDR_ERR_SHAPE"),
        (lambda: gdr.rms_norm_quant(x, w, format="int4"), "GDR_ERR_ARG"),
        (lambda: gdr.rms_norm_quant(x, w, format=None), "GDR_ERR_ARG"),
        (lambda: gdr.rms_norm_quant(x, w, group_size=64), "GDR_ERR_ARG"),
        (lambda: gdr.rms_norm_bwd(t["dy"], x, w, x[:, 0].float(), t["dh"]), "GDR_ERR_ARG"),
        (lambda: gdr.rms_norm_bwd(t["dy"], x[:2], w, x[:, 0].float()), "GDR_ERR_SHAPE"),
    ]:
        with pytest.raises(gdr.GdrError) as e:
            call()
        assert e.value.name == name
