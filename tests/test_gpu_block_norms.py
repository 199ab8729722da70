"""The gated norm and the sandwich norm on the GPU against plain 64-bit forms
(needs an MI355X).

Tolerances: outputs are one rounding to their type plus fp32 arithmetic.  The
statistics are formed in 64 bits.  A gate's sigmoid is 1 / (1 + e^-z): the
exponent's argument is rounded twice (2^-24 |z| log2(e) each, |z| <= 6 here),
exponential, sum and reciprocal add a few 2^-24: within 2^-19 in all.  Sums over
a group or row of up to 16,384 columns pass through at most 64 + 10 + 16
additions in a row: 90 2^-24 < 2^-17 of the magnitudes.  Parameters' gradients
add rows / blocks + blocks / 16 + 16 values in a row, below 512 here: 2^-15."""
import pytest
import torch

import _block_ref as bref
import _layer_ref as ref
import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
OUT, SLACK, SUM_SLACK = 2.0 ** -19, 2.0 ** -17, 2.0 ** -15
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def dev(t):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in t.items()}


def leaves_of(t, names):
    return [t[k].requires_grad_(True) for k in names if torch.is_tensor(t[k])]


# ---- gated ---------------------------------------------------------------------

def make_gated(rows, D, size, dtype, shared=True, wdt=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=r(rows, D).to(dtype), z=r(rows, D).to(dtype),
                w=(1 + r(size if shared else D) / 4).to(wdt or dtype), dy=r(rows, D).to(dtype))


# rows, columns, group, type, shared weights, weights' type
GATED = {
    "one_value": (1, 1, 1, F32, True, None),
    "one_head": (1, 128, 128, BF, True, F32),
    "heads": (37, 4096, 128, BF, True, None),
    "heads_own_weights": (9, 4096, 128, HF, False, F32),
    "narrow_groups": (130, 64, 8, F32, True, None),
    "groups_of_16": (5, 1040, 16, BF, True, None),
    "half_wave": (70, 768, 256, BF, False, None),
    "whole_wave": (3, 16384, 512, HF, True, None),
    "row_ends_in_a_step": (11, 2304, 64, F32, True, None),
    "few_columns": (6, 7, 7, BF, True, None),
    "few_in_segments": (6, 18, 9, BF, True, None),
    "segments_that_end_in_vectors": (5, 1001, 13, F32, False, None),
    "many_segments": (3, 16380, 12, HF, True, F32),
    "wide_segments": (3, 15990, 5330, BF, False, None),
    "odd_groups": (17, 5005, 715, HF, False, F32),
    "odd_groups_shared": (33, 4995, 45, BF, True, None),
    "wide_groups": (4, 8192, 4096, BF, False, None),
    "one_group": (66, 1000, 1000, F32, True, None),
    "widest": (2, 16384, 16384, BF, True, F32),
    "many_rows": (5000, 256, 128, BF, True, F32),
    "many_rows_odd": (3000, 150, 75, BF, True, None),
}


@pytest.mark.parametrize("first,act", [(True, "silu"), (False, "silu"), (True, "sigmoid"),
                                       (False, "sigmoid")])
@pytest.mark.parametrize("name", list(GATED))
def test_gated_forward_and_gradients(name, first, act):
    rows, D, size, dtype, shared, wdt = GATED[name]
    t = make_gated(rows, D, size, dtype, shared, wdt)
    g = dev(t)
    leaves = leaves_of(g, ("x", "z", "w"))
    y = gdr.gated_rms_norm(g["x"], g["z"], g["w"], EPS, size, first, act)
    dx, dz, dw = torch.autograd.grad(y, leaves, g["dy"])
    torch.cuda.synchronize()
    r = bref.gated(t["x"], t["z"], t["w"], EPS, size, first, act, t["dy"])
    ref.held("y", y, r["y"], r["y"].abs(), dtype, OUT)
    ref.held("dx", dx, r["dx"], r["dxm"], dtype, SLACK)
    ref.held("dz", dz, r["dz"], r["dzm"], dtype, SLACK)
    ref.held("dw", dw, r["dw"], r["dwm"], dw.dtype, SUM_SLACK)


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("name", ["one_value", "heads", "heads_own_weights", "groups_of_16", "whole_wave",
                                  "few_in_segments", "segments_that_end_in_vectors", "many_segments",
                                  "wide_segments",
                                  "row_ends_in_a_step", "few_columns", "odd_groups",
                                  "odd_groups_shared", "wide_groups", "one_group", "widest"])
def test_gated_eight_bits(name, fmt, group):
    rows, D, size, dtype, shared, wdt = GATED[name]
    for first in (True, False):
        t = make_gated(rows, D, size, dtype, shared, wdt, 3)
        t["x"][0] = 0                            # a row of zeros stays zeros
        g = dev(t)
        q, scale = gdr.gated_rms_norm_quant(g["x"], g["z"], g["w"], EPS, size, first, "silu", fmt, group)
        assert q.shape == t["x"].shape and scale.shape == (rows, -(-D // group) if group else 1)
        r = bref.gated(t["x"], t["z"], t["w"], EPS, size, first, "silu")
        qv = bref.quantised(r["y"], q, scale, fmt, group, SLACK)
        assert qv[0].abs().max() == 0


def test_gated_nans_and_infinities_stay_in_their_group():
    for size in (128, 75):
        t = dev(make_gated(6, 4 * size, size, BF))
        call = lambda **k: gdr.gated_rms_norm(**{**t, **k}, norm_group=size, eps=EPS)  # noqa: E731
        t = dict(x=t["x"], gate=t["z"], weight=t["w"])
        clean = call()
        x = t["x"].clone()
        x[1, size + 3] = float("nan")
        x[2, 3 * size] = float("inf")
        y = call(x=x)
        bad = torch.zeros_like(y, dtype=torch.bool)
        bad[1, size:2 * size] = True
        bad[2, 3 * size] = True
        assert y[bad].isnan().all() and torch.equal(y[~bad & (torch.arange(6, device="cuda") != 2)[:, None]],
                                                    clean[~bad & (torch.arange(6, device="cuda") != 2)[:, None]])
        assert (y[2, 3 * size + 1:] == 0).all() and torch.equal(y[2, :3 * size], clean[2, :3 * size])
        q, scale = gdr.gated_rms_norm_quant(x, t["gate"], t["weight"], EPS, size, format="int8")
        assert scale[1:3].isnan().all() and scale[[0, 3, 4, 5]].isfinite().all()
        assert (q[1:3] == 0).all()


def test_gates_at_their_limits():
    """silu(-inf) = 0, sigmoid(-inf) = 0, sigmoid(inf) = 1, and their slopes are
    0; large finite gates too.  Every type, both orders."""
    for dtype in (BF, HF, F32):
        big = 6e4 if dtype == HF else 1e30
        z = torch.tensor([-float("inf"), -big, -200.0, -80.0, 0.0, 80.0, 200.0, big], dtype=dtype).cuda()
        z = z.repeat(4, 2)
        x = torch.ones_like(z)
        w = torch.ones(16, dtype=dtype, device="cuda")
        for act in ("silu", "sigmoid"):
            y, rstd = gdr.gated_rms_norm_fwd(x, z, w, EPS, activation=act)
            _, dz, _ = gdr.gated_rms_norm_bwd(torch.ones_like(x), x, z, w, rstd, activation=act)
            assert y.isfinite().all() and dz.isfinite().all()
            # e^-80 is 1.8e-35: nothing next to a value of 16 bits
            assert (y[:, [0, 1, 2, 3]].float().abs() <= 2e-33).all()
            assert (dz[:, [0, 1, 2, 3]].float().abs() <= 2e-33).all()
            want = z[:, 4:8] if act == "silu" else torch.tensor([0.5, 1, 1, 1], device="cuda")
            # rstd = 1 / sqrt(1 + 1e-6) and a rounding
            assert ((y[:, 4:8].float() - want.float()).abs() <= want.float().abs() *
                    (1e-6 + torch.finfo(dtype).eps)).all()
    v = torch.full((1, 8), -float("inf"), device="cuda")
    one = torch.ones(1, 8, device="cuda")
    y = gdr.gated_rms_norm(one, v, one[0], EPS, norm_before_gate=False)
    # x act(z) is 80 e^-80: the root is that of eps
    assert (y.abs() <= 80 * 2.0 ** -115 * 1001).all()


def test_gated_slices_and_leading_dimensions():
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(3, 7, 400, generator=g).to(BF).cuda()
    for size, w in ((32, 32), (33, 99), (0, 96)):
        D = size * 3 or 96
        x, z = wide[:, :, 3:3 + D], wide[:, :, 200:200 + D]
        wt = torch.ones(w, dtype=BF, device="cuda")
        dy = torch.randn(3, 7, D, generator=g).to(BF).cuda()
        a = [x.detach().requires_grad_(True), z.detach().requires_grad_(True)]
        b = [v.detach().contiguous().requires_grad_(True) for v in (x, z)]
        ya, yb = gdr.gated_rms_norm(*a, wt, EPS, size), gdr.gated_rms_norm(*b, wt, EPS, size)
        assert ya.shape == (3, 7, D) and torch.equal(ya, yb)
        for p, q in zip(torch.autograd.grad(ya, a, dy), torch.autograd.grad(yb, b, dy)):
            assert torch.equal(p, q)
        assert torch.equal(gdr.gated_rms_norm(x.transpose(0, 1), z.transpose(0, 1), wt, EPS, size),
                           yb.transpose(0, 1))
        assert torch.equal(gdr.gated_rms_norm(x[0, 0], z[0, 0], wt, EPS, size), yb[0, 0])
        qa = gdr.gated_rms_norm_quant(x, z, wt, EPS, size, format="int8")
        qb = gdr.gated_rms_norm_quant(*[v.detach() for v in b], wt, EPS, size, format="int8")
        assert torch.equal(qa[0], qb[0]) and torch.equal(qa[1], qb[1]) and qa[1].shape == (3, 7, 1)


# ---- sandwich -------------------------------------------------------------------

def make_sandwich(rows, D, dtype, rdt, post=True, gate=True, scale=True, wdt=None, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = lambda m: (m + r(D) / 4).to(wdt or dtype)  # noqa: E731
    t = dict(x=r(rows, D).to(dtype), res=(2 * r(rows, D)).to(rdt), pre=w(1), post=w(1), gate=r(rows, D).to(dtype),
             scale=w(0.5), dy=r(rows, D).to(dtype), dh=r(rows, D).to(rdt))
    for k, on in (("post", post), ("gate", gate)):
        t[k] = t[k] if on else None
    if scale is not True:
        t["scale"] = scale
    return t


SANDWICH = {
    "one_value": (1, 1, F32, F32, True, True, True, None),
    "few_columns": (5, 6, BF, F32, True, True, True, F32),
    "one_row": (1, 4096, BF, BF, True, True, True, None),
    "narrow_odd": (7, 45, HF, F32, True, True, None, F32),
    "wave": (130, 512, BF, F32, True, False, True, None),
    "two_steps": (33, 1000, F32, F32, True, True, 0.22, None),
    "no_post": (9, 4096, BF, BF, False, True, True, F32),
    "only_the_addition": (9, 2049, BF, F32, False, False, None, None),
    "odd": (5, 5003, HF, HF, True, True, True, None),
    "half_rows": (3, 8192, BF, BF, True, True, True, None),
    "wide": (3, 16000, BF, F32, True, True, True, None),
    "widest": (2, 16384, F32, F32, True, True, True, None),
    "many_rows": (5000, 72, BF, BF, True, True, -1.5, None),
    "many_rows_wide": (1100, 2056, BF, BF, True, True, True, None),
}


def sandwich_args(t):
    return (t["x"], t["res"], t["post"], t["pre"], t["gate"], t["scale"])


@pytest.mark.parametrize("act", ["sigmoid", "silu", None])
@pytest.mark.parametrize("name", list(SANDWICH))
def test_sandwich_forward_and_gradients(name, act):
    rows, D, dtype, rdt, *how, wdt = SANDWICH[name]
    t = make_sandwich(rows, D, dtype, rdt, *how, wdt)
    g = dev(t)
    names = [k for k in ("x", "res", "post", "pre", "gate", "scale") if torch.is_tensor(g[k])]
    leaves = leaves_of(g, names)
    y, h = gdr.sandwich_rms_norm(*sandwich_args(g), act, EPS)
    grads = dict(zip(names, torch.autograd.grad([y, h], leaves, [g["dy"], g["dh"]])))
    torch.cuda.synchronize()
    assert h.dtype == rdt and y.dtype == dtype
    r = bref.sandwich(t["x"], t["res"], t["post"], t["pre"], EPS, t["gate"], t["scale"], act, h, t["dy"],
                      t["dh"])
    ref.held("h", h, r["h"], r["hm"], rdt, OUT)
    ref.held("y", y, r["y"], r["y"].abs(), dtype, OUT)
    for k, dt, slack in (("x", dtype, SLACK), ("res", rdt, SLACK), ("gate", dtype, SLACK),
                         ("post", wdt or dtype, SUM_SLACK), ("pre", wdt or dtype, SUM_SLACK),
                         ("scale", wdt or dtype, SUM_SLACK)):
        if k in grads:
            assert grads[k].dtype == dt
            ref.held("d" + k, grads[k], r["d" + k], r["d" + k + "m"], dt, slack)


def test_sandwich_gradient_of_one_output_only():
    t = dev(make_sandwich(20, 300, BF, F32))
    names = ("x", "res", "post", "pre", "gate", "scale")
    leaves = leaves_of(t, names)
    y, h = gdr.sandwich_rms_norm(*sandwich_args(t))
    only_y = torch.autograd.grad(y, leaves, t["dy"], retain_graph=True)
    zero = torch.autograd.grad([y, h], leaves, [t["dy"], torch.zeros_like(h)], retain_graph=True)
    assert all(torch.equal(a, b) for a, b in zip(only_y, zero))
    only_h = torch.autograd.grad(h, leaves, t["dh"], retain_graph=True, allow_unused=True)
    zero = torch.autograd.grad([y, h], leaves, [torch.zeros_like(y), t["dh"]])
    assert all(torch.equal(a, b) for a, b in zip(only_h, zero))
    assert not only_h[3].any()


@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("name", [k for k in SANDWICH if "many" not in k])
def test_sandwich_eight_bits(name, fmt, group):
    rows, D, dtype, rdt, *how, wdt = SANDWICH[name]
    t = make_sandwich(rows, D, dtype, rdt, *how, wdt, seed=2)
    t["x"][0], t["res"][0] = 0, 0
    g = dev(t)
    q, scale, h = gdr.sandwich_rms_norm_quant(*sandwich_args(g), "silu", EPS, fmt, group)
    r = bref.sandwich(t["x"], t["res"], t["post"], t["pre"], EPS, t["gate"], t["scale"], "silu", h)
    ref.held("h", h, r["h"], r["hm"], rdt, OUT)
    qv = bref.quantised(r["y"], q, scale, fmt, group, SLACK)
    assert qv[0].abs().max() == 0


def test_sandwich_nans_stay_in_their_row():
    t = dev(make_sandwich(5, 300, BF, BF))
    y0, h0, _, _ = gdr.sandwich_rms_norm_fwd(*sandwich_args(t))
    t["x"][1, 7] = float("nan")
    t["res"][3, 9] = float("nan")
    y, h, _, _ = gdr.sandwich_rms_norm_fwd(*sandwich_args(t))
    assert torch.equal(y[[0, 2, 4]], y0[[0, 2, 4]]) and torch.equal(h[[0, 2, 4]], h0[[0, 2, 4]])
    assert y[1].isnan().all() and h[1].isnan().all()
    assert y[3].isnan().all() and h[3].isnan().sum() == 1


def test_sandwich_slices_and_leading_dimensions():
    g = torch.Generator().manual_seed(1)
    wide = torch.randn(3, 7, 300, generator=g).to(BF).cuda()
    t = dev(make_sandwich(21, 99, BF, F32))
    x, gate = wide[:, :, 3:102], wide[:, :, 150:249]
    res = t["res"].view(3, 7, 99)
    a = [v.detach().requires_grad_(True) for v in (x, gate)]
    b = [v.detach().contiguous().requires_grad_(True) for v in (x, gate)]
    ra = gdr.sandwich_rms_norm(a[0], res, t["post"], t["pre"], a[1], t["scale"])
    rb = gdr.sandwich_rms_norm(b[0], res, t["post"], t["pre"], b[1], t["scale"])
    go = [torch.ones_like(v) for v in ra]
    for p, q in zip(ra + torch.autograd.grad(ra, a, go), rb + torch.autograd.grad(rb, b, go)):
        assert torch.equal(p, q)
    rt = gdr.sandwich_rms_norm(x.transpose(0, 1), res.transpose(0, 1), t["post"], t["pre"],
                               gate.transpose(0, 1), t["scale"])
    assert torch.equal(rt[0], rb[0].transpose(0, 1)) and torch.equal(rt[1], rb[1].transpose(0, 1))
    one = gdr.sandwich_rms_norm(x[0, 0], res[0, 0], t["post"], t["pre"], gate[0, 0], t["scale"])
    assert torch.equal(one[0], rb[0][0, 0])


# ---- both -------------------------------------------------------------------------

def test_gradients_against_differences():
    """fp32, random directions; with step 2^-7 the central difference is off
    by about h^2 and 2^-23 / h of the outputs, under 2e-3 of the root of the
    summed squares."""
    gen = torch.Generator().manual_seed(2)
    h = 2.0 ** -7

    def follow(t, names, grads, value):
        for k in names:
            v = torch.randn(t[k].shape, generator=gen).cuda()
            diff = (value({**t, k: t[k] + h * v}) - value({**t, k: t[k] - h * v})) / (2 * h)
            p = grads[k].double() * v
            assert abs(diff - p.sum()) <= 2e-3 * p.square().sum().sqrt(), (k, float(diff), float(p.sum()))

    for size, first in ((40, True), (64, False)):
        t = dev(make_gated(6, 5 * size, size, F32, seed=4))
        y, rstd = gdr.gated_rms_norm_fwd(t["x"], t["z"], t["w"], EPS, size, first)
        got = dict(zip("xzw", gdr.gated_rms_norm_bwd(t["dy"], t["x"], t["z"], t["w"], rstd, size, first)))
        follow(t, "xzw", got, lambda q: (gdr.gated_rms_norm_fwd(
            q["x"], q["z"], q["w"], EPS, size, first)[0].double() * t["dy"]).sum())
    t = dev(make_sandwich(6, 200, F32, F32, seed=4))
    names = ("x", "res", "post", "pre", "gate", "scale")
    y, hh, rx, rh = gdr.sandwich_rms_norm_fwd(*sandwich_args(t))
    got = dict(zip(names, gdr.sandwich_rms_norm_bwd(t["dy"], t["dh"], t["x"], hh, t["post"], t["pre"], rx,
                                                    rh, t["gate"], t["scale"])))

    def value(q):
        y, hh, _, _ = gdr.sandwich_rms_norm_fwd(*sandwich_args(q))
        return (y.double() * t["dy"]).sum() + (hh.double() * t["dh"]).sum()

    follow(t, names, got, value)


def test_norms_past_two_to_the_31_elements():
    """The last rows of tensors of more than 2^31 elements equal their own run."""
    rows, D = (1 << 17) + 300, 16384
    x = torch.empty(rows, D, device="cuda", dtype=BF)
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(0))
    w = torch.ones(D, device="cuda")
    end = slice(rows - 5, rows)
    for size in (128, 8192):
        args = (x, x, w, EPS, size)
        tail = (x[end], x[end], w, EPS, size)
        y, rstd = gdr.gated_rms_norm_fwd(*args)
        yt, rt = gdr.gated_rms_norm_fwd(*tail)
        assert torch.equal(y[end], yt) and torch.equal(rstd[end], rt)
        dx, dz, _ = gdr.gated_rms_norm_bwd(y, x, x, w, rstd, size)
        dt = gdr.gated_rms_norm_bwd(yt, x[end], x[end], w, rt, size)
        assert torch.equal(dx[end], dt[0]) and torch.equal(dz[end], dt[1])
        del y, dx, dz
        q, s = gdr.gated_rms_norm_quant(*args, format="int8", group_size=128)
        qt, st = gdr.gated_rms_norm_quant(*tail, format="int8", group_size=128)
        assert torch.equal(q[end], qt) and torch.equal(s[end], st)
        del q
    y, h, rx, rh = gdr.sandwich_rms_norm_fwd(x, x, w, w, x, w)
    t = gdr.sandwich_rms_norm_fwd(x[end], x[end], w, w, x[end], w)
    assert all(torch.equal(a[end], b) for a, b in zip((y, h, rx, rh), t))
    g = gdr.sandwich_rms_norm_bwd(y, h, x, h, w, w, rx, rh, x, w)
    gt = gdr.sandwich_rms_norm_bwd(t[0], t[1], x[end], t[1], w, w, t[2], t[3], x[end], w)
    for i in (0, 1, 4):
        assert torch.equal(g[i][end], gt[i])
    del g, y, h
    q, s = gdr.quantize_rows(x)
    qt, st = gdr.quantize_rows(x[end])
    assert torch.equal(q[end], qt) and torch.equal(s[end], st)
