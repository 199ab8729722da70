"""Gates far from zero in the gated norm and the sandwich norm, on the GPU
against plain 64-bit forms (needs an MI355X).

Tolerances, relative to a value's own terms: the smaller of a gate's sigmoid and
its complement passes through an exponential and a reciprocal (an instruction's
2^-23 each), a correction, a sum and a product (2^-24 each): within 2^-21; the
larger is one less it.  A slope is a product of two such factors (silu's second
factor 1 + z (1 - s) is at least 1/8 of its terms' sum for |z| >= 8): within 2^-20.
The products with the unit row and the weights add six roundings: 2^-19 in all
where no sum over the row takes part, and 2^-17 of the magnitudes where one does
(at most 90 additions in a row)."""
import pytest
import torch

import _block_ref as bref
import _layer_ref as ref
import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
OUT, SLACK = 2.0 ** -19, 2.0 ** -17
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
EPS = 1e-6


def gates(rows, D, low, high, dtype, seed=0):
    """Magnitudes from low to high, of both signs in turn."""
    g = torch.Generator().manual_seed(seed)
    z = low + (high - low) * torch.rand(rows, D, generator=g)
    return (z * (1 - 2 * (torch.arange(rows * D).view(rows, D) % 2))).to(dtype)


def values(rows, D, dtype, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=r(rows, D).to(dtype), dy=r(rows, D).to(dtype), dh=r(rows, D).to(dtype),
                res=r(rows, D).to(dtype), w=(1 + r(D) / 4).to(dtype), v=(1 + r(D) / 4).to(dtype))


def act(z, name):
    """As the references' own, with the complement s(-z), of which 1 - s(z) keeps
    nothing beyond z = 37 in 64 bits either; a slope's magnitude is its own."""
    s, rest = torch.sigmoid(z), torch.sigmoid(-z)
    if name == "silu":
        return z * s, s * (1 + z * rest), (s * (1 + z * rest)).abs()
    return s, s * rest, s * rest


@pytest.fixture(autouse=True)
def exact_slopes(monkeypatch):
    monkeypatch.setattr(bref, "act", act)


# ---- slopes --------------------------------------------------------------------

@pytest.mark.parametrize("name", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("D,size", [(320, 320), (384, 128), (300, 75), (1000, 1000), (8200, 8200)])
def test_slopes_of_open_and_closed_gates(D, size, dtype, name):
    """An open sigmoid's slope is its complement, which one less the sigmoid
    would lose."""
    rows = 5
    t, z = values(rows, D, dtype), gates(rows, D, 8, 40, dtype)
    w = t["w"][:size].contiguous()
    for first in (True, False):
        y, rstd = gdr.gated_rms_norm_fwd(t["x"].cuda(), z.cuda(), w.cuda(), EPS, size, first, name)
        _, dz, _ = gdr.gated_rms_norm_bwd(t["dy"].cuda(), t["x"].cuda(), z.cuda(), w.cuda(), rstd, size,
                                          first, name)
        r = bref.gated(t["x"], z, w, EPS, size, first, name, t["dy"])
        ref.held("y", y, r["y"], r["y"].abs(), dtype, SLACK)
        ref.held("dz", dz, r["dz"], r["dzm"], dtype, OUT if first else SLACK)


@pytest.mark.parametrize("name", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF, HF])
@pytest.mark.parametrize("D", [320, 1001, 8200])
def test_sandwich_slopes_of_open_and_closed_gates(D, dtype, name):
    t, z = values(5, D, dtype), gates(5, D, 8, 40, dtype)
    g = {k: v.cuda() for k, v in t.items()}
    y, h, rx, rh = gdr.sandwich_rms_norm_fwd(g["x"], g["res"], g["w"], g["v"], z.cuda(), 0.5, name, EPS)
    got = gdr.sandwich_rms_norm_bwd(g["dy"], g["dh"], g["x"], h, g["w"], g["v"], rx, rh, z.cuda(), 0.5, name)
    r = bref.sandwich(t["x"], t["res"], t["w"], t["v"], EPS, z, 0.5, name, h, t["dy"], t["dh"])
    ref.held("dgate", got[4], r["dgate"], r["dgatem"], dtype, SLACK)


# ---- the range -------------------------------------------------------------------

@pytest.mark.parametrize("name", ["silu", "sigmoid"])
@pytest.mark.parametrize("dtype", [F32, BF])
def test_closed_gates_to_the_end_of_fp32(dtype, name):
    """Down to -104, where the sigmoid leaves fp32, and to 0 at minus infinity.
    Beyond OUT a sigmoid is off by fp32's smallest step 2^-149, silu and its slope
    by |z| of it, and every product by half a step."""
    t = values(4, 320, dtype)
    z = torch.linspace(-79, -110, 320).repeat(4, 1).to(dtype)
    z[2, ::7], z[3, ::5] = -float("inf"), -3e38
    closed = z < -200
    zr = z.clone()
    zr[closed] = -200.0                       # 0 in fp32, and no 0 times an infinity in the reference
    r = bref.gated(t["x"], zr, t["w"], EPS, 0, True, name, t["dy"])
    u = ref.d(t["x"]) * r["rstd"]
    step = 2.0 ** -149 * (2 + 2 * ref.d(zr).abs())
    y, rstd = gdr.gated_rms_norm_fwd(t["x"].cuda(), z.cuda(), t["w"].cuda(), EPS, 0, True, name)
    _, dz, _ = gdr.gated_rms_norm_bwd(t["dy"].cuda(), t["x"].cuda(), z.cuda(), t["w"].cuda(), rstd, 0, True,
                                      name)
    uw = (u * ref.d(t["w"])).abs()
    for got, want, size in ((y, r["y"], 1 + uw), (dz, r["dz"], 1 + uw * ref.d(t["dy"]).abs())):
        bar = (OUT + ref.half_step(dtype) * 1.01) * want.abs() + step * size + \
            torch.finfo(dtype).tiny * torch.finfo(dtype).eps
        assert ((ref.d(got) - want).abs() <= bar).all()
        assert (got.cpu()[closed] == 0).all()
    # the sandwich norm's gate: h = 0 + act(g) x
    nil = torch.zeros(4, 320, device="cuda")
    h = gdr.sandwich_rms_norm_fwd(t["x"].cuda(), nil, None, t["v"].cuda(), z.cuda(), None, name, EPS)[1]
    want = act(ref.d(zr), name)[0] * ref.d(t["x"])
    bar = OUT * want.abs() + step * (1 + ref.d(t["x"]).abs())
    assert ((ref.d(h) - want).abs() <= bar).all() and (h.cpu()[closed] == 0).all()


@pytest.mark.parametrize("name", ["silu", "sigmoid"])
@pytest.mark.parametrize("low,high", [(81, 87), (86.8, 87.2), (60, 70)])
@pytest.mark.parametrize("D,size", [(320, 320), (384, 128), (300, 75), (8200, 8200)])
def test_groups_of_closed_gates_without_eps(D, size, low, high, name):
    """eps = 0 and the gate first: groups of closed gates are scaled up to unit
    rows, whose gradients pass through inverse roots of up to 1e38.  A product
    x act(z) below 2^-126 is rounded to a multiple of 2^-149, so a unit row is off
    by 2^-150 of the inverse root beside its 2^-17: the output by its weight of it,
    the weight's gradient by dy of it.  (In dx and dz this is beside the group's mean
    and its own dy: 2^-150 1e38 is less than 2^-23.)"""
    t = values(5, D, F32)
    z = -gates(5, D, low, high, F32).abs()
    w = t["w"][:size].contiguous()
    y, rstd = gdr.gated_rms_norm_fwd(t["x"].cuda(), z.cuda(), w.cuda(), 0.0, size, False, name)
    got = gdr.gated_rms_norm_bwd(t["dy"].cuda(), t["x"].cuda(), z.cuda(), w.cuda(), rstd, size, False, name)
    r = bref.gated(t["x"], z, w, 0.0, size, False, name, t["dy"])
    low = 2.0 ** -150 / SLACK * r["rstd"].repeat_interleave(size, -1)
    ref.held("y", y, r["y"], r["y"].abs() + low * ref.d(w).abs().repeat(D // size), F32, SLACK)
    r["dwm"] = r["dwm"] + (low * ref.d(t["dy"]).abs()).view(-1, size).sum(0)
    for g, k in zip(got, ("dx", "dz", "dw")):
        ref.held(k, g, r[k], r[k + "m"], F32, SLACK)


@pytest.mark.parametrize("dtype", [F32, BF, HF])
def test_slopes_at_plus_infinity(dtype):
    """sigmoid: value 1, slope 0; silu: slope 1 (its value is infinite, and what
    is made of it)."""
    t = values(4, 96, dtype)
    z = gates(4, 96, 1, 3, dtype)
    open_ = torch.zeros(4, 96, dtype=torch.bool)
    open_[:, ::9] = True
    z[open_] = float("inf")
    x, w, dy = t["x"].cuda(), t["w"].cuda(), t["dy"].cuda()
    for size in (96, 32, 12):
        v = w[:size].contiguous()
        u = ref.d(x).view(-1, size)
        u = (u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * ref.d(v)).view(4, 96)
        for name in ("sigmoid", "silu"):
            y, rstd = gdr.gated_rms_norm_fwd(x, z.cuda(), v, EPS, size, True, name)
            _, dz, _ = gdr.gated_rms_norm_bwd(dy, x, z.cuda(), v, rstd, size, True, name)
            want = u * ref.d(dy) * (1.0 if name == "silu" else 0.0)
            ref.held("dz", dz.cpu()[open_], want[open_], want[open_].abs(), dtype, OUT)
            if name == "sigmoid":
                ref.held("y", y.cpu()[open_], u[open_], u[open_].abs(), dtype, OUT)
    one = x.new_ones(96)
    y, h, rx, rh = gdr.sandwich_rms_norm_fwd(x, x, w, one, z.cuda(), None, "sigmoid", EPS)
    dgate = gdr.sandwich_rms_norm_bwd(dy, None, x, h, w, one, rx, rh, z.cuda(), None, "sigmoid")[4]
    assert y.isfinite().all() and dgate.isfinite().all() and (dgate.cpu()[open_] == 0).all()


def test_gates_that_are_no_numbers():
    """A NaN in the gate reaches its own output after the norm, its group's
    before it, and the gradients of its group (of its row, in the sandwich norm)."""
    t = values(4, 96, F32)
    z = gates(4, 96, 1, 3, F32)
    z[1, 40] = float("nan")
    x, w, dy, zc = t["x"].cuda(), t["w"].cuda(), t["dy"].cuda(), z.cuda()
    own, row = (torch.zeros(4, 96, dtype=torch.bool) for _ in range(2))
    own[1, 40], row[1] = True, True
    for size in (96, 32, 24):
        group = torch.zeros(4, 96, dtype=torch.bool)
        group[1, 40 // size * size:(40 // size + 1) * size] = True
        v = w[:size].contiguous()
        for name in ("silu", "sigmoid"):
            for first in (True, False):
                y, rstd = gdr.gated_rms_norm_fwd(x, zc, v, EPS, size, first, name)
                assert torch.equal(y.isnan().cpu(), own if first else group)
                dx, dz, _ = gdr.gated_rms_norm_bwd(dy, x, zc, v, rstd, size, first, name)
                assert torch.equal(dx.isnan().cpu(), group)
                assert torch.equal(dz.isnan().cpu(), own if first else group)
    for name in ("silu", "sigmoid", None):
        y, h, rx, rh = gdr.sandwich_rms_norm_fwd(x, x, w, w, zc, None, name, EPS)
        assert torch.equal(h.isnan().cpu(), own) and torch.equal(y.isnan().cpu(), row)
        got = gdr.sandwich_rms_norm_bwd(dy, None, x, h, w, w, rx, rh, zc, None, name)
        assert all(torch.equal(g.isnan().cpu(), row) for g in (got[0], got[1], got[4]))
