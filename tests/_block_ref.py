"""Plain 64-bit references of the operators at a layer's ends, on the CPU.
Names with an m are the magnitudes that a value's terms add up to, which the
errors of its 32-bit arithmetic scale with."""
import torch

from _layer_ref import d


def act(z, name):
    """(value, derivative, magnitude of the derivative's terms)."""
    if name is None:
        return z, torch.ones_like(z), torch.ones_like(z)
    s = torch.sigmoid(z)
    if name == "silu":
        return z * s, s * (1 + z * (1 - s)), s * (1 + z.abs())
    return s, s * (1 - s), s


def norm_grad(du, dum, u, r):
    """Gradient of the unit rows u = r v from du, and its magnitude."""
    g = r * (du - u * (du * u).mean(-1, keepdim=True))
    return g, r * (dum + u.abs() * (dum * u.abs()).mean(-1, keepdim=True))


def gated(x, z, w, eps, size=0, first=True, name="silu", dy=None):
    x, z, w, dy = d(x), d(z), d(w), d(dy)
    D = x.shape[-1]
    size = size or D
    cut = lambda v: v.reshape(-1, D // size, size)  # noqa: E731
    shape = x.shape
    shared = w.shape[0] == size
    wg = w.reshape(-1, size)
    a, slope, slopem = (cut(v) for v in act(z, name))
    xg = cut(x)
    v = xg if first else xg * a
    r = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    u = v * r
    y = u * wg * (a if first else 1.0)
    out = {"y": y.reshape(shape), "rstd": r[..., 0].reshape(shape[:-1] + (D // size,))}
    if dy is not None:
        g = cut(dy)
        k = a if first else torch.ones_like(a)
        du = g * wg * k
        dv, dvm = norm_grad(du, du.abs(), u, r)
        if first:
            dx, dxm, dz, dzm = dv, dvm, g * wg * u * slope, (g * wg * u).abs() * slopem
        else:
            dx, dxm = dv * a, dvm * a.abs()
            dz, dzm = dv * xg * slope, dvm * xg.abs() * slopem
        dw = g * u * k
        over = (0, 1) if shared else 0
        out.update(dx=dx.reshape(shape), dxm=dxm.reshape(shape), dz=dz.reshape(shape),
                   dzm=dzm.reshape(shape), dw=dw.sum(over).flatten(), dwm=dw.abs().sum(over).flatten())
    return out


def sandwich(x, res, post, pre, eps, gate=None, scale=None, name="sigmoid", h=None, dy=None, dh=None):
    """With h, the stored stream, y and the gradients are those of this h."""
    rdt = res.dtype
    number = 1.0 if scale is None or torch.is_tensor(scale) else float(scale)
    x, res, post, pre, gate, dy, dh = (d(t) for t in (x, res, post, pre, gate, dy, dh))
    sc = (d(scale) if torch.is_tensor(scale) else torch.ones_like(pre)) * number
    w1 = torch.ones_like(pre) if post is None else post
    a, slope, slopem = (torch.ones_like(x),) * 3 if gate is None else act(gate, name)
    rx = 1 / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    ux = x if post is None else x * rx
    add = sc * a * w1 * ux
    out = {"h": res + add, "hm": res.abs() + add.abs()}
    s = out["h"].to(rdt).double() if h is None else d(h)
    rh = 1 / torch.sqrt((s * s).mean(-1, keepdim=True) + eps)
    u = s * rh
    out["y"] = u * pre
    if dy is None:
        return out
    dH, dHm = norm_grad(dy * pre, (dy * pre).abs(), u, rh)
    if dh is not None:
        dH, dHm = dH + dh, dHm + dh.abs()
    c = sc * a * w1
    du, dum = dH * c, dHm * c.abs()
    dx, dxm = (du, dum) if post is None else norm_grad(du, dum, ux, rx)
    rows = lambda v: v.flatten(0, -2).sum(0)  # noqa: E731
    P, Pm = dH * a * ux, dHm * (a * ux).abs()
    out.update(dx=dx, dxm=dxm, dres=dH, dresm=dHm, dpre=rows(dy * u), dprem=rows((dy * u).abs()),
               dpost=rows(P) * sc, dpostm=rows(Pm) * sc.abs(), dscale=rows(P) * w1 * number,
               dscalem=rows(Pm) * w1.abs() * abs(number), dgate=dH * sc * w1 * ux * slope,
               dgatem=dHm * (sc * w1 * ux).abs() * slopem)
    return out


def quantised(y, q, scale, fmt, group, slack):
    """Holds (q, scale) against the values y: scales within slack, a value
    within half a step of y / scale (int8 1/2; e4m3 2^-4 relative, 2^-10 below
    its normal range), which is off by slack itself."""
    D = y.shape[-1]
    y = d(y).reshape(-1, D)
    top = 448.0 if fmt == "fp8" else 127.0
    width = group or D
    yg = torch.nn.functional.pad(y, (0, (-D) % width)).unflatten(1, (-1, width))
    want = (yg.abs().amax(-1) / top).clamp_min(2.0 ** -126)
    got = d(scale).reshape(want.shape)
    assert ((got - want).abs() <= slack * want).all()
    v = (yg / got[..., None]).flatten(1)[:, :D]
    qv = q.cpu().reshape(-1, D).float().double()
    bar = (v.abs() * 2.0 ** -4).clamp_min(2.0 ** -10) if fmt == "fp8" else torch.full_like(v, 0.5)
    off = (qv - v).abs()
    assert (off <= bar * (1 + slack) + 2 * slack * v.abs()).all(), float((off - bar).max())
    return qv


def product(x, xs, w, ws, bias=None):
    """y and the magnitude of its two terms."""
    acc = d(x) @ d(w).t()
    y = acc * d(xs).reshape(acc.shape[:-1] + (1,)) * d(ws).flatten()
    if bias is None:
        return y, y.abs()
    return y + d(bias), y.abs() + d(bias).abs()
