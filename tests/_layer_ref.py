"""Plain 64-bit references of the layer operators, on the CPU, and the error
bars they are compared with."""
import torch


def d(t):
    return None if t is None else t.detach().cpu().double()


def half_step(dtype):
    """A rounding is off by at most half a step, relative to the value."""
    return torch.finfo(dtype).eps / 2


def spans(x, cu):
    """(row, first, end, sequence)."""
    if cu is None:
        return [(b, 0, x.shape[1], b) for b in range(x.shape[0])]
    cu = [int(v) for v in cu]
    return [(0, a, b, n) for n, (a, b) in enumerate(zip(cu, cu[1:]))]


def conv(x, w, bias=None, silu=True, state=None, cu=None, dy=None, dlast=None):
    """{name: (value, sum of its terms' magnitudes)}: the second is what the
    rounding of the sums scales with."""
    x, w, bias, state, dy, dlast = (d(t) for t in (x, w, bias, state, dy, dlast))
    W, D = w.shape[1], x.shape[2]
    n = len(spans(x, cu))
    y, ym = torch.zeros_like(x), torch.zeros_like(x)
    last = x.new_zeros(n, W - 1, D)
    dx, dxm = torch.zeros_like(x), torch.zeros_like(x)
    ds, dsm = torch.zeros_like(last), torch.zeros_like(last)
    dw, dwm = torch.zeros_like(w), torch.zeros_like(w)
    db, dbm = x.new_zeros(D), x.new_zeros(D)
    for row, a, b, i in spans(x, cu):
        L = b - a
        ext = torch.cat([x.new_zeros(W - 1, D) if state is None else state[i], x[row, a:b]])
        z, zm = x.new_zeros(L, D), x.new_zeros(L, D)
        for j in range(W):
            z += ext[j:j + L] * w[:, j]
            zm += (ext[j:j + L] * w[:, j]).abs()
        if bias is not None:
            z, zm = z + bias, zm + bias.abs()
        sg = torch.sigmoid(z)
        y[row, a:b] = z * sg if silu else z
        ym[row, a:b] = zm * 1.1 + z.abs() * 2
        last[i] = ext[L:]
        if dy is not None:
            act = sg * (1 + z * (1 - sg)) if silu else torch.ones_like(z)
            g = dy[row, a:b] * act
            gm = dy[row, a:b].abs() * (1.1 + zm)      # |act''| <= 1/2, z is off by its own rounding
            e, em = torch.zeros_like(ext), torch.zeros_like(ext)
            for j in range(W):
                e[j:j + L] += g * w[:, j]
                em[j:j + L] += gm * w[:, j].abs()
                dw[:, j] += (g * ext[j:j + L]).sum(0)
                dwm[:, j] += (gm * ext[j:j + L].abs()).sum(0)
            db += g.sum(0)
            dbm += gm.sum(0)
            if dlast is not None:
                e[L:] += dlast[i]
                em[L:] += dlast[i].abs()
            dx[row, a:b], dxm[row, a:b] = e[W - 1:], em[W - 1:]
            ds[i], dsm[i] = e[:W - 1], em[:W - 1]
    return {"y": (y, ym), "last": (last, 0 * last), "dx": (dx, dxm), "dw": (dw, dwm), "db": (db, dbm),
            "ds": (ds, dsm)}


def norm(x, w, eps, res=None, dy=None, dh=None):
    """y, h, dx (before the stream's rounding), dw, and the magnitudes their
    fp32 arithmetic scales with."""
    if res is None:
        h = d(x)
    else:  # the stored stream: one fp32 addition, rounded to the residual's type
        h = d((x.detach().cpu().float() + res.detach().cpu().float()).to(res.dtype))
    w, dy, dh = d(w), d(dy), d(dh)
    inv = 1 / torch.sqrt((h * h).mean(-1, keepdim=True) + eps)
    u = h * inv
    out = {"h": h, "y": u * w}
    if dy is not None:
        du = dy * w
        mean = (du * u).mean(-1, keepdim=True)
        g = inv * (du - u * mean)
        gm = inv * (du.abs() + u.abs() * (du * u).abs().mean(-1, keepdim=True))
        if dh is not None:
            g, gm = g + dh, gm + dh.abs()
        out.update(dx=g, dxm=gm, dw=(dy * u).flatten(0, -2).sum(0),
                   dwm=(dy * u).abs().flatten(0, -2).sum(0))
    return out


def held(name, got, ref, mag, dtype, slack):
    """|got - ref| <= half a step of the output's type relative to ref, plus
    slack times the magnitude of what was summed (and the type's smallest
    step, for values below its normal range)."""
    got, ref = d(got), ref.double()
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bar = half_step(dtype) * ref.abs() * (1 + 2 * slack) + slack * mag + torch.finfo(dtype).tiny * \
        torch.finfo(dtype).eps
    off = (got - ref).abs()
    bad = ~(off <= bar)
    assert not bad.any(), (name, int(bad.sum()), float((off / bar).nan_to_num(9e9).max()))
