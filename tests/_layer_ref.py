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


def scan(x, raw, A_log, B, C, D=None, bias=None, softplus=True, state=None, cu=None, dy=None,
         dlast=None):
    """The selective scan token by token.  y, last and, with dy, the gradients;
    a name with m is the magnitude that the value's terms add up to."""
    x, raw, A_log, B, C, D, bias, state, dy, dlast = (
        d(t) for t in (x, raw, A_log, B, C, D, bias, state, dy, dlast))
    H, V = x.shape[2:]
    G, K = B.shape[2:]
    R = H // G
    z = raw if bias is None else raw + bias
    step = torch.nn.functional.softplus(z, threshold=1e9) if softplus else z
    dz = torch.sigmoid(z) if softplus else torch.ones_like(z)
    rate = -torch.exp(A_log)
    n = len(spans(x, cu))
    y, ym = torch.zeros_like(x), torch.zeros_like(x)
    last = x.new_zeros(n, H, K, V)
    lastm = torch.zeros_like(last)
    out = {}
    if dy is not None:
        dx, dxm = torch.zeros_like(x), torch.zeros_like(x)
        dstep, dstepm = torch.zeros_like(step), torch.zeros_like(step)
        dB, dBm, dC, dCm = (torch.zeros_like(B) for _ in range(4))
        ds, dsm = torch.zeros_like(last), torch.zeros_like(last)
        dA, sfxm = torch.zeros_like(rate), torch.zeros_like(step)
        group = lambda v: v.reshape(G, R, K).sum(1)  # noqa: E731
    for row, a, b, i in spans(x, cu):
        S = x.new_zeros(H, K, V) if state is None else state[i]
        Sm = S.abs()
        S_all, Sm_all = [S], [Sm]
        for t in range(a, b):
            e = torch.exp(rate * step[row, t])[:, None, None]
            add = (step[row, t, :, None] * B[row, t].repeat_interleave(R, 0))[:, :, None] * x[row, t][:, None]
            S, Sm = e * S + add, e * Sm + add.abs()
            c = C[row, t].repeat_interleave(R, 0)
            y[row, t] = (c[:, :, None] * S).sum(1)
            ym[row, t] = (c.abs()[:, :, None] * Sm).sum(1)
            if D is not None:
                y[row, t] += D[:, None] * x[row, t]
                ym[row, t] += (D[:, None] * x[row, t]).abs()
            S_all.append(S)
            Sm_all.append(Sm)
        last[i], lastm[i] = S, Sm
        if dy is None:
            continue
        P = x.new_zeros(H, K, V) if dlast is None else dlast[i]
        Pm = P.abs()
        later = torch.zeros_like(rate)     # what the suffix sum behind dg has added up
        for t in reversed(range(a, b)):
            st, xt, g = step[row, t], x[row, t], dy[row, t]
            bt, c = B[row, t].repeat_interleave(R, 0), C[row, t].repeat_interleave(R, 0)
            S, Sm, S0, Sm0 = S_all[t - a + 1], Sm_all[t - a + 1], S_all[t - a], Sm_all[t - a]
            dC[row, t] = group((S * g[:, None]).sum(-1))
            dCm[row, t] = group((Sm * g.abs()[:, None]).sum(-1))
            cg = c[:, :, None] * g[:, None]
            P, Pm = P + cg, Pm + cg.abs()
            px, pxm = (P * xt[:, None]).sum(-1), (Pm * xt.abs()[:, None]).sum(-1)
            dB[row, t], dBm[row, t] = group(st[:, None] * px), group(st.abs()[:, None] * pxm)
            u, um = (P * bt[:, :, None]).sum(1), (Pm * bt.abs()[:, :, None]).sum(1)
            dx[row, t], dxm[row, t] = st[:, None] * u, st.abs()[:, None] * um
            if D is not None:
                dx[row, t] += D[:, None] * g
                dxm[row, t] += (D[:, None] * g).abs()
            e = torch.exp(rate * st)
            da, dam = (P * S0).sum((1, 2)) * e, (Pm * Sm0).sum((1, 2)) * e
            later = later + (Sm * cg.abs()).sum((1, 2)) + st.abs() * (xt.abs() * um).sum(-1)
            sfxm[row, t] = dam + later
            dstep[row, t] = (xt * u).sum(-1) + rate * da
            dstepm[row, t] = (xt.abs() * um).sum(-1) + rate.abs() * sfxm[row, t]
            dA += rate * st * da
            P, Pm = e[:, None, None] * P, e[:, None, None] * Pm
        ds[i], dsm[i] = P, Pm
    out.update(y=y, ym=ym, last=last, lastm=lastm)
    if dy is not None:
        draw, drawm = dstep * dz, dstepm * dz
        out.update(dx=dx, dxm=dxm, ddt=draw, ddtm=drawm, dB=dB, dBm=dBm, dC=dC, dCm=dCm, ds=ds,
                   dsm=dsm, dA=dA, dAm=(rate.abs() * step.abs() * sfxm).sum((0, 1)), dbias=draw.sum((0, 1)), dbiasm=drawm.sum((0, 1)),
                   dD=(dy * x).sum((0, 1, 3)), dDm=(dy * x).abs().sum((0, 1, 3)))
    return out
