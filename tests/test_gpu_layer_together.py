"""The layer operators as a mixer layer runs them, one after the other (needs
an MI355X): residual norm, projection, convolution on a slice of it, the scan
and the delta rule on slices of that, the norm of what they give; a training
step, and a prompt continued token by token.  Every operator's output and
gradient is held against the 64-bit reference applied to the tensors that it
really got, so each keeps the tolerance that its own tests derive.  Also here:
the operators on other streams, two calls at once, and tensors past 2^31
elements."""
import pytest
import torch

import _layer_ref as ref
import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
H, G, K, V, DM = 4, 2, 128, 128, 256
XBC = H * V + 2 * G * K
EPS = 1e-5
NORM, CONV = 2.0 ** -20, 2.0 ** -20   # fp32 sums of at most 2048 or 5 terms, in blocks
STATE = 2.0 ** -15                    # the scan's 16-bit pairs and exponentials


def weights(seed=0, dtype=BF):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = dict(n1=1 + r(DM) / 8, win=r(DM, XBC + H) / 16, cw=r(XBC, 4) / 2, cb=r(XBC) / 4,
             A_log=torch.log(torch.rand(H, generator=g) * 15 + 1), D=r(H), dt_bias=r(H) - 4,
             n2=1 + r(H * V) / 8, wout=r(H * V, DM) / 16)
    f32 = ("cw", "cb", "A_log", "D", "dt_bias")
    return {k: (v if k in f32 else v.to(dtype)).cuda() for k, v in w.items()}


def inputs(B, T, n, seed=1):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(x=r(B, T, DM).to(BF).cuda(), res=r(B, T, DM).cuda(),
                cs=r(n, 3, XBC).to(BF).cuda(), ss=r(n, H, K, V).cuda())


def split(c, dt):
    B, T = c.shape[:2]
    return (c[..., :H * V].view(B, T, H, V), c[..., H * V:H * V + G * K].view(B, T, G, K),
            c[..., H * V + G * K:].view(B, T, G, K), dt)


def layer(w, t, cu=None, cu_cpu=None, mid=lambda name, v: v):
    """The layer's outputs; `mid` sees every tensor between two operators."""
    y, h = gdr.rms_norm(t["x"], w["n1"], EPS, residual=t["res"])
    mid("y", y), mid("h", h)
    p = mid("p", y @ w["win"])
    xbc, dt = p[..., :XBC], p[..., XBC:]
    c, cs = gdr.causal_conv1d(xbc, w["cw"], w["cb"], "silu", t["cs"], True, cu, cu_cpu)
    mid("c", c)
    x, b, k, dt = split(c, dt)
    s, ss = gdr.chunk_selective_scan(x, dt, w["A_log"], b, k, w["D"], w["dt_bias"], True, t["ss"], True,
                                     cu, cu_cpu)
    mid("s", s)
    o, _ = gdr.chunk_gated_delta_rule(k, b, x, dt.float(), torch.full_like(dt, 0.5),
                                      use_qk_l2norm_in_kernel=True, use_gate_in_kernel=True,
                                      A_log=w["A_log"], dt_bias=w["dt_bias"], cu_seqlens=cu,
                                      cu_seqlens_cpu=cu_cpu)
    mid("o", o)
    z = mid("z", (s + o).flatten(-2))
    u = mid("u", gdr.rms_norm(z, w["n2"], EPS))
    return u @ w["wout"], h, cs, ss


@pytest.mark.parametrize("B,T,lens", [(2, 150, None), (1, 333, [100, 0, 1, 232]), (1, 1400, None)])
def test_a_training_step(B, T, lens):
    n = B if lens is None else len(lens)
    cu_cpu = None if lens is None else torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    cu = None if cu_cpu is None else cu_cpu.cuda()
    w, t = weights(), inputs(B, T, n)
    for v in (w, t):
        for q in v.values():
            q.requires_grad_(True)
    m = {}

    def mid(name, v):
        v.retain_grad()
        m[name] = v
        return v

    out, h, cs, ss = layer(w, t, cu, cu_cpu, mid)
    gen = torch.Generator().manual_seed(9)
    dout = torch.randn(out.shape, generator=gen).to(BF).cuda()
    dh = torch.randn(h.shape, generator=gen).cuda()
    dcs = torch.randn(cs.shape, generator=gen).to(BF).cuda()
    dss = torch.randn(ss.shape, generator=gen).cuda()
    torch.autograd.backward([out, h, cs, ss], [dout, dh, dcs, dss])
    torch.cuda.synchronize()
    hs = ref.half_step(BF)

    # the first norm: y, h; its gradient from y's and from the residual stream's
    r = ref.norm(t["x"], w["n1"], EPS, t["res"], m["y"].grad, dh)
    ref.held("y", m["y"], r["y"], r["y"].abs(), BF, NORM)
    ref.held("h", h, r["h"], r["h"].abs(), F32, 0.0)
    ref.held("dres", t["res"].grad, r["dx"], r["dxm"], F32, NORM)
    ref.held("dx", t["x"].grad, r["dx"], r["dxm"], BF, NORM)
    ref.held("dn1", w["n1"].grad, r["dw"], r["dwm"], BF, NORM)

    # the convolution, on the projection's slice
    xbc, raw = m["p"][..., :XBC], m["p"][..., XBC:]
    r = ref.conv(xbc, w["cw"], w["cb"], True, t["cs"], cu_cpu, m["c"].grad, dcs)
    ref.held("c", m["c"], *r["y"], BF, CONV)
    ref.held("cs", cs, *r["last"], BF, 0.0)
    for name, got, dt in (("dx", m["p"].grad[..., :XBC], BF), ("dw", w["cw"].grad, F32),
                          ("db", w["cb"].grad, F32), ("ds", t["cs"].grad, BF)):
        ref.held("conv " + name, got, *r[name], dt, CONV)

    # the scan.  Its inputs feed the delta rule as well, whose gradients torch
    # adds to its own: those are taken from a second run of the delta rule alone
    leaf = {k: v.detach().requires_grad_(True) for k, v in (("c", m["c"]), ("p", raw.contiguous()))}
    x, b, k, dt = split(leaf["c"], leaf["p"])
    o, _ = gdr.chunk_gated_delta_rule(k, b, x, dt.float(), torch.full_like(dt, 0.5),
                                      use_qk_l2norm_in_kernel=True, use_gate_in_kernel=True,
                                      A_log=w["A_log"].detach(), dt_bias=w["dt_bias"].detach(),
                                      cu_seqlens=cu, cu_seqlens_cpu=cu_cpu)
    assert torch.equal(o, m["o"])
    o.backward(m["o"].grad)
    x, b, k, dt = split(m["c"].detach(), raw.detach())
    r = ref.scan(x, dt, w["A_log"], b, k, w["D"], w["dt_bias"], True, t["ss"], cu_cpu, m["s"].grad, dss)
    ref.held("s", m["s"], r["y"], r["ym"], BF, 1.25 * hs)
    ref.held("ss", ss, r["last"], r["lastm"], F32, STATE)
    ref.held("dss", t["ss"].grad, r["ds"], r["dsm"], F32, STATE)
    ref.held("dD", w["D"].grad, r["dD"], r["dDm"], F32, 2.0 ** -17)
    # a sum of two bf16 gradients is rounded once more: half a step of each
    # summand and of the sum
    dx, db, dk, _ = split(m["c"].grad, raw)
    ox, ob, ok, _ = split(leaf["c"].grad, raw)
    for name, got, other in (("dx", dx, ox), ("dB", db, ob), ("dC", dk, ok)):
        other = ref.d(other)
        # k, b and x are slices of one tensor: nothing else adds to them
        ref.held("scan " + name, got, r[name] + other,
                 r[name + "m"] + (r[name].abs() + other.abs()) / 1.25, BF, 1.25 * hs)
    other = ref.d(leaf["p"].grad)
    ref.held("scan ddt", m["p"].grad[..., XBC:], r["ddt"] + other,
             2.0 ** -16 / hs * r["ddtm"] + r["ddt"].abs() + other.abs(), BF, hs)

    # the second norm
    r = ref.norm(m["z"], w["n2"], EPS, None, m["u"].grad)
    ref.held("u", m["u"], r["y"], r["y"].abs(), BF, NORM)
    ref.held("dz", m["z"].grad, r["dx"], r["dxm"], BF, NORM)
    ref.held("dn2", w["n2"].grad, r["dw"], r["dwm"], BF, NORM)


def decode(w, x, res, cs, ss, ds):
    """One token per sequence on cached states, all updated in place."""
    y, h, _ = gdr.rms_norm_fwd(x, w["n1"], EPS, res)
    p = y @ w["win"]
    c = gdr.causal_conv1d_update(p[..., :XBC], cs, w["cw"], w["cb"], "silu")
    xs, b, k, dt = split(c, p[..., XBC:])
    s, _ = gdr.fused_recurrent_selective_scan(xs, dt, w["A_log"], b, k, w["D"], w["dt_bias"], True, ss,
                                              inplace_final_state=True)
    o, _ = gdr.fused_recurrent_gated_delta_rule(
        k, b, xs, dt.float(), torch.full_like(dt, 0.5), initial_state=ds,
        use_qk_l2norm_in_kernel=True, use_gate_in_kernel=True, A_log=w["A_log"], dt_bias=w["dt_bias"],
        inplace_final_state=True)
    z = (s + o).flatten(-2)
    q, scale, _ = gdr.rms_norm_quant(z, w["n2"], EPS, format="fp8")
    return y, h, p, c, s, z, q, scale


def test_a_prompt_and_steps_in_a_graph():
    """A decode step captured into a graph and replayed over eight tokens, the
    states carried in place: every operator is held against the reference over
    the whole sequence (the convolution's and the scan's from the first
    token on)."""
    B, T, S = 3, 130, 8
    w, t = weights(3), inputs(B, T + S, B, 4)
    y, h, _ = gdr.rms_norm_fwd(t["x"][:, :T], w["n1"], EPS, t["res"][:, :T].contiguous())
    p = y @ w["win"]
    c, cs = gdr.causal_conv1d_fwd(p[..., :XBC], w["cw"], w["cb"], "silu", t["cs"])
    x, b, k, dt = split(c, p[..., XBC:])
    s, ss = gdr.chunk_selective_scan_fwd(x, dt, w["A_log"], b, k, w["D"], w["dt_bias"], True, t["ss"])
    ds = torch.zeros(B, H, K, V, device="cuda")
    seen = dict(p=[p], c=[c], s=[s])
    xt, rt = t["x"][:, :1].clone(), t["res"][:, :1].clone()
    states = (cs, ss, ds)
    kept = [v.clone() for v in states]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        decode(w, xt, rt, *states)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = decode(w, xt, rt, *states)
    for v, q in zip(states, kept):
        v.copy_(q)
    for i in range(T, T + S):
        xt.copy_(t["x"][:, i:i + 1])
        rt.copy_(t["res"][:, i:i + 1])
        graph.replay()
        y, h, p, c, s, z, q, scale = (v.clone() for v in out)
        r = ref.norm(xt, w["n1"], EPS, rt)
        ref.held("y", y, r["y"], r["y"].abs(), BF, NORM)
        ref.held("h", h, r["h"], r["h"].abs(), F32, 0.0)
        # e4m3 of the row's largest: the scale is one fp32 division of it, a
        # value's quotient is rounded by half a step, below the type's normal
        # range (2^-6) by half of 2^-9
        r = ref.norm(z, w["n2"], EPS)["y"]
        top = r.abs().amax(-1, keepdim=True)
        assert ((ref.d(scale) * 448 / top - 1).abs() < 2.0 ** -19).all()
        off = (ref.d(q.float()) * ref.d(scale) - r).abs()
        assert (off <= 2.0 ** -4 * r.abs() * (1 + 2.0 ** -15) + 2.0 ** -10 * ref.d(scale) * 1.001).all()
        for name, v in (("p", p), ("c", c), ("s", s)):
            seen[name].append(v)
    torch.cuda.synchronize()
    p, c, s = (torch.cat(seen[k], 1) for k in ("p", "c", "s"))
    r = ref.conv(p[..., :XBC], w["cw"], w["cb"], True, t["cs"])
    ref.held("c", c, *r["y"], BF, CONV)
    ref.held("cs", cs, *r["last"], BF, 0.0)
    x, b, k, dt = split(c, p[..., XBC:])
    r = ref.scan(x, dt, w["A_log"], b, k, w["D"], w["dt_bias"], True, t["ss"])
    ref.held("s", s, r["y"], r["ym"], BF, 1.25 * ref.half_step(BF))
    ref.held("ss", ss, r["last"], r["lastm"], F32, STATE)


def test_two_layers_at_once_on_two_streams():
    """Two training steps on streams of their own, launched in turn, have the
    bits of the same steps alone; tensors made on one stream are used on
    another after a wait."""
    jobs = [(weights(s), inputs(2, 700, 2, s + 1)) for s in (5, 7)]
    for w, t in jobs:
        for v in (w, t):
            for q in v.values():
                q.requires_grad_(True)

    def step(w, t):
        out, h, cs, ss = layer(w, t)
        leaves = list(w.values()) + list(t.values())
        return [out, ss] + list(torch.autograd.grad(
            [out, h, cs, ss], leaves, [torch.ones_like(v) for v in (out, h, cs, ss)]))

    want = [step(*j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(3):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(step(*jobs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def scan_args(B, T, h, g, k, v, seed=0, dtype=BF):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=gen, device="cuda", dtype=dtype)  # noqa: E731
    return dict(x=r(B, T, h, v), dt=r(B, T, h), A_log=torch.rand(h, generator=gen, device="cuda") * 2,
                B=r(B, T, g, k), C=r(B, T, g, k), D=torch.ones(h, device="cuda"),
                dt_bias=torch.full((h,), -4.0, device="cuda"))


@pytest.mark.parametrize("T,lens", [(64, None), (3000, None), (3000, [5, 1500, 0, 1, 1430, 64])])
def test_kept_states_and_recomputed_ones_give_the_same_gradients(T, lens):
    """Also twice through one graph, which must leave the kept states as they
    were, and with gradients of some inputs only."""
    cu = None if lens is None else torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    a = scan_args(1, T, 4, 2, 64, 128)
    n = 1 if lens is None else len(lens)
    a["initial_state"] = torch.randn(n, 4, 64, 128, device="cuda")
    a = {k: v.requires_grad_(True) for k, v in a.items()}
    kw = dict(output_final_state=True, cu_seqlens=None if cu is None else cu.cuda(), cu_seqlens_cpu=cu)
    res = []
    for again in (False, True):
        y, s = gdr.chunk_selective_scan(**a, **kw, recompute_states=again)
        gs = [torch.ones_like(y), torch.ones_like(s)]
        res += [torch.autograd.grad([y, s], list(a.values()), gs, retain_graph=True) for _ in range(2)]
    for r in res[1:]:
        assert all(torch.equal(p, q) for p, q in zip(r, res[0]))
    only = {k: v.detach().requires_grad_(k == "dt") for k, v in a.items()}
    y, _ = gdr.chunk_selective_scan(**only, **kw)
    y.sum().backward()
    full, _ = gdr.chunk_selective_scan(**a, **kw)
    want = torch.autograd.grad(full.sum(), [a["dt"]])[0]
    assert torch.equal(only["dt"].grad, want)
    with torch.no_grad():
        z, _ = gdr.chunk_selective_scan(**a, **kw)
        z2, _ = gdr.chunk_selective_scan_fwd(**a, **kw)
    assert torch.equal(z, z2) and not z.requires_grad


def test_a_gradient_of_the_state_alone():
    a = {k: v.requires_grad_(True) for k, v in scan_args(2, 100, 2, 1, 64, 64).items()}
    _, s = gdr.chunk_selective_scan(**a, output_final_state=True)
    s.square().sum().backward()
    zero = torch.zeros(2, 100, 2, 64, device="cuda", dtype=BF)
    plain = [a[k].detach() for k in ("x", "dt", "A_log", "B", "C")]
    want = gdr.chunk_selective_scan_bwd(*plain, zero, a["D"].detach(), a["dt_bias"].detach(), True,
                                        2 * s.detach())
    for k, v in zip(("x", "dt", "A_log", "B", "C", "D", "dt_bias"), want):
        assert torch.equal(a[k].grad, v)
    assert not a["C"].grad.any() and not a["D"].grad.any()


def test_past_two_to_the_31_elements():
    """Outputs at the end of tensors of more than 2^31 elements equal those of
    the end alone."""
    T, D = (1 << 20) + 700, 2048
    big = torch.empty(1, T, D, device="cuda", dtype=BF)
    gen = torch.Generator(device="cuda").manual_seed(0)
    big.normal_(generator=gen)
    w = torch.randn(D, 4, device="cuda")
    y, last = gdr.causal_conv1d_fwd(big, w)
    tail, tail_last = gdr.causal_conv1d_fwd(big[:, -500:], w, initial_state=big[:, -503:-500].clone())
    assert torch.equal(y[:, -500:], tail) and torch.equal(last, tail_last)
    dx, _, _, _ = gdr.causal_conv1d_bwd(big, w, None, y)
    dtail, _, _, _ = gdr.causal_conv1d_bwd(big[:, -500:], w, None, y[:, -500:],
                                           initial_state=big[:, -503:-500].clone())
    assert torch.equal(dx[:, -490:], dtail[:, -490:])
    del dx
    n = torch.randn(D, device="cuda")
    u, _, rstd = gdr.rms_norm_fwd(big, n)
    assert torch.equal(u[:, -500:], gdr.rms_norm_fwd(big[:, -500:], n)[0])
    dx, _, _ = gdr.rms_norm_bwd(y, big, n, rstd)
    assert torch.equal(dx[:, -500:], gdr.rms_norm_bwd(y[:, -500:], big[:, -500:].contiguous(), n,
                                                      rstd[:, -500:].contiguous())[0])
    del u, dx, y
    q, scale, _ = gdr.rms_norm_quant(big, n, format="int8", group_size=128)
    q2, scale2, _ = gdr.rms_norm_quant(big[:, -500:], n, format="int8", group_size=128)
    assert torch.equal(q[:, -500:], q2) and torch.equal(scale[:, -500:], scale2)


def test_a_long_scan_past_two_to_the_31_elements():
    """x, y and dx of 2^31 elements and more; the last 10,000 tokens alone,
    from the state that the tokens before them leave: the two runs' 64-token
    chunks coincide, so only the way the start state was reached differs, by
    rounding of fp32 states (2^-15 of the magnitudes, which decay by far more
    than that in between)."""
    T, cut = (1 << 20) + 640, (1 << 20) - 9360 + 640 - 640 % 64
    cut -= cut % 64
    a = scan_args(1, T, 16, 1, 64, 128)
    y, s = gdr.chunk_selective_scan_fwd(**a)
    seq = ("x", "dt", "B", "C")
    head = {k: (v[:, :cut] if k in seq else v) for k, v in a.items()}
    tail = {k: (v[:, cut:] if k in seq else v) for k, v in a.items()}
    _, mid = gdr.chunk_selective_scan_fwd(**head)
    y2, s2 = gdr.chunk_selective_scan_fwd(**tail, initial_state=mid)
    assert (s - s2).norm() <= 2.0 ** -14 * s.norm()
    assert (y[:, cut:].float() - y2.float()).norm() <= ref.half_step(BF) * y2.float().norm()
    names = ("x", "dt", "A_log", "B", "C")
    full = gdr.chunk_selective_scan_bwd(*[a[k] for k in names], y, a["D"], a["dt_bias"])
    part = gdr.chunk_selective_scan_bwd(*[tail[k] for k in names], y[:, cut:].contiguous(), a["D"],
                                        a["dt_bias"], initial_state=mid)
    for k, u, v in zip(names, full, part):
        if k != "A_log":
            u, v = u[:, cut:].float(), v.float()
            assert (u - v).norm() <= 2 * ref.half_step(BF) * v.norm(), k


def test_many_cached_states():
    """Decode on 2^31 fp32 elements of states and more: the last sequences
    equal their own run."""
    B, h = 4200, 32
    a = scan_args(B, 1, h, 2, 128, 128)
    st = torch.empty(B, h, 128, 128, device="cuda").normal_()
    own = st[-2:].clone()
    y, _ = gdr.fused_recurrent_selective_scan(**a, initial_state=st, inplace_final_state=True)
    b = {k: (v[-2:] if v.dim() > 1 else v) for k, v in a.items()}
    y2, own = gdr.fused_recurrent_selective_scan(**b, initial_state=own, inplace_final_state=True)
    assert torch.equal(y[-2:], y2) and torch.equal(st[-2:], own)


def test_strides_beyond_a_tile_are_copied():
    """Tokens further apart than a tile's addresses reach."""
    wide = torch.randn(1, 70, (1 << 23) + 8, device="cuda", dtype=BF)
    a = scan_args(1, 70, 2, 1, 64, 64)
    x = wide[..., 8:8 + 128].unflatten(-1, (2, 64))
    a.pop("x")
    y, s = gdr.chunk_selective_scan_fwd(x, **a)
    y2, s2 = gdr.chunk_selective_scan_fwd(x.contiguous(), **a)
    assert torch.equal(y, y2) and torch.equal(s, s2)
