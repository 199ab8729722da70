"""The selective state space scan on the GPU against the token recurrence in
64 bits (needs an MI355X).

Tolerances.  States (fp32): every term is a product of exact 16-bit inputs
and fp32 factors; the 16-bit pair that stands for an fp32 factor is off by
2^-18 (bf16), the gate's exponentials by (|exponent| + 2) 2^-23 with exponents
that matter below 16, sums of 64 terms a chunk by their order.  So each state
is within 2^-15 of the magnitudes that were added into it, plus what the decay
of earlier chunks carries: the reference returns those magnitudes.  Outputs
(16 bits): one rounding of the output; the decayed scores and the chunk's
start state are rounded to the type as operands, half a step each, relative to
the magnitudes of the products: so half a step of the value and a little over
one half step of the sum of magnitudes.  The gradients of x, B and C round one
operand in the same way.  The step sizes' gradient is a suffix sum of fp32
values, each within 2^-16 of its terms' magnitudes (pairs to 2^-18, exponentials
and sums as above), so its bar is 2^-16 of the magnitudes of everything that is
summed behind a token; dA_log and ddt_bias add those bars up.  dD sums exact
products in fp32: 2^-17."""
import pytest
import torch

import _layer_ref as ref
import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32
STATE_SLACK = 2.0 ** -15


def make(B, T, H, G, K, V, dtype, dt_dtype=None, p_dtype=F32, skip=True, bias=True, state=True,
         lens=None, softplus=True, fast=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n = B if lens is None else len(lens)
    t = dict(x=r(B, T, H, V).to(dtype), B=r(B, T, G, K).to(dtype), C=r(B, T, G, K).to(dtype),
             A_log=torch.log(torch.rand(H, generator=g) * 15 + 1).to(p_dtype),
             D=r(H).to(p_dtype) if skip else None,
             dt_bias=(r(H) - (0 if fast else 4)).to(p_dtype) if bias else None,
             state=r(n, H, K, V) if state else None,
             cu=None if lens is None else torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32),
             dy=r(B, T, H, V).to(dtype), dlast=r(n, H, K, V))
    raw = r(B, T, H) if softplus else torch.rand(B, T, H, generator=g) / 8
    t["dt"] = raw.to(dt_dtype or dtype)
    return t


def dev(t):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in t.items()}


CASES = {
    # name: (B, T, H, G, K, V, dtype), options
    "one_token": ((1, 1, 2, 1, 64, 64, BF), {}),
    "chunk": ((1, 64, 1, 1, 128, 64, BF), dict(state=False)),
    "chunk_and_one": ((2, 65, 3, 1, 64, 128, HF), dict(skip=False)),
    "ragged": ((2, 150, 4, 2, 128, 128, BF), dict(dt_dtype=F32)),
    "no_bias": ((1, 100, 2, 2, 64, 64, HF), dict(bias=False, p_dtype=HF)),
    "plain_steps": ((1, 130, 2, 1, 128, 64, BF), dict(softplus=False, bias=False)),
    "fast_decay": ((1, 200, 2, 1, 64, 64, BF), dict(fast=True)),
    "packed": ((1, 400, 4, 2, 128, 64, HF), dict(lens=[1, 0, 63, 64, 65, 0, 200, 7, 0])),
    "packed_first_empty": ((1, 70, 2, 1, 64, 128, BF), dict(lens=[0, 70], state=False)),
    "cut": ((1, 2500, 2, 1, 128, 64, BF), {}),
    "cut_packed": ((1, 3000, 2, 2, 64, 128, HF), dict(lens=[5, 1500, 0, 1, 1430, 64])),
    "cut_dense": ((2, 1111, 1, 1, 128, 128, HF), dict(state=False)),
}


def case(name):
    shape, kw = CASES[name]
    return make(*shape, **kw), kw.get("softplus", True)


def args(g):
    return (g["x"], g["dt"], g["A_log"], g["B"], g["C"], g["D"], g["dt_bias"])


def check_forward(t, y, last, r):
    eps = ref.half_step(t["x"].dtype)
    ref.held("y", y, r["y"], r["ym"], t["x"].dtype, 1.25 * eps)
    ref.held("state", last, r["last"], r["lastm"], F32, STATE_SLACK)


@pytest.mark.parametrize("name", list(CASES))
def test_forward(name):
    t, sp = case(name)
    g = dev(t)
    y, last = gdr.chunk_selective_scan_fwd(*args(g), sp, g["state"], True, g["cu"], t["cu"])
    torch.cuda.synchronize()
    r = ref.scan(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["D"], t["dt_bias"], sp, t["state"],
                 t["cu"])
    check_forward(t, y, last, r)


@pytest.mark.parametrize("name", ["one_token", "chunk_and_one", "ragged", "packed", "plain_steps"])
def test_token_by_token(name):
    t, sp = case(name)
    g = dev(t)
    kw = dict(cu_seqlens=g["cu"], cu_seqlens_cpu=t["cu"])
    y, last = gdr.fused_recurrent_selective_scan(*args(g), sp, g["state"], True, **kw)
    r = ref.scan(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["D"], t["dt_bias"], sp, t["state"],
                 t["cu"])
    check_forward(t, y, last, r)
    if g["state"] is not None:
        st = g["state"].clone()
        y2, last2 = gdr.fused_recurrent_selective_scan(*args(g), sp, st, inplace_final_state=True, **kw)
        assert last2.data_ptr() == st.data_ptr()
        assert torch.equal(y, y2) and torch.equal(last, last2)


GRADS = ("dx", "ddt", "dA", "dB", "dC", "dD", "dbias", "ds")


def grad_slack(name, dtype):
    if name in ("dx", "dB", "dC"):
        return 1.25 * ref.half_step(dtype)
    return {"ds": STATE_SLACK, "dD": 2.0 ** -17}.get(name, 2.0 ** -16)


MORE = {
    "shared_by_3": ((1, 130, 6, 2, 64, 64, BF), {}),
    "shared_by_8": ((2, 77, 8, 1, 128, 64, HF), dict(p_dtype=HF)),
    "cut_shared": ((1, 1500, 4, 1, 64, 64, BF), dict(lens=[700, 1, 0, 799])),
}


@pytest.mark.parametrize("name", list(CASES) + list(MORE))
def test_gradients(name):
    shape, kw = {**CASES, **MORE}[name]
    t = make(*shape, **kw)
    sp = kw.get("softplus", True)
    g = dev(t)
    names = [n for n, k in zip(GRADS, ("x", "dt", "A_log", "B", "C", "D", "dt_bias", "state"))
             if g[k] is not None]
    leaves = [g[k].requires_grad_(True) for k in ("x", "dt", "A_log", "B", "C", "D", "dt_bias", "state")
              if g[k] is not None]
    y, last = gdr.chunk_selective_scan(*args(g), sp, g["state"], True, g["cu"], t["cu"])
    got = torch.autograd.grad([y, last], leaves, [g["dy"], g["dlast"]])
    torch.cuda.synchronize()
    r = ref.scan(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["D"], t["dt_bias"], sp, t["state"],
                 t["cu"], t["dy"], t["dlast"])
    check_forward(t, y.detach(), last.detach(), r)
    for n, v in zip(names, got):
        err = (ref.d(v) - r[n]).norm() / r[n].norm()
        print(name, n, "%.2e" % float(err), flush=True)
        ref.held(n, v, r[n], r[n + "m"], v.dtype, grad_slack(n, t["x"].dtype))
    # without the final state's gradient, and the same bits twice
    a1 = gdr.chunk_selective_scan_bwd(*args(g)[:5], g["dy"], g["D"], g["dt_bias"], sp, None, g["state"],
                                      g["cu"], t["cu"])
    a2 = gdr.chunk_selective_scan_bwd(*args(g)[:5], g["dy"], g["D"], g["dt_bias"], sp,
                                      torch.zeros_like(g["dlast"]), g["state"], g["cu"], t["cu"])
    for u, v in zip(a1, a2):
        assert (u is None) == (v is None) and (u is None or torch.equal(u, v))


def test_gradient_against_differences():
    """Random directions, dt, its bias, A_log, D and the state in fp32; x, B and
    C move on their 16-bit grid, so their differences are taken against the
    exact step.  The outputs round to 2^-9 of themselves, which a step of 2^-4
    turns into 2^-5 per output, random over 8,000 outputs; the curvature adds
    h^2 / 6: 5 % of the directional derivative's own root of squares."""
    t = dev(make(2, 70, 2, 1, 64, 64, HF, dt_dtype=F32, seed=3))
    keys = ("x", "dt", "A_log", "B", "C", "D", "dt_bias", "state")
    got = gdr.chunk_selective_scan_bwd(*args(t)[:5], t["dy"], t["D"], t["dt_bias"], True, t["dlast"],
                                       t["state"])
    gen = torch.Generator().manual_seed(2)
    h = 2.0 ** -4
    for k, g in zip(keys, got):
        v = torch.randn(t[k].shape, generator=gen).cuda()

        def value(s):
            q = dict(t)
            q[k] = (t[k].float() + s * v).to(t[k].dtype)
            y, last = gdr.chunk_selective_scan_fwd(*args(q), True, q["state"])
            return (y.double() * t["dy"]).sum() + (last.double() * t["dlast"]).sum(), q[k].double()

        (up, a), (down, b) = value(h), value(-h)
        want = (g.double() * (a - b)).sum()
        scale = (g.double() * (a - b)).square().sum().sqrt()
        assert abs(up - down - want) <= 0.05 * scale + 2e-3 * abs(want), (k, float(up - down), float(want))


def test_captured_and_replayed():
    """A training step in a graph, replayed with eager work in between; two
    graphs with workspaces of their own."""
    t = dev(make(1, 1500, 4, 2, 64, 64, BF, lens=[900, 0, 600]))
    cu = t["cu"].cpu()

    def step():
        y, last = gdr.chunk_selective_scan_fwd(*args(t), True, t["state"], True, t["cu"], cu)
        g = gdr.chunk_selective_scan_bwd(*args(t)[:5], t["dy"], t["D"], t["dt_bias"], True, t["dlast"],
                                         t["state"], t["cu"], cu)
        return (y, last) + g

    want = step()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    graphs = []
    for _ in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        graphs.append((graph, out))
    for _ in range(3):
        for graph, out in graphs:
            for o in out:
                o.zero_()
            graph.replay()
        torch.cuda.synchronize()
        for graph, out in graphs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))
        step()


def test_steps_continue_a_prompt():
    t = make(2, 140, 4, 2, 128, 64, BF)
    g = dev(t)
    r = ref.scan(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["D"], t["dt_bias"], True, t["state"])
    cut = lambda a, b: [g[k][:, a:b] for k in ("x", "dt", "B", "C")]  # noqa: E731
    x, dt, b, c = cut(0, 130)
    y, st = gdr.chunk_selective_scan_fwd(x, dt, g["A_log"], b, c, g["D"], g["dt_bias"], True, g["state"])
    ys = [y]
    for i in range(130, 140):
        x, dt, b, c = cut(i, i + 1)
        y, st = gdr.fused_recurrent_selective_scan(x, dt, g["A_log"], b, c, g["D"], g["dt_bias"], True,
                                                   st, inplace_final_state=True)
        ys.append(y)
    check_forward(t, torch.cat(ys, 1), st, r)


def test_slices_of_one_projection_are_read_in_place():
    g = torch.Generator().manual_seed(0)
    H, G, K, V = 4, 2, 64, 64
    wide = torch.randn(2, 90, H * V + 2 * G * K + 3, generator=g).to(BF).cuda()
    x = wide[..., 1:1 + H * V].unflatten(-1, (H, V))     # odd offsets and stride: no alignment
    b = wide[..., 1 + H * V:1 + H * V + G * K].unflatten(-1, (G, K))
    c = wide[..., 2 + H * V + G * K:2 + H * V + 2 * G * K].unflatten(-1, (G, K))
    t = dev(make(2, 90, H, G, K, V, BF))
    kw = dict(D=t["D"], dt_bias=t["dt_bias"], initial_state=t["state"])
    for f in (gdr.chunk_selective_scan_fwd, gdr.fused_recurrent_selective_scan):
        y, s = f(x, t["dt"], t["A_log"], b, c, **kw)
        y2, s2 = f(x.contiguous(), t["dt"], t["A_log"], b.contiguous(), c.contiguous(), **kw)
        assert torch.equal(y, y2) and torch.equal(s, s2)


@pytest.mark.parametrize("K,V,dtype", [(64, 64, HF), (128, 128, BF)])
def test_negative_steps(K, V, dtype):
    """Without softplus a step may be negative: the state then grows.  Log
    decays are up to 1 a token here and sum to a few, so the tolerances' bound
    on the exponents (16) holds."""
    t = make(1, 300, 2, 1, K, V, dtype, dt_dtype=F32, softplus=False, bias=False, lens=[130, 170])
    t["dt"] = torch.randn(t["dt"].shape, generator=torch.Generator().manual_seed(5)) / 64
    g = dev(t)
    y, last = gdr.chunk_selective_scan_fwd(*args(g), False, g["state"], True, g["cu"], t["cu"])
    got = gdr.chunk_selective_scan_bwd(*args(g)[:5], g["dy"], g["D"], None, False, g["dlast"], g["state"],
                                       g["cu"], t["cu"])
    r = ref.scan(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["D"], None, False, t["state"], t["cu"],
                 t["dy"], t["dlast"])
    check_forward(t, y, last, r)
    for n, v in zip(GRADS, got):
        if v is not None:
            ref.held(n, v, r[n], r[n + "m"], v.dtype, grad_slack(n, dtype))
    y, last = gdr.fused_recurrent_selective_scan(*args(g), False, g["state"], True, g["cu"], t["cu"])
    check_forward(t, y, last, r)


def test_many_short_sequences():
    """More sequences than the cut looks at one by one, some of one token."""
    lens = [1 + (i * 7) % 40 for i in range(150)] + [0, 900]
    t = make(1, sum(lens), 2, 1, 64, 64, BF, lens=lens)
    g = dev(t)
    y, last = gdr.chunk_selective_scan_fwd(*args(g), True, g["state"], True, g["cu"], t["cu"])
    r = ref.scan(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["D"], t["dt_bias"], True, t["state"],
                 t["cu"])
    check_forward(t, y, last, r)


def test_packed_sequences_are_independent():
    """Each packed sequence has the bits of its own dense run when neither is
    cut; NaNs stay in their sequence."""
    lens = [70, 3, 129]
    t = make(1, sum(lens), 2, 1, 64, 64, BF, lens=lens)
    g = dev(t)
    y, last = gdr.chunk_selective_scan_fwd(*args(g), True, g["state"], True, g["cu"], t["cu"])
    at = 0
    for i, n in enumerate(lens):
        sl = [g[k][:, at:at + n] for k in ("x", "dt", "B", "C")]
        y1, l1 = gdr.chunk_selective_scan_fwd(sl[0], sl[1], g["A_log"], sl[2], sl[3], g["D"],
                                              g["dt_bias"], True, g["state"][i:i + 1])
        assert torch.equal(y[:, at:at + n], y1) and torch.equal(last[i:i + 1], l1)
        at += n
    x = g["x"].clone()
    x[0, 71] = float("nan")
    y2, l2 = gdr.chunk_selective_scan_fwd(x, *args(g)[1:], True, g["state"], True, g["cu"], t["cu"])
    assert y2[0, 71:73].isnan().all() and l2[1].isnan().all()
    keep = [i for i in range(sum(lens)) if not 70 <= i < 73]
    assert torch.equal(y2[:, keep], y[:, keep]) and torch.equal(l2[[0, 2]], last[[0, 2]])


def test_python_refusals():
    t = dev(make(2, 8, 4, 2, 64, 64, BF))
    a = args(t)

    def f(**kw):
        q = {**t, **kw}
        return gdr.chunk_selective_scan_fwd(*args(q), initial_state=q["state"], cu_seqlens=kw.get("cu"))

    for call, name in [
        (lambda: f(x=t["x"][..., :32]), "GDR_ERR_SHAPE"),
        (lambda: gdr.chunk_selective_scan_fwd(t["x"][..., :32], *a[1:]), "GDR_ERR_HEAD_DIM"),
        (lambda: f(B=t["B"].half()), "GDR_ERR_DTYPE"),
        (lambda: f(C=t["C"][:, :4]), "GDR_ERR_SHAPE"),
        (lambda: f(dt=t["dt"].half()), "GDR_ERR_DTYPE"),
        (lambda: f(A_log=t["A_log"][:2]), "GDR_ERR_SHAPE"),
        (lambda: f(D=t["D"].bfloat16()), "GDR_ERR_DTYPE"),
        (lambda: f(state=t["state"].half()), "GDR_ERR_DTYPE"),
        (lambda: f(state=t["state"][:1]), "GDR_ERR_SHAPE"),
        (lambda: f(x=t["x"].float(), B=t["B"].float(), C=t["C"].float(), dt=t["dt"].float()),
         "GDR_ERR_DTYPE"),
        (lambda: gdr.chunk_selective_scan_fwd(t["x"][:, :, :3], t["dt"][:, :, :3], t["A_log"][:3], t["B"],
                                              t["C"]), "GDR_ERR_HEADS"),
        (lambda: f(cu=torch.tensor([0, 8]), state=None), "GDR_ERR_VARLEN"),
        (lambda: gdr.fused_recurrent_selective_scan(*a, initial_state=t["state"].transpose(2, 3),
                                                    inplace_final_state=True), "GDR_ERR_ARG"),
        (lambda: gdr.fused_recurrent_selective_scan(*a, inplace_final_state=True), "GDR_ERR_ARG"),
    ]:
        with pytest.raises(gdr.GdrError) as e:
            call()
        assert e.value.name == name, (e.value, name)
