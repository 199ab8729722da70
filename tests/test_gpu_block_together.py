"""The operators at a layer's ends as a stack runs them, with the recurrence
between them (needs an MI355X): projection in 8 bits, convolution, gated delta
rule, the norm of its output with its gate, the projection back, and the norms
around the residual's addition; a prompt and decode steps in a graph, and a
training step.  Every operator's output and gradient is held against the
64-bit reference applied to the tensors that it really got, so each keeps the
tolerance that its own tests derive.  Also here: captured gradients, and two
calls at once."""
import pytest
import torch

import _block_ref as bref
import _layer_ref as ref
import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
H, K, V, DM = 4, 128, 128, 320
QKV, HV = H * (2 * K + V), H * V
WIN = QKV + HV + 2 * H                 # q, k, v, the gate, and two values a head
EPS = 1e-5
OUT, SLACK, SUM_SLACK, PRODUCT = 2.0 ** -19, 2.0 ** -17, 2.0 ** -15, 2.0 ** -21


def weights(seed=0):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    w = dict(win=r(WIN, DM) / DM ** 0.5, wout=r(DM, HV) / HV ** 0.5, cw=r(QKV, 4) / 2, nv=1 + r(V) / 8,
             post=1 + r(DM) / 8, pre=1 + r(DM) / 8, scale=0.5 + r(DM) / 16, pre0=1 + r(DM) / 8)
    return {k: v.to(F32 if k == "cw" else BF).cuda() for k, v in w.items()}


def eight(w):
    """The weights of a model in 8 bits."""
    return {**w, "qin": gdr.quantize_rows(w["win"]), "qout": gdr.quantize_rows(w["wout"])}


def mixer(p, cs, ds, update, cu=None, cu_cpu=None):
    """From the projection p [B, T, WIN] to the recurrence's output [B, T, H V]."""
    B, T = p.shape[:2]
    if update:
        c = gdr.causal_conv1d_update(p[..., :QKV], cs, w_conv(cs), None)
    else:
        c, cs = gdr.causal_conv1d_fwd(p[..., :QKV], w_conv(cs), None, "silu", cs, True, cu, cu_cpu)
    q, k, v = (c[..., i:j].unflatten(-1, (H, -1)).contiguous()
               for i, j in ((0, H * K), (H * K, 2 * H * K), (2 * H * K, QKV)))
    g = -torch.nn.functional.softplus(p[..., QKV + HV:QKV + HV + H].float())
    beta = torch.sigmoid(p[..., QKV + HV + H:].float()).to(BF)
    if update:
        o, ds = gdr.fused_recurrent_gated_delta_rule(q, k, v, g, beta, initial_state=ds,
                                                     use_qk_l2norm_in_kernel=True,
                                                     inplace_final_state=True)
    else:
        o, ds = gdr.chunk_gated_delta_rule(q, k, v, g, beta, initial_state=ds, output_final_state=True,
                                           use_qk_l2norm_in_kernel=True, cu_seqlens=cu,
                                           cu_seqlens_cpu=cu_cpu)
    return o.reshape(B, T, HV), cs, ds


CONV = {}


def w_conv(cs):
    return CONV["w"]


def layer8(w, xq, xs, res, cs, ds, update, see, cu=None, cu_cpu=None):
    """One layer in 8 bits: from its quantised input to the next one's."""
    p = see("p", gdr.int8_matmul(xq, xs, *w["qin"]), x=xq, xs=xs)
    o, cs, ds = mixer(p, cs, ds, update, cu, cu_cpu)
    z = p[..., QKV:QKV + HV]                                   # a slice, read in place
    gq, gs = gdr.gated_rms_norm_quant(o, z, w["nv"], EPS, V, format="int8")
    see("g", (gq, gs), o=o, z=z)
    b = see("b", gdr.int8_matmul(gq, gs, *w["qout"]), x=gq, xs=gs)
    q, s, h = gdr.sandwich_rms_norm_quant(b, res, w["post"], w["pre"], None, w["scale"], eps=EPS,
                                          format="int8")
    see("s", (q, s, h), b=b, res=res)
    return q, s, h, cs, ds


def held8(w, name, out, t):
    """One operator's outputs against the reference of what it got."""
    if name in "pb":
        wq, ws = w["qin" if name == "p" else "qout"]
        x = t["x"].reshape(-1, t["x"].shape[-1])
        want, mag = bref.product(x, t["xs"].reshape(-1), wq, ws)
        ref.held(name, out.reshape(want.shape), want, mag, BF, PRODUCT)
    elif name == "g":
        r = bref.gated(t["o"], t["z"], w["nv"], EPS, V)
        bref.quantised(r["y"], *out, "int8", 0, SLACK)
    else:
        r = bref.sandwich(t["b"], t["res"], w["post"], w["pre"], EPS, None, w["scale"], h=out[2])
        ref.held("h", out[2], r["h"], r["hm"], F32, OUT)
        bref.quantised(r["y"], out[0], out[1], "int8", 0, SLACK)


def start(w, B, T, n, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    res = r(B, T, DM)
    q, s, _ = gdr.rms_norm_quant(res.to(BF), w["pre0"], EPS, format="int8")
    return q, s, res, torch.zeros(n, 3, QKV, device="cuda", dtype=BF), torch.zeros(n, H, K, V, device="cuda")


@pytest.mark.parametrize("B,T,lens", [(2, 150, None), (1, 333, [100, 0, 1, 232])])
def test_a_prompt_in_eight_bits(B, T, lens):
    """Two layers over dense and packed prompts."""
    n = B if lens is None else len(lens)
    cu_cpu = None if lens is None else torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    cu = None if cu_cpu is None else cu_cpu.cuda()
    w = eight(weights())
    CONV["w"] = w["cw"]
    seen = []

    def see(name, out, **t):
        seen.append((name, out, t))
        return out

    q, s, res, cs, ds = start(w, B, T, n, 1)
    for _ in range(2):
        q, s, res, _, _ = layer8(w, q, s, res, cs, ds, False, see, cu, cu_cpu)
    torch.cuda.synchronize()
    assert len(seen) == 8
    for name, out, t in seen:
        held8(w, name, out, t)


def test_decode_steps_in_a_graph():
    """One token of five sequences captured into a graph and replayed over six
    steps, the program's own work between the replays; every replay's
    operators are held against the reference, and its outputs equal the eager
    run's."""
    B = 5
    w = eight(weights(3))
    CONV["w"] = w["cw"]
    steps = [start(w, B, 1, B, 10 + i)[:3] for i in range(6)]
    _, _, _, cs, ds = start(w, B, 1, B, 2)
    eager, ecs, eds = [], cs.clone(), ds.clone()
    for q, s, res in steps:
        eager.append(layer8(w, q, s, res, ecs, eds, True, lambda name, out, **t: out)[:3])
    q, s, res = (v.clone() for v in steps[0])
    keep = cs.clone(), ds.clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        layer8(w, q, s, res, cs, ds, True, lambda name, out, **t: out)
    torch.cuda.current_stream().wait_stream(stream)
    seen = []

    def see(name, out, **t):
        seen.append((name, out, t))
        return out

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer8(w, q, s, res, cs, ds, True, see)
    cs.copy_(keep[0]), ds.copy_(keep[1])
    for i, step in enumerate(steps):
        for dst, src in zip((q, s, res), step):
            dst.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        for name, o, t in seen:
            held8(w, name, o, t)
        assert all(torch.equal(a, b) for a, b in zip(out[:3], eager[i])), i
        gdr.quantize_rows(w["win"])                            # the program's own work
    assert torch.equal(cs, ecs) and torch.equal(ds, eds)


def train_layer(w, x, res, gate, mid):
    """The same layer in bf16 under autograd, the block's output gated."""
    h0 = mid("h0", gdr.rms_norm(x, w["pre0"], EPS))
    p = mid("p", h0 @ w["win"].t())
    B, T = p.shape[:2]
    c, _ = gdr.causal_conv1d(p[..., :QKV], w["cw"])
    q, k, v = (c[..., i:j].unflatten(-1, (H, -1)) for i, j in ((0, H * K), (H * K, 2 * H * K), (2 * H * K, QKV)))
    g = -torch.nn.functional.softplus(p[..., QKV + HV:QKV + HV + H].float())
    beta = torch.sigmoid(p[..., QKV + HV + H:])
    o, _ = gdr.chunk_gated_delta_rule(q, k, v, g, beta, use_qk_l2norm_in_kernel=True)
    o = mid("o", o.reshape(B, T, HV))
    z = mid("z", p[..., QKV:QKV + HV])
    u = mid("u", gdr.gated_rms_norm(o, z, w["nv"], EPS, V))
    b = mid("b", u @ w["wout"].t())
    return gdr.sandwich_rms_norm(b, res, w["post"], w["pre"], gate, w["scale"], "sigmoid", EPS)


@pytest.mark.parametrize("B,T", [(2, 150), (1, 700)])
def test_a_training_step(B, T):
    w = weights(5)
    g = torch.Generator().manual_seed(6)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    x, res, gate = r(B, T, DM).to(BF), r(B, T, DM), r(B, T, DM).to(BF)
    for t in list(w.values()) + [x, res, gate]:
        t.requires_grad_(True)
    m = {}

    def mid(name, t):
        t.retain_grad()
        m[name] = t
        return t

    y, h = train_layer(w, x, res, gate, mid)
    dy, dh = r(B, T, DM).to(BF), r(B, T, DM)
    torch.autograd.backward([y, h], [dy, dh])
    torch.cuda.synchronize()
    q = bref.sandwich(m["b"], res, w["post"], w["pre"], EPS, gate, w["scale"], "sigmoid", h, dy, dh)
    ref.held("h", h, q["h"], q["hm"], F32, OUT)
    ref.held("y", y, q["y"], q["y"].abs(), BF, OUT)
    for name, got, dt, slack in (("x", m["b"].grad, BF, SLACK), ("res", res.grad, F32, SLACK),
                                 ("gate", gate.grad, BF, SLACK), ("post", w["post"].grad, BF, SUM_SLACK),
                                 ("pre", w["pre"].grad, BF, SUM_SLACK),
                                 ("scale", w["scale"].grad, BF, SUM_SLACK)):
        ref.held("sandwich d" + name, got, q["d" + name], q["d" + name + "m"], dt, slack)
    q = bref.gated(m["o"], m["z"], w["nv"], EPS, V, dy=m["u"].grad)
    ref.held("u", m["u"], q["y"], q["y"].abs(), BF, OUT)
    ref.held("gated dx", m["o"].grad, q["dx"], q["dxm"], BF, SLACK)
    ref.held("gated dz", m["z"].grad, q["dz"], q["dzm"], BF, SLACK)
    ref.held("gated dw", w["nv"].grad, q["dw"], q["dwm"], BF, SUM_SLACK)
    # the projections' gradients have passed every operator: finite and there
    assert all(w[k].grad.isfinite().all() and w[k].grad.any() for k in ("win", "wout", "cw", "pre0"))


def gradients(t):
    """Forward and gradient forms of both norms, one after the other."""
    y, r = gdr.gated_rms_norm_fwd(t["x"], t["z"], t["w"], EPS, t["size"], t["first"])
    a = gdr.gated_rms_norm_bwd(t["dy"], t["x"], t["z"], t["w"], r, t["size"], t["first"])
    s = gdr.sandwich_rms_norm_fwd(y, t["res"], t["post"], t["pre"], t["z"], t["scale"])
    b = gdr.sandwich_rms_norm_bwd(t["dy"], t["res"], y, s[1], t["post"], t["pre"], s[2], s[3], t["z"],
                                  t["scale"])
    q = gdr.quantize_rows(s[0])
    p = gdr.int8_matmul(*q, t["wq"], t["ws"])
    return (y, r) + a + s + b + q + (p,)


def job(rows, D, size, shared, first, N, seed):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g).cuda()  # noqa: E731
    wq, ws = gdr.quantize_rows(r(N, D).to(BF))
    return dict(x=r(rows, D).to(BF), z=r(rows, D).to(BF), w=r(size if shared else D).to(BF), size=size,
                first=first, dy=r(rows, D).to(BF), res=r(rows, D), post=r(D), pre=r(D), scale=r(D), wq=wq,
                ws=ws)


JOBS = [(300, 512, 128, True, True, 700), (70, 1500, 300, True, False, 999), (1200, 1040, 65, True, True, 300),
        (33, 600, 600, False, False, 5000)]


@pytest.mark.parametrize("args", JOBS)
def test_captured_gradients(args):
    """Replays after the first too, with the program's own work and
    synchronizations between them; also while an eager graph of the same
    leaves lives."""
    t = job(*args, 1)
    x = t["x"].clone().requires_grad_(True)
    alive = gdr.gated_rms_norm(x, t["z"], t["w"], EPS, t["size"])
    t["x"] = x.detach()
    want = gradients(t)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        gradients(t)
    torch.cuda.current_stream().wait_stream(stream)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gradients(t)
    for _ in range(4):
        for o in out:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        gradients(t)
    alive.sum().backward()
    assert x.grad.isfinite().all()


def test_calls_at_once_on_two_streams():
    """Two jobs on streams of their own have the bits of the same jobs alone."""
    jobs = [job(*JOBS[i], 7 + i) for i in (0, 2)]
    for j in jobs:                                             # rows enough to overlap
        for k in ("x", "z", "dy", "res"):
            j[k] = j[k].repeat(20, 1)
    want = [gradients(j) for j in jobs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    got = [[], []]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(4):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(gradients(jobs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_python_refusals():
    t = job(4, 32, 32, True, True, 8, 1)
    x, z, w = t["x"], t["z"], t["w"]
    q, s = gdr.quantize_rows(x)
    y, r = gdr.gated_rms_norm_fwd(x, z, w)
    yy, h, rx, rh = gdr.sandwich_rms_norm_fwd(x, t["res"], t["post"], t["pre"])
    back = (t["dy"], None, x, h, t["post"], t["pre"], rx, rh)
    for call, name in [
        (lambda: gdr.gated_rms_norm(x, z[:2], w), "GDR_ERR_SHAPE"),
        (lambda: gdr.gated_rms_norm(x, z.half(), w), "GDR_ERR_DTYPE"),
        (lambda: gdr.gated_rms_norm(x, z, w[:16]), "GDR_ERR_SHAPE"),
        (lambda: gdr.gated_rms_norm(x, z, w, norm_group=5), "GDR_ERR_SHAPE"),
        (lambda: gdr.gated_rms_norm(x, z, w, norm_group=4), "GDR_ERR_SHAPE"),
        (lambda: gdr.gated_rms_norm(x, z, w.half()), "GDR_ERR_DTYPE"),
        (lambda: gdr.gated_rms_norm(x, z.cpu(), w), "GDR_ERR_DEVICE"),
        (lambda: gdr.gated_rms_norm(x, z, w, eps=-1.0), "GDR_ERR_ARG"),
        (lambda: gdr.gated_rms_norm(x[:0], z[:0], w), "GDR_ERR_SHAPE"),
        (lambda: gdr.gated_rms_norm_bwd(t["dy"][:2], x, z, w, r), "GDR_ERR_SHAPE"),
        (lambda: gdr.gated_rms_norm_bwd(t["dy"], x, z, w, r[:2]), "GDR_ERR_SHAPE"),
        (lambda: gdr.gated_rms_norm_bwd(t["dy"], x, z, w, r, norm_group=16), "GDR_ERR_SHAPE"),
        (lambda: gdr.sandwich_rms_norm(x, t["res"][:2], t["post"], t["pre"]), "GDR_ERR_SHAPE"),
        (lambda: gdr.sandwich_rms_norm(x, t["res"].half(), t["post"], t["pre"]), "GDR_ERR_DTYPE"),
        (lambda: gdr.sandwich_rms_norm(x, t["res"], w, t["pre"]), "GDR_ERR_DTYPE"),
        (lambda: gdr.sandwich_rms_norm(x, t["res"], None, t["pre"], gate=z[:, :8]), "GDR_ERR_SHAPE"),
        (lambda: gdr.sandwich_rms_norm(x, t["res"], None, t["pre"], residual_scale=float("nan")),
         "GDR_ERR_ARG"),
        (lambda: gdr.sandwich_rms_norm_bwd(*back[:6], None, rh), "GDR_ERR_ARG"),
        (lambda: gdr.sandwich_rms_norm_bwd(t["dy"], h[:2], *back[2:]), "GDR_ERR_SHAPE"),
        (lambda: gdr.sandwich_rms_norm_bwd(t["dy"], None, x, h.half(), *back[4:]), "GDR_ERR_DTYPE"),
        (lambda: gdr.quantize_rows(x[:, :0]), "GDR_ERR_SHAPE"),
        (lambda: gdr.quantize_rows(x.double()), "GDR_ERR_DTYPE"),
        (lambda: gdr.int8_matmul(q, s[:2], t["wq"], t["ws"]), "GDR_ERR_SHAPE"),
        (lambda: gdr.int8_matmul(q, s.half(), t["wq"], t["ws"]), "GDR_ERR_DTYPE"),
        (lambda: gdr.int8_matmul(q, s, t["wq"][:, :16], t["ws"]), "GDR_ERR_SHAPE"),
        (lambda: gdr.int8_matmul(q, s, t["wq"], t["ws"][:3]), "GDR_ERR_SHAPE"),
        (lambda: gdr.int8_matmul(q, s, t["wq"].float(), t["ws"]), "GDR_ERR_DTYPE"),
        (lambda: gdr.int8_matmul(q, s, t["wq"], t["ws"], w[:8].half()), "GDR_ERR_DTYPE"),
        (lambda: gdr.int8_matmul(q[:0], s[:0], t["wq"], t["ws"]), "GDR_ERR_SHAPE"),
        (lambda: gdr.int8_matmul(q, s, t["wq"].cpu(), t["ws"]), "GDR_ERR_DEVICE"),
    ]:
        with pytest.raises(gdr.GdrError) as e:
            call()
        assert e.value.name == name, e.value
