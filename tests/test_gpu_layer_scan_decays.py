"""The selective scan's gradients of the step sizes, their bias and the decay
rates against the token recurrence in 64 bits, relative to the gradients
themselves (needs an MI355X).

Tolerances.  The log decay's gradient dg_t is formed from fp32 sums over the
pairs of tokens that t lies between.  Each of the sums' terms is within 2^-18
of itself (the 16-bit pair that stands for a state; exponentials and fp32 sums
are finer), its error of either sign, and at most 512 tokens' errors are added
up before the chain begins anew.  A token's dg is then off by the root of 512
of them, 2^-13.5, next to sums of its own size: 2^-13 of the root of the summed
squares of a head's terms.  dA_log adds g_t dg_t, and the errors of 512
neighbours are one another's: 512 / 2 times 2^-18, 2^-9, for the root of the
summed squares of g_t dg_t if every token's error has one sign, half that for
a random walk, 2^-10; the step sizes' bias in the same way.  What is stored in
16 bits adds half a step.  That the bars are far below the gradients is checked
as well."""
import pytest
import torch

import _layer_ref as ref
import gated_delta_rule_66_amd as gdr
from test_gpu_layer_scan import CASES, MORE, args, dev, make

pytestmark = pytest.mark.gpu
BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def reference(t, softplus, heads=None):
    """dt's, dt_bias's and A_log's gradients and the sizes their errors scale
    with, of the given heads (whole groups), all sequences side by side."""
    H, G = t["x"].shape[2], t["B"].shape[2]
    heads = range(H) if heads is None else heads
    R = H // G
    hs = torch.tensor(list(heads), device="cuda")
    dd = lambda v: None if v is None else v.detach().cuda().double()  # noqa: E731
    pick = lambda k, dim: None if t[k] is None else dd(t[k].index_select(dim, hs.to(t[k].device)))  # noqa: E731
    x, dy, raw = pick("x", 2), pick("dy", 2), pick("dt", 2)
    A_log, bias, h0, dlast = pick("A_log", 0), pick("dt_bias", 0), pick("state", 1), pick("dlast", 1)
    grp = (hs // R).to(t["B"].device)
    Bm, Cm = dd(t["B"].index_select(2, grp)), dd(t["C"].index_select(2, grp))
    z = raw if bias is None else raw + bias
    step = torch.nn.functional.softplus(z, threshold=1e9) if softplus else z
    dz = torch.sigmoid(z) if softplus else torch.ones_like(z)
    spans = ref.spans(t["x"], t["cu"])
    n, L = len(spans), max(b - a for _, a, b, _ in spans)

    def gather(v):
        out = v.new_zeros((n, L) + v.shape[2:])
        for row, a, b, i in spans:
            out[i, :b - a] = v[row, a:b]
        return out

    xs, bs, cs, ys, st, dzs = (gather(v) for v in (x, Bm, Cm, dy, step, dz))
    rate = -torch.exp(A_log)
    g = rate * st
    S = x.new_zeros(n, len(hs), Bm.shape[3], x.shape[3]) if h0 is None else h0.clone()
    kept = []
    for i in range(L):
        kept.append(S)
        S = torch.exp(g[:, i])[..., None, None] * S + \
            (st[:, i, :, None] * bs[:, i])[..., :, None] * xs[:, i][..., None, :]
    P = torch.zeros_like(S) if dlast is None else dlast.clone()
    dg, q = torch.zeros_like(st), torch.zeros_like(st)
    for i in reversed(range(L)):
        P = P + cs[:, i][..., :, None] * ys[:, i][..., None, :]
        e = torch.exp(g[:, i])
        dg[:, i] = e * (kept.pop() * P).sum((-1, -2))
        q[:, i] = ((P * xs[:, i][..., None, :]).sum(-1) * bs[:, i]).sum(-1)
        P = e[..., None, None] * P
    live = torch.zeros(n, L, 1, dtype=torch.bool, device="cuda")
    for _, a, b, i in spans:
        live[i, :b - a] = True
    dg, q = dg * live, q * live
    ddt = (rate * dg + q) * dzs
    size = ((rate * dg).abs() + q.abs()) * dzs
    back = torch.cat([ddt[i, :b - a] for _, a, b, i in spans])
    return dict(ddt=back, ddt_size=size.square().sum((0, 1)).sqrt(),
                dbias=ddt.sum((0, 1)), dA=(g * dg).sum((0, 1)),
                dA_size=(g * dg).square().sum((0, 1)).sqrt())


def check(got, r, t, heads=None):
    pick = (lambda v, dim: v) if heads is None else \
        (lambda v, dim: v.index_select(dim, torch.tensor(list(heads), device=v.device)))  # noqa: E731
    _, ddt, dA, _, _, _, dbias, _ = got
    ddt = pick(ddt, 2).flatten(0, 1).double()
    half = ref.half_step
    err = (ddt - r["ddt"]).square().sum(0).sqrt()
    bar = 2.0 ** -13 * r["ddt_size"] + half(t["dt"].dtype) * r["ddt"].square().sum(0).sqrt()
    print("ddt %.2g of its bar" % float((err / bar).max()))
    assert (err <= bar).all()
    pt = t["A_log"].dtype
    for name, v, want, size in (("dA", dA, r["dA"], r["dA_size"]), ("dbias", dbias, r["dbias"], r["ddt_size"])):
        if v is None:
            continue
        err = (pick(v, 0).double() - want).abs()
        bar = 2.0 ** -10 * size + half(pt) * want.abs()
        print(name, "%.2g of its bar, which is %.2g of the gradient" % (float((err / bar).max()),
                                                                      float(bar.norm() / want.norm())))
        assert (err <= bar).all(), (name, err / bar)
        if len(want) > 2:
            assert bar.norm() < 0.02 * want.norm(), name


def run(t, softplus, **kw):
    """Through autograd, with the states that the forward keeps."""
    g = dev(t)
    keys = ("x", "dt", "A_log", "B", "C", "D", "dt_bias", "state")
    leaves = [g[k].requires_grad_(True) for k in keys if g[k] is not None]
    y, last = gdr.chunk_selective_scan(*args(g), softplus, g["state"], True, g["cu"],
                                       None if t["cu"] is None else t["cu"].cpu(), **kw)
    got = iter(torch.autograd.grad([y, last], leaves, [g["dy"], g["dlast"]]))
    return [next(got) if g[k] is not None else None for k in keys]


SHORT = {**CASES, **MORE,
         "uncut_and_cut": ((1, 3700, 2, 2, 64, 64, BF), dict(lens=[0, 1100, 2600], fast=True)),
         "half_wide": ((1, 200, 4, 2, 128, 128, HF), dict(dt_dtype=F32)),
         "one_head_wide": ((1, 150, 3, 3, 128, 128, BF), {}),
         "one_head_half": ((2, 190, 2, 2, 128, 64, HF), {}),
         "one_head_narrow": ((2, 130, 3, 3, 64, 64, BF), dict(fast=True)),
         "one_head_64_128": ((1, 333, 2, 2, 64, 128, BF), dict(p_dtype=BF))}


@pytest.mark.parametrize("name", list(SHORT))
def test_step_and_decay_gradients(name):
    shape, kw = SHORT[name]
    t = make(*shape, **kw)
    sp = kw.get("softplus", True)
    check(run(t, sp), reference(t, sp), t)


# as many workgroups as the chip runs at once: no sequence is cut, so the chain
# runs along the whole of it.  (A_log, dt_bias): log decays of some -13 and -23 a
# token, of -0.5, and of -0.03 (memory over chunks).
@pytest.mark.parametrize("rate,bias", [(16, 0), (16, 1), (16, -4), (1, -4), (4, -2)])
@pytest.mark.parametrize("B,T,H,G,K,V", [(2, 4096, 256, 128, 64, 64), (4, 1500, 64, 64, 128, 64),
                                         (2, 2100, 256, 128, 128, 128)])
def test_long_uncut_segments(rate, bias, B, T, H, G, K, V):
    gen = torch.Generator(device="cuda").manual_seed(rate + T)
    r = lambda *s, dt=BF: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    t = dict(x=r(B, T, H, V), B=r(B, T, G, K), C=r(B, T, G, K), dt=r(B, T, H, dt=F32), D=None, cu=None, state=None,
             A_log=torch.full((H,), float(rate), device="cuda").log(),
             dt_bias=torch.full((H,), float(bias), device="cuda"), dy=r(B, T, H, V), dlast=None)
    got = gdr.chunk_selective_scan_bwd(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["dy"], None,
                                       t["dt_bias"], True, None)
    heads = [0, 1, H // 2, H // 2 + 1, H - 2, H - 1]
    check(got, reference(t, True, heads), t, heads)


# sequences in one run of up to 33 chunks each, then sequences cut into segments
# of more than 512 tokens, so that kept states and segment ends take turns
@pytest.mark.parametrize("lens,H,G,K,V", [([700, 1, 1300, 64, 0, 2100, 1030], 128, 64, 64, 64),
                                          ([9000, 300, 7084], 64, 16, 64, 64),
                                          ([0, 513, 1025, 512, 1024], 256, 128, 128, 128)])
@pytest.mark.parametrize("rate,bias", [(16, 0), (1, -4)])
def test_long_packed_sequences(lens, H, G, K, V, rate, bias):
    gen = torch.Generator(device="cuda").manual_seed(rate + H)
    r = lambda *s, dt=BF: torch.randn(*s, generator=gen, device="cuda").to(dt)  # noqa: E731
    T, n = sum(lens), len(lens)
    cu = torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    t = dict(x=r(1, T, H, V), B=r(1, T, G, K), C=r(1, T, G, K), dt=r(1, T, H, dt=F32), D=None,
             cu=cu.cuda(), state=r(n, H, K, V, dt=F32), A_log=torch.full((H,), float(rate), device="cuda").log(),
             dt_bias=torch.full((H,), float(bias), device="cuda"), dy=r(1, T, H, V),
             dlast=r(n, H, K, V, dt=F32))
    heads = [0, 1, H // 2, H // 2 + 1, H - 2, H - 1]
    want = reference(t, True, heads)
    got = run(t, True)
    check(got, want, t, heads)
    again = run(t, True, recompute_states=True)     # the same cut, the states formed anew
    assert torch.equal(got[1], again[1]) and torch.equal(got[2], again[2])
