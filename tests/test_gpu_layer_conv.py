"""The short causal convolution on the GPU against a plain 64-bit form (needs
an MI355X).

Tolerances: an output is one rounding to its type plus fp32 arithmetic.  A sum
of k products in fp32 is off by at most (k + 1) 2^-24 of the sum of the
products' magnitudes (here k <= 5 with the bias); the exponential and the
reciprocal of the sigmoid add (|z| + 4) 2^-23 relative.  2^-19 of the
magnitudes that the reference returns covers both.  The weight gradient sums
up to 64 tokens per run, 64 runs and 512 blocks one after the other: (64 + 64
+ 128) 2^-24 = 2^-16."""
import pytest
import torch

import _layer_ref as ref
import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
SLACK, SUM_SLACK = 2.0 ** -19, 2.0 ** -16

BF, HF, F32 = torch.bfloat16, torch.float16, torch.float32


def make(B, T, D, W, dtype, wdtype=None, bias=True, state=True, lens=None, seed=0, train=True):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    n = B if lens is None else len(lens)
    wd = wdtype or dtype
    cu = None if lens is None else torch.tensor([0] + list(lens)).cumsum(0).to(torch.int32)
    t = dict(x=r(B, T, D).to(dtype), w=(r(D, W) / 2).to(wd), bias=r(D).to(wd) if bias else None,
             state=r(n, W - 1, D).to(dtype) if state else None, cu=cu)
    if train:
        t.update(dy=r(B, T, D).to(dtype), dlast=r(n, W - 1, D).to(dtype))
    return t


def dev(t):
    return {k: (v.cuda() if isinstance(v, torch.Tensor) else v) for k, v in t.items()}


CASES = {
    # name: (B, T, D, W, dtype, weight dtype, bias, state, lens, silu)
    "one_token": (1, 1, 8, 4, BF, None, True, True, None, True),
    "two_tokens": (3, 2, 1, 4, F32, None, True, True, None, True),
    "odd_width": (2, 37, 45, 3, HF, F32, False, True, None, True),
    "no_state": (2, 65, 64, 4, BF, F32, True, False, None, True),
    "linear_w2": (1, 130, 100, 2, F32, None, True, True, None, False),
    "wide": (1, 70, 1032, 4, BF, None, True, True, None, True),
    "packed": (1, 214, 72, 4, HF, None, True, True, [1, 0, 2, 3, 128, 0, 80, 0], True),
    "packed_first_empty": (1, 66, 520, 3, BF, None, False, False, [0, 0, 66], True),
    "packed_one_token_each": (1, 9, 16, 4, F32, None, True, True, [1] * 9, True),
    "long": (1, 5000, 24, 4, BF, None, True, False, None, True),
}


@pytest.mark.parametrize("name", list(CASES))
def test_forward_and_gradients(name):
    B, T, D, W, dtype, wd, bias, state, lens, silu = CASES[name]
    t = make(B, T, D, W, dtype, wd, bias, state, lens)
    g = dev(t)
    act = "silu" if silu else None
    cu = dict(cu_seqlens=g["cu"], cu_seqlens_cpu=t["cu"])
    leaves = [g[k].requires_grad_(True) for k in ("x", "w", "bias", "state") if g[k] is not None]
    y, last = gdr.causal_conv1d(g["x"], g["w"], g["bias"], act, g["state"], True, **cu)
    grads = torch.autograd.grad([y, last], leaves, [g["dy"], g["dlast"]])
    torch.cuda.synchronize()
    r = ref.conv(t["x"], t["w"], t["bias"], silu, t["state"], t["cu"], t["dy"], t["dlast"])
    ref.held("y", y, *r["y"], dtype, SLACK)
    assert torch.equal(last.cpu().double(), r["last"][0])       # copies of inputs
    names = ["dx", "dw"] + (["db"] if bias else []) + (["ds"] if state else [])
    for k, v in zip(names, grads):
        ref.held(k, v, *r[k], v.dtype, SUM_SLACK if k in ("dw", "db") else SLACK)


@pytest.mark.parametrize("dtype,W,D", [(BF, 4, 12301), (HF, 3, 12296), (F32, 2, 6151)])
def test_large_gradients(dtype, W, D):
    """Sizes whose gradient takes the wide form; the reference on some channels
    (they are independent), the last ones among them."""
    B, T = 2, 4100 if dtype != F32 else 4200
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s, dt=dtype: torch.randn(*s, generator=g, device="cuda").to(dt)  # noqa: E731
    t = dict(x=r(B, T, D), w=r(D, W, dt=F32), b=r(D, dt=F32), s=r(B, W - 1, D), dy=r(B, T, D),
             ds=r(B, W - 1, D))
    dx, dw, db, ds = gdr.causal_conv1d_bwd(t["x"], t["w"], t["b"], t["dy"], t["ds"], "silu", t["s"])
    pick = torch.tensor(list(range(5)) + [D // 2, D // 2 + 1] + list(range(D - 9, D)))
    c = lambda v, dim: v.index_select(dim, pick.cuda())  # noqa: E731
    want = ref.conv(c(t["x"], 2), c(t["w"], 0), c(t["b"], 0), True, c(t["s"], 2), None, c(t["dy"], 2),
                    c(t["ds"], 2))
    for name, got, dt in (("dx", c(dx, 2), dtype), ("dw", c(dw, 0), F32), ("db", c(db, 0), F32),
                          ("ds", c(ds, 2), dtype)):
        ref.held(name, got, *want[name], dt, SUM_SLACK if name in ("dw", "db") else SLACK)


def test_a_slice_of_a_wider_tensor_is_read_in_place():
    g = torch.Generator().manual_seed(3)
    wide = torch.randn(2, 50, 77, generator=g).to(BF).cuda()
    x = wide[:, :, 5:46]
    t = make(1, 1, 41, 4, BF, train=False, state=False)
    y, _ = gdr.causal_conv1d_fwd(x, t["w"].cuda(), t["bias"].cuda())
    y2, _ = gdr.causal_conv1d_fwd(x.contiguous(), t["w"].cuda(), t["bias"].cuda())
    assert torch.equal(y, y2)
    assert not x.is_contiguous()
    swapped = wide.transpose(0, 1)[:, :, :41]                   # another order of tokens: copied
    y3, _ = gdr.causal_conv1d_fwd(swapped, t["w"].cuda(), t["bias"].cuda())
    y4, _ = gdr.causal_conv1d_fwd(swapped.contiguous(), t["w"].cuda(), t["bias"].cuda())
    assert torch.equal(y3, y4)


@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_steps_continue_a_prompt(W, dtype):
    """A prompt, then tokens one and three at a time on its state: the same
    bits as the whole sequence at once."""
    t = dev(make(3, 20, 43, W, dtype, train=False, state=False))
    whole, last = gdr.causal_conv1d_fwd(t["x"], t["w"], t["bias"])
    y, st = gdr.causal_conv1d_fwd(t["x"][:, :13], t["w"], t["bias"])
    parts = [y]
    for a, b in ((13, 14), (14, 17), (17, 20)):
        parts.append(gdr.causal_conv1d_update(t["x"][:, a:b], st, t["w"], t["bias"]))
    assert torch.equal(torch.cat(parts, 1), whole)
    assert torch.equal(st, last)
    one = gdr.causal_conv1d_update(t["x"][:, 0], st, t["w"], t["bias"])
    assert one.shape == (3, 43)


def test_gradient_against_differences():
    """Along random directions in fp32: the change of a fixed weighting of the
    outputs.  The central difference is off by the curvature, h^2/6 of the
    third derivative, and by 2^-23 of the outputs over h; with h = 2^-7 both
    are below 1e-4 of the sum of magnitudes' root."""
    t = dev(make(2, 40, 24, 4, F32, seed=5))
    keys = ("x", "w", "bias", "state")
    gen = torch.Generator().manual_seed(9)
    grads = gdr.causal_conv1d_bwd(t["x"], t["w"], t["bias"], t["dy"], t["dlast"],
                                  initial_state=t["state"])
    h = 2.0 ** -7
    for k, g in zip(keys, grads):
        v = torch.randn(t[k].shape, generator=gen).cuda()

        def value(s):
            q = dict(t)
            q[k] = t[k] + s * v
            y, last = gdr.causal_conv1d_fwd(q["x"], q["w"], q["bias"], "silu", q["state"])
            return (y.double() * t["dy"]).sum() + (last.double() * t["dlast"]).sum()

        diff = (value(h) - value(-h)) / (2 * h)
        want = (g.double() * v).sum()
        scale = (g.double() * v).square().sum().sqrt()
        assert abs(diff - want) <= 1e-3 * scale, (k, float(diff), float(want))


def test_infinities_and_nans_stay_in_their_window():
    t = dev(make(1, 30, 16, 4, BF, train=False, state=False))
    clean, _ = gdr.causal_conv1d_fwd(t["x"], t["w"], t["bias"])
    x = t["x"].clone()
    x[0, 10, 3] = float("nan")
    x[0, 20, 5] = float("inf")
    y, _ = gdr.causal_conv1d_fwd(x, t["w"], t["bias"])
    changed = torch.zeros_like(y, dtype=torch.bool)
    changed[0, 10:14, 3] = True
    changed[0, 20:24, 5] = True
    assert torch.equal(y[~changed], clean[~changed])
    assert y[0, 10:14, 3].isnan().all()


def test_captured_and_replayed():
    """A training step in a graph, replayed with eager work in between."""
    t = dev(make(2, 90, 40, 4, BF))
    args = (t["x"], t["w"], t["bias"])

    def step():
        y, last = gdr.causal_conv1d_fwd(*args, "silu", t["state"])
        return (y, last) + gdr.causal_conv1d_bwd(*args, t["dy"], t["dlast"], "silu", t["state"])

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
    t = dev(make(2, 8, 16, 4, BF))
    x, w = t["x"], t["w"]
    for call, name in [
        (lambda: gdr.causal_conv1d(x, w[:8]), "GDR_ERR_SHAPE"),
        (lambda: gdr.causal_conv1d(x, w.half()), "GDR_ERR_DTYPE"),
        (lambda: gdr.causal_conv1d(x, w, t["bias"].float()), "GDR_ERR_DTYPE"),
        (lambda: gdr.causal_conv1d(x, w, initial_state=t["state"][:1]), "GDR_ERR_SHAPE"),
        (lambda: gdr.causal_conv1d(x, w, activation="gelu"), "GDR_ERR_ARG"),
        (lambda: gdr.causal_conv1d(x.double(), w), "GDR_ERR_DTYPE"),
        (lambda: gdr.causal_conv1d(x[0], w), "GDR_ERR_SHAPE"),
        (lambda: gdr.causal_conv1d(x, w, cu_seqlens=torch.tensor([0, 8])), "GDR_ERR_VARLEN"),
        (lambda: gdr.causal_conv1d_update(x, t["state"].transpose(0, 1), w), "GDR_ERR_ARG"),
        (lambda: gdr.causal_conv1d_update(x, t["state"].cpu(), w), "GDR_ERR_DEVICE"),
    ]:
        with pytest.raises(gdr.GdrError) as e:
            call()
        assert e.value.name == name
