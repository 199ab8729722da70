"""A mixer layer's training step: the gradients of the decay rates and the step
sizes' bias, which the scan and the delta rule share (needs an MI355X).  The
scan's part is what is left after the delta rule's, taken from a run of the
delta rule alone; it is held against the 64-bit recurrence on the tensors that
the scan got, with the bars of the scan's own tests (2^-10 of the root of the
summed squares) and the rounding of the two parts' fp32 sum."""
import pytest
import torch

import gated_delta_rule_66_amd as gdr
import test_gpu_layer_scan_decays as decays
import test_gpu_layer_together as whole

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("B,T,lens", [(2, 150, None), (1, 333, [100, 0, 1, 232]), (1, 1400, None)])
def test_shared_decay_parameters(B, T, lens):
    n = B if lens is None else len(lens)
    cu_cpu = None if lens is None else torch.tensor([0] + lens).cumsum(0).to(torch.int32)
    cu = None if cu_cpu is None else cu_cpu.cuda()
    w, t = whole.weights(), whole.inputs(B, T, n)
    for q in w.values():
        q.requires_grad_(True)
    m = {}

    def mid(name, v):
        v.retain_grad()
        m[name] = v
        return v

    out, h, cs, ss = whole.layer(w, t, cu, cu_cpu, mid)
    gen = torch.Generator().manual_seed(9)
    dout = torch.randn(out.shape, generator=gen).to(torch.bfloat16).cuda()
    dss = torch.randn(ss.shape, generator=gen).cuda()
    torch.autograd.backward([out, ss], [dout, dss])

    x, b, k, dt = whole.split(m["c"].detach(), m["p"][..., whole.XBC:].detach())
    A, bias = (w[v].detach().clone().requires_grad_(True) for v in ("A_log", "dt_bias"))
    o, _ = gdr.chunk_gated_delta_rule(k, b, x, dt.float(), torch.full_like(dt, 0.5),
                                      use_qk_l2norm_in_kernel=True, use_gate_in_kernel=True, A_log=A,
                                      dt_bias=bias, cu_seqlens=cu, cu_seqlens_cpu=cu_cpu)
    assert torch.equal(o, m["o"])
    o.backward(m["o"].grad)

    s = dict(x=x, dt=dt.contiguous(), A_log=w["A_log"], B=b, C=k, D=w["D"], dt_bias=w["dt_bias"], state=t["ss"],
             cu=cu_cpu, dy=m["s"].grad, dlast=dss)
    r = decays.reference(s, True)
    for name, got, other, want, size in (("dA", w["A_log"].grad, A.grad, r["dA"], r["dA_size"]),
                                         ("dbias", w["dt_bias"].grad, bias.grad, r["dbias"], r["ddt_size"])):
        err = (got.double() - other.double() - want).abs()
        bar = 2.0 ** -10 * size + 2.0 ** -23 * (got.abs() + other.abs()).double()
        print(name, "%.2g of its bar, which is %.2g of the gradient" % (float((err / bar).max()),
                                                                      float(bar.norm() / want.norm())))
        assert (err <= bar).all(), (name, err / bar)
        assert bar.norm() < 0.02 * want.norm(), name
