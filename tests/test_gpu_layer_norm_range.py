"""The RMS norm of rows whose squares leave fp32's range (needs an MI355X).

The row's statistic is formed in 64 bits and rounded once to fp32, the outputs
are two fp32 products and one rounding to the type: 2^-22 of the value next to
the type's half step.  The gradient's row mean adds up to 64 + 16 fp32 terms in
a row: 2^-17 of the magnitudes, as where the squares stay in range."""
import pytest
import torch

import _layer_ref as ref
import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("scale,eps", [(2.0 ** 70, 1e-6), (2.0 ** 110, 1e-6), (2.0 ** -80, 0.0),
                                       (2.0 ** -100, 0.0), (1.0, 0.0)])
@pytest.mark.parametrize("rows,D", [(3, 45), (2, 1000), (2, 4096), (2, 20000), (2, 5)])
def test_rows_out_of_the_range_of_fp32_squares(rows, D, scale, eps, dtype):
    g = torch.Generator().manual_seed(D)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    x, w, dy = (r(rows, D) * scale).to(dtype), 1 + r(D) / 4, r(rows, D).to(dtype)
    y, _, rstd = gdr.rms_norm_fwd(x.cuda(), w.cuda(), eps)
    want = ref.norm(x, w, eps, dy=dy)
    ref.held("y", y, want["y"], want["y"].abs(), dtype, 2.0 ** -22)
    dx, _, dw = gdr.rms_norm_bwd(dy.cuda(), x.cuda(), w.cuda(), rstd)
    if scale >= 1:      # below, the true dx is past fp32's range or close to it
        ref.held("dx", dx, want["dx"], want["dxm"], dtype, 2.0 ** -17)
    ref.held("dw", dw, want["dw"], want["dwm"], F32, 2.0 ** -15)
    q, s, _ = gdr.rms_norm_quant(x.cuda(), w.cuda(), eps, format="int8")
    top = want["y"].abs().amax(-1, keepdim=True) / 127
    assert ((s.cpu().double() - top).abs() <= 2.0 ** -21 * top).all()
