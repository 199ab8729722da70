"""The selective scan in fp16 where its scores leave fp16's range: step sizes
and gradients that make them tiny, gradients and inputs that make them pass
65504, while inputs and results are ordinary fp16 values (needs an MI355X).

Tolerances.  As in the scan's own tests: the products in a chunk round one
operand to the type, half a step of the magnitudes that the reference adds up,
and a quarter for the start state's rounding and the rest; states are within
2^-15 of theirs, dD within 2^-17; the gradients of step sizes, bias and rates
are within 2^-13 and 2^-10 of the roots of summed squares."""
import pytest
import torch

import _layer_ref as ref
import gated_delta_rule_66_amd as gdr
import test_gpu_layer_scan as scan
import test_gpu_layer_scan_decays as decays

pytestmark = pytest.mark.gpu
HF, F32 = torch.float16, torch.float32

# how large the values are: (x, B and C, step sizes, dy)
SIZES = {
    "tiny_steps": (64, 1 / 8, 1e-5, 8),          # scores of 1e-6
    "tiny_gradients": (1, 16, 1e-3, 1e-4),       # (dy . x) dt of 1e-6
    "small_loss": (1, 4, 1 / 32, 1e-4),
    "scaled_loss": (8, 1 / 256, 1, 4096),        # (dy . x) dt of 3e5
    "large_scores": (1, 64, 1e-3, 1 / 64),       # C . B of 3e4 and more
    "large_steps": (1 / 256, 64, 8, 1 / 1024),   # C . B dt of 3e5
    "ordinary": (1, 1, 1 / 16, 1),
}
SHAPES = [(1, 150, 4, 2, 64, 64), (2, 70, 3, 1, 64, 128), (1, 130, 2, 2, 128, 64), (1, 140, 4, 2, 128, 128),
          (1, 100, 2, 2, 128, 128), (1, 90, 6, 2, 128, 64)]


@pytest.mark.parametrize("sizes", list(SIZES))
@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_scores_out_of_range(shape, sizes):
    B, T, H, G, K, V = shape
    sx, sb, sd, sy = SIZES[sizes]
    g = torch.Generator().manual_seed(T)
    r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    t = dict(x=(r(B, T, H, V) * sx).to(HF), B=(r(B, T, G, K) * sb).to(HF), C=(r(B, T, G, K) * sb).to(HF),
             dt=(0.5 + torch.rand(B, T, H, generator=g)) * sd, A_log=torch.log(r(H).abs() / (8 * sd) + 1e-3),
             D=None, dt_bias=None, state=None, cu=None, dy=(r(B, T, H, V) * sy).to(HF), dlast=None)
    d = scan.dev(t)
    y, last = gdr.chunk_selective_scan_fwd(*scan.args(d), False, None, True)
    got = gdr.chunk_selective_scan_bwd(*scan.args(d)[:5], d["dy"], None, None, False)
    want = ref.scan(t["x"], t["dt"], t["A_log"], t["B"], t["C"], None, None, False, None, None, t["dy"])
    for n in ("y", "dx", "dB", "dC"):            # the case is one that fp16 results can hold
        top = want[n].abs().max()
        assert 2.0 ** -14 < top < 60000, (n, float(top))
    slack = 1.25 * ref.half_step(HF)
    ref.held("y", y, want["y"], want["ym"], HF, slack)
    ref.held("state", last, want["last"], want["lastm"], F32, scan.STATE_SLACK)
    for n, v in zip(scan.GRADS, got):
        if n in ("dx", "dB", "dC"):
            print(n, "%.2e" % float((ref.d(v) - want[n]).norm() / want[n].norm()))
            ref.held(n, v, want[n], want[n + "m"], HF, slack)
    decays.check(got, decays.reference(t, False), t)
    y2, last2 = gdr.fused_recurrent_selective_scan(*scan.args(d), False, None, True)
    ref.held("y", y2, want["y"], want["ym"], HF, slack)


def test_infinities_and_nans_are_not_lost():
    """A score tile without a finite largest value is left unscaled."""
    t = scan.dev(scan.make(1, 100, 2, 1, 64, 64, HF, state=False))
    t["x"][0, 70, 0, 3] = float("inf")
    t["x"][0, 80, 1, 5] = float("nan")
    y, last = gdr.chunk_selective_scan_fwd(*scan.args(t), True, None, True)
    assert not y[0, 70:, 0, 3].isfinite().any() and y[0, 80:, 1, 5].isnan().all()
    assert y[0, :64].isfinite().all()
    assert not last[0, 0, :, 3].isfinite().any() and last[0, 1, :, 5].isnan().all()
