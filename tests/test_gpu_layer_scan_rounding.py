"""Where the selective scan's 16-bit outputs round once (needs an MI355X).

dB and dC inside a chunk: the scores that make them are a pair of 16-bit values,
off by 2^-17 of each score with bf16 (16 bits and a sign) and less with fp16, so
without states before or behind the chunk only the output's own rounding is
left, next to fp32 sums: 2^-16 of the magnitudes.  y and dx of a single token:
the score of a token with itself enters in fp32, sums of K = 64 or 128 products
and a few roundings: 2^-20 of the magnitudes, softplus and exponential included.
Longer sequences keep one rounded operand in y and dx and in what passes through
the state."""
import pytest
import torch

import _layer_ref as ref
import gated_delta_rule_66_amd as gdr
import test_gpu_layer_scan as scan

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16
FORMS = [(4, 2, 64, 64), (3, 1, 64, 128), (2, 2, 128, 64), (4, 2, 128, 128), (2, 2, 128, 128), (8, 1, 128, 64),
         (2, 2, 64, 64), (2, 2, 64, 128)]


def run(T, form, dtype, lens=None, **kw):
    H, G, K, V = form
    t = scan.make(1, T, H, G, K, V, dtype, state=False, lens=lens, **kw)
    t["dlast"] = None
    g = scan.dev(t)
    cu = t["cu"]
    y, _ = gdr.chunk_selective_scan_fwd(*scan.args(g), True, None, False, g["cu"], cu)
    got = gdr.chunk_selective_scan_bwd(*scan.args(g)[:5], g["dy"], g["D"], g["dt_bias"], True, None, None,
                                       g["cu"], cu)
    r = ref.scan(t["x"], t["dt"], t["A_log"], t["B"], t["C"], t["D"], t["dt_bias"], True, None, cu, t["dy"])
    return y, got, r


@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("form", FORMS, ids=str)
@pytest.mark.parametrize("T", [1, 5, 40, 64])
def test_key_gradients_inside_a_chunk(T, form, dtype):
    _, got, r = run(T, form, dtype, skip=False)
    for n, v in (("dB", got[3]), ("dC", got[4])):
        print(n, "%.2e" % float((ref.d(v) - r[n]).norm() / r[n].norm()))
        ref.held(n, v, r[n], r[n + "m"], dtype, 2.0 ** -16)


@pytest.mark.parametrize("skip", [False, True])
@pytest.mark.parametrize("dtype", [BF, HF])
@pytest.mark.parametrize("form", FORMS, ids=str)
def test_single_tokens(form, dtype, skip):
    lens = [1] * 9 + [0, 1]
    y, got, r = run(10, form, dtype, lens=lens, skip=skip)
    ref.held("y", y, r["y"], r["ym"], dtype, 2.0 ** -20)
    ref.held("dx", got[0], r["dx"], r["dxm"], dtype, 2.0 ** -20)
