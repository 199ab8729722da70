"""How far an infinity or a NaN reaches in the selective scan's outputs (needs
an MI355X): from its own token on, in x from the start of its 64-token chunk,
and never into another sequence; what it does not reach keeps its bits."""
import pytest
import torch

import gated_delta_rule_66_amd as gdr
import test_gpu_layer_scan as scan

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("key", ["x", "B", "C", "dt"])
@pytest.mark.parametrize("dtype,K,V,G", [(BF, 64, 64, 1), (BF, 128, 128, 2), (BF, 64, 64, 2), (HF, 128, 64, 2)])
def test_reach(dtype, K, V, G, key, bad):
    lens, at = [150, 90], 100                   # at: in the first sequence's second chunk
    t = scan.dev(scan.make(1, sum(lens), 2, G, K, V, dtype, lens=lens))
    cu = t["cu"].cpu()
    f = lambda q: gdr.chunk_selective_scan_fwd(*scan.args(q), True, q["state"], True, q["cu"], cu)  # noqa: E731
    y, last = f(t)
    q = {**t, key: t[key].clone()}
    q[key][0, at] = bad
    y2, last2 = f(q)
    assert not y2[0, at].isfinite().any()
    keep = torch.ones(sum(lens), dtype=torch.bool, device="cuda")
    keep[64 if key == "x" else at:lens[0]] = False
    if key == "C":                              # an output's own factor: it goes no further
        keep[at + 1:] = True
    if dtype == HF and key != "C":              # a tile with an infinity is not scaled: its other values
        keep[64:at] = False                     # may round differently, but stay values
        assert key == "x" or torch.allclose(y2[0, 64:at].float(), y[0, 64:at].float(), rtol=2e-3, atol=2e-3)
    assert torch.equal(y2[0, keep], y[0, keep])
    assert torch.equal(last2[1], last[1])
    if key != "C":
        assert not last2[0].isfinite().all()
    else:
        assert torch.equal(last2[0], last[0])
