"""The 8-bit outputs of the RMS norm next to ties (needs an MI355X).  Rows of
+1 and -1 have a mean square of exactly 1, so with eps = 0 the values to be
quantised are the weights themselves: no tolerance is left, q is the fp32
quotient rounded to nearest even."""
import pytest
import torch

import gated_delta_rule_66_amd as gdr

pytestmark = pytest.mark.gpu


def tie_points(fmt):
    """Halfway points between neighbouring 8-bit values, the largest excluded."""
    if fmt == "int8":
        v = torch.arange(0, 128).float()
    else:
        v = torch.arange(0, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).float()
    return (v[1:] + v[:-1]) / 2


@pytest.mark.parametrize("fmt", ["fp8", "int8"])
@pytest.mark.parametrize("group", [0, 128])
@pytest.mark.parametrize("seed", range(4))
def test_values_next_to_ties(fmt, group, seed):
    g = torch.Generator().manual_seed(seed)
    D, top = 2048, 448.0 if fmt == "fp8" else 127.0
    ties = tie_points(fmt)
    w = torch.empty(D)
    for a in range(0, D, group or D):
        b = a + (group or D)
        largest = float(torch.rand(1, generator=g) + 0.5) * 2.0 ** int(torch.randint(-20, 20, (1,), generator=g))
        scale = torch.tensor(largest) / top
        pick = ties[torch.randint(len(ties), (b - a,), generator=g)]
        w[a:b] = pick * scale * (1 + torch.randint(-1, 2, (b - a,), generator=g) * 2.0 ** -24)
        w[a] = largest
    x = torch.randint(0, 2, (3, D), generator=g).float() * 2 - 1
    width = group or D
    y = x * w
    scale = y.view(3, -1, width).abs().amax(-1) / top
    want = (y.view(3, -1, width) / scale[..., None]).clamp(-top, top).view(3, D)
    q, s, _ = gdr.rms_norm_quant(x.cuda(), w.cuda(), 0.0, format=fmt, group_size=group)
    assert torch.equal(s.cpu(), scale)
    if fmt == "int8":
        assert torch.equal(q.cpu(), torch.round(want).to(torch.int8))
    else:
        assert torch.equal(q.cpu().float(), want.to(torch.float8_e4m3fn).float())
