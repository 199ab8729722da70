"""Rows that the operators at a layer's ends take: as many as their launches of
fewer than 2^32 threads hold, counted for the form that runs (no GPU); and, on
an MI355X, a call beyond what a thread count of another form allows."""
import ctypes

import pytest
import torch

import gated_delta_rule_66_amd as gdr
from gated_delta_rule_66_amd import _lib
from gated_delta_rule_66_amd._lib import GDR_BF16, GatedNormProblem, QuantizeProblem, SandwichNormProblem, lib

MOST = 0xffff0000 // 64          # waves of a launch


def gated(rows, D, size, quant=0):
    return GatedNormProblem(rows, D, size, GDR_BF16, GDR_BF16, 1, 0, 1, quant, 0, 1e-6, D, D)


def sandwich(rows, D):
    return SandwichNormProblem(rows, D, GDR_BF16, GDR_BF16, GDR_BF16, 2, 0, 0, 1e-6, 1.0, D, D)


def quantize(rows, D):
    return QuantizeProblem(rows, D, GDR_BF16, 2, 0, D)


@pytest.mark.parametrize("problem,check,waves", [
    # lanes: a wave holds a row of up to 1024 columns, a block's waves 1024 each
    (lambda n: gated(n, 4096, 8), lib.gdr_gated_norm_check, 4),
    (lambda n: gated(n, 4096, 512), lib.gdr_gated_norm_check, 4),
    (lambda n: gated(n, 1024, 8), lib.gdr_gated_norm_check, 1),
    (lambda n: gated(n, 1040, 16), lib.gdr_gated_norm_check, 2),
    # units: a wave or more a group
    (lambda n: gated(n, 2000, 250), lib.gdr_gated_norm_check, 8),
    (lambda n: gated(n, 8160, 2040), lib.gdr_gated_norm_check, 8),
    # segments: a block of 512 columns a wave, beyond 8192 of 1024
    (lambda n: gated(n, 2000, 250, 2), lib.gdr_gated_norm_check, 4),
    (lambda n: gated(n, 4096, 64 + 64, 2), lib.gdr_gated_norm_check, 4),
    (lambda n: gated(n, 16380, 12), lib.gdr_gated_norm_check, 16),
    (lambda n: sandwich(n, 512), lib.gdr_sandwich_norm_check, 1),
    (lambda n: sandwich(n, 8192), lib.gdr_sandwich_norm_check, 16),
    (lambda n: sandwich(n, 16384), lib.gdr_sandwich_norm_check, 16),
    (lambda n: quantize(n, 1024), lib.gdr_quantize_check, 1),
    (lambda n: quantize(n, 16384), lib.gdr_quantize_check, 4),
    (lambda n: quantize(n, 65536), lib.gdr_quantize_check, 16),
])
def test_rows_up_to_a_launchs_threads(problem, check, waves):
    def verdict(rows):
        return _lib.STATUS[check(ctypes.byref(problem(rows)), None, 0)]
    most = MOST // waves
    assert verdict(most - 3) == "GDR_OK"          # (a block may hold four rows)
    assert verdict(most + 4) == "GDR_ERR_SHAPE"
    assert "too many rows" in lib.gdr_last_error().decode()


@pytest.mark.gpu
def test_many_narrow_groups():
    """131,072 rows of 512 groups of 8: 2^26 groups, but a row's waves hold them."""
    rows, D = 131072, 4096
    g = torch.Generator(device="cuda").manual_seed(0)
    x, z = (torch.randn(rows, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    w = torch.ones(8, dtype=torch.bfloat16, device="cuda")
    y, rstd = gdr.gated_rms_norm_fwd(x, z, w, norm_group=8)
    grads = gdr.gated_rms_norm_bwd(y, x, z, w, rstd, norm_group=8)
    for part in (slice(0, 5), slice(rows - 5, rows)):
        ys, rs = gdr.gated_rms_norm_fwd(x[part], z[part], w, norm_group=8)
        assert torch.equal(y[part], ys) and torch.equal(rstd[part], rs)
        small = gdr.gated_rms_norm_bwd(ys, x[part], z[part], w, rs, norm_group=8)
        assert torch.equal(grads[0][part], small[0]) and torch.equal(grads[1][part], small[1])
