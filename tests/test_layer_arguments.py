"""Arguments of the layer operators that the host has to look at before the
library does (no GPU)."""
import pytest
import torch

import gated_delta_rule_66_amd as gdr
from gated_delta_rule_66_amd import _layer_ops

BIG = (1 << 32) + 8        # 8 once its higher bits are dropped


def meta(*shape, dtype=torch.bfloat16):
    return torch.empty(*shape, dtype=dtype, device="meta")


def refused(call, name):
    with pytest.raises(gdr.GdrError) as e:
        call()
    assert e.value.name == name, e.value


def test_sizes_beyond_32_bits():
    for x in (meta(1, BIG, 1), meta(BIG, 1, 1)):
        refused(lambda: gdr.causal_conv1d(x, meta(1, 4)), "GDR_ERR_SHAPE")
        refused(lambda: gdr.causal_conv1d_update(x, meta(x.shape[0], 3, 1), meta(1, 4)), "GDR_ERR_SHAPE")
    refused(lambda: gdr.causal_conv1d(meta(1, 8, 1), meta(1, (1 << 32) + 4)), "GDR_ERR_SHAPE")
    for shape in ((BIG, 4), (1 << 16, (1 << 16) + 1, 4), (2, (1 << 32) + 128)):
        x = meta(*shape)
        refused(lambda: gdr.rms_norm(x, meta(shape[-1])), "GDR_ERR_SHAPE")
        refused(lambda: gdr.rms_norm_quant(x, meta(shape[-1])), "GDR_ERR_SHAPE")
    for x, b in ((meta(1, BIG, 2, 64), meta(1, BIG, 1, 64)), (meta(1, 8, 2, BIG * 8), meta(1, 8, 1, 64)),
                 (meta(1, 8, 2, 64), meta(1, 8, 1, (1 << 32) + 64))):
        dt, a = meta(*x.shape[:3]), meta(2)
        refused(lambda: gdr.chunk_selective_scan(x, dt, a, b, b), "GDR_ERR_SHAPE")
        refused(lambda: gdr.fused_recurrent_selective_scan(x, dt, a, b, b), "GDR_ERR_SHAPE")


@pytest.mark.parametrize("group", [(1 << 32) + 128, 1 << 32, -1, 64, 127.5, None])
def test_group_sizes(group):
    """The binding sizes the scales from it: 2^32 + 128 would give one scale a
    row to a kernel that writes one per 128 columns."""
    refused(lambda: gdr.rms_norm_quant(torch.zeros(2, 512), torch.ones(512), group_size=group),
            "GDR_ERR_ARG")


def test_offsets_beyond_32_bits_and_other_types():
    x = torch.zeros(1, 8, 4)
    ok = torch.tensor([0, 3, 8])
    for cu in (ok, ok.int(), ok.short()):
        n, dev, host = _layer_ops._seqs(x, cu, None)
        assert n == 2 and host.dtype == dev.dtype == torch.int32 and host.tolist() == [0, 3, 8]
    far = torch.tensor([0, 3, (1 << 32) + 8])
    for cu, cpu in ((far, None), (far, far), (ok, far), (ok.float(), None), (ok, ok.double()),
                    (ok.bool(), None)):
        refused(lambda: _layer_ops._seqs(x, cu, cpu), "GDR_ERR_VARLEN")
