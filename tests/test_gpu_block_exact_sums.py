"""The 8-bit product's sums over long rows are exact: values whose partial sums
pass 2^24 by far, where fp32 holds even numbers only, while the whole sum stays
below it, so that an fp32 output with scales of one shows every bit of it.  Here
without a GPU: an fp32 sum of them, added in any of the orders that the kernels
have, is another number.  (The GPU tests need an MI355X.)"""
import numpy as np
import pytest
import torch

import gated_delta_rule_66_amd as gdr

K = 65536
SHARE = K // 8            # of a row that one of eight waves adds up


def operands(M, N, run, K=K, seed=0):
    """Magnitudes of 64 to 127; the products' sign changes every `run` values."""
    g = torch.Generator().manual_seed(seed)
    r = lambda *s: torch.randint(64, 128, s, generator=g, dtype=torch.int8)  # noqa: E731
    sign = 1 - 2 * (torch.arange(K) // run % 2)
    return r(M, K), r(N, K) * sign.to(torch.int8)


def exact(x, w):
    y = x.double() @ w.double().t()               # integers below 2^53
    assert y.abs().max() < 2 ** 24
    return y


def added(terms):
    """One after the other in fp32."""
    return np.add.accumulate(terms.astype(np.float32), axis=-1, dtype=np.float32)[..., -1]


@pytest.mark.parametrize("run", [SHARE // 2, SHARE])
def test_fp32_sums_are_other_numbers(run):
    """Added value by value, in the matrix instructions' pieces of 32 or 64, or
    exactly within each wave's share and in fp32 only from share to share."""
    x, w = operands(4, 8, run)
    want = exact(x, w).numpy()
    p = x.numpy().astype(np.int64)[:, None] * w.numpy().astype(np.int64)[None]
    assert (p.sum(-1) == want).all() and (want % 2 == 1).any()
    pieces = [1, 32, 64] + ([SHARE] if run == SHARE else [])
    for n in pieces:
        s = added(p.reshape(4, 8, K // n, n).sum(-1))
        assert (s != want).mean() > 0.5, n
        # waves' sums in fp32 that are added as integers afterwards
        if n < SHARE:
            s = added(p.reshape(4, 8, 8, SHARE // n, n).sum(-1)).astype(np.int64).sum(-1)
            assert (s != want).mean() > 0.5, n


@pytest.mark.gpu
@pytest.mark.parametrize("run", [SHARE // 2, SHARE])
@pytest.mark.parametrize("K", [65536, 65535, 65521])
@pytest.mark.parametrize("M,N", [(1, 33), (16, 4096), (17, 40), (32, 1000), (50, 100), (64, 4100), (200, 300),
                                 (500, 2000), (1100, 1100), (2100, 4200)])
def test_sums_are_exact(M, N, K, run):
    x, w = (t.cuda() for t in operands(M, N, run, K, M))
    one = torch.ones(max(M, N), device="cuda")
    y = gdr.int8_matmul(x, one[:M], w, one[:N], out_dtype=torch.float32)
    assert torch.equal(y.double(), exact(x, w))
