"""The convolution at the most tokens that a call takes: counts and offsets next to 2^31."""
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda

pytestmark = pytest.mark.gpu


def test_convolution():
    """Both directions of one channel, slice by slice against 64 bits: p of four terms is off by 5 2^-24 of their
    magnitudes, the output is rounded to bf16."""
    T, W, step = 2 ** 31 - 65536 - 1, 4, 1 << 26
    x, dy = torch.empty(1, T, 1, dtype=torch.bfloat16, device="cuda").normal_(), torch.empty(1, T, 1, dtype=torch.bfloat16, device="cuda").normal_()
    w = torch.randn(1, W, generator=torch.Generator().manual_seed(1)).cuda()
    y, final = kda.short_conv_fwd(x, w)
    dx = kda.short_conv_bwd(x, w, dy)["dx"]
    assert torch.equal(final[0], x[0, -(W - 1):])
    for lo in range(0, T, step):
        hi = min(T, lo + step)
        for got, line, taps, first in ((y, x, range(W), lo - (W - 1)), (dx, dy, range(W - 1, -1, -1), lo)):
            a, b = max(first, 0), min(first + hi - lo + W - 1, T)
            part = torch.zeros(hi - lo + W - 1, dtype=torch.float64, device="cuda")
            part[a - first:b - first] = line[0, a:b, 0]
            want = sum(part[k:k + hi - lo] * w[0, j].double() for k, j in enumerate(taps))
            size = sum((part[k:k + hi - lo] * w[0, j].double()).abs() for k, j in enumerate(taps))
            off = (got[0, lo:hi, 0].double() - want).abs() - (2.0 ** -8 * want.abs() + 5 * 2.0 ** -24 * size * (1 + 2.0 ** -8))
            assert bool((off <= 0).all()), lo
