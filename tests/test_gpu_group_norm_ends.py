"""Group norm at the ends of its numbers: infinite values, variances and eps near the least of fp32."""
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.test_gpu_group_norm import BF16, F32, check, make

pytestmark = pytest.mark.gpu

INF = float("inf")


@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("over", ["token", "sequence"])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,C,G", [(70, 32, 4), (40, 2048, 16), (9, 515, 1), (6, 4096, 2), (3, 12288, 1), (20, 90, 9)])
def test_an_infinite_value_leaves_its_group_without_a_mean(T, C, G, dtype, over, act):
    """The group's mean is infinite and its variance is not a number, nor is anything that is normalised by them: all of the
    group (of the token, or of the sequence), and nothing else."""
    x, w, b, dy = make((1, T), C, dtype, T + C, True)
    dy, cg = dy.to(dtype).cuda(), C // G
    kw = dict(weight=w, bias=b, act=act, over=over)
    clean, grads = kda.group_norm_fwd(x, G, **kw), kda.group_norm_bwd(x, G, dy, **kw)
    row, group = T // 2, G // 2
    for inf in (INF, -INF):
        bad = x.clone()
        bad[0, row, group * cg + cg // 3] = inf
        where = torch.zeros(1, T, C, dtype=torch.bool, device="cuda")
        where[0, row if over == "token" else slice(None), group * cg:(group + 1) * cg] = True
        y, out = kda.group_norm_fwd(bad, G, **kw), kda.group_norm_bwd(bad, G, dy, **kw)
        for got, want in ((y, clean), (out["dx"], grads["dx"])):
            assert bool(torch.isnan(got[where]).all()) and torch.equal(got[~where], want[~where])
        channels = where[0, row]
        assert bool(torch.isnan(out["dweight"][channels]).all()) and torch.equal(out["dweight"][~channels], grads["dweight"][~channels])
        assert torch.equal(out["dbias"][~channels], grads["dbias"][~channels])
        if act == 0:  # sum dy
            assert torch.equal(out["dbias"], grads["dbias"])


@pytest.mark.parametrize("eps", [2.0 ** -120, 2.0 ** -130])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("over", ["token", "sequence"])
def test_the_least_variances(over, dtype, eps):
    """Any eps > 0, a subnormal one too: values of some 2^-64, whose variance is 2^-128 and next to eps."""
    T, C, G = 60, 96, 3
    x, w, b, dy = make((1, T), C, dtype, 5, True)
    x = x * 2.0 ** -64
    check(x, G, w, b, dy, 0, [(0, T)], over, 96, dtype, eps=eps)
