"""Rows that are no whole pieces: B and C behind an odd number of other values in the rows of one projection, u, delta
and z as slices that start at odd elements, and convolution inputs of such rows.  The results equal those of
contiguous tensors bit for bit: the layout decides how values are loaded, not what is computed with them."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.test_gpu_ssm import make

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def odd(t, lead, before=1, behind=2):
    """t's values as the slice [before, before + width) of wider rows."""
    width = int(np.prod(t.shape[lead:]))
    wide = torch.zeros(*t.shape[:lead], before + width + behind, dtype=t.dtype, device=t.device)
    cut = wide[..., before:before + width]
    cut.copy_(t.reshape(*t.shape[:lead], width))
    return cut.unflatten(-1, t.shape[lead:]) if t.dim() > lead + 1 else cut


def variants(d, lead):
    """Which of the inputs are slices: B and C (at an odd element and 8 bytes from a piece's start), the channels' rows,
    all of them."""
    plain = {k: d[k].contiguous() for k in ("u", "delta", "z", "B", "C")}
    for names, before, behind in ((("B", "C"), 1, 2), (("B", "C"), 4, 4), (("B",), 3, 5), (("u", "delta", "z"), 1, 2), (("u", "delta", "z"), 2, 2),
                                  (("delta",), 1, 1), (("u", "delta", "z", "B", "C"), 5, 2)):
        yield plain, {k: odd(v, lead, before, behind) if k in names else v for k, v in plain.items()}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("C,G", [(72, 1), (256, 2), (37, 1)])
def test_scan(C, G, S, dtype):
    lengths = [33, 90, 1, 70]
    T = sum(lengths)
    d = make((1, T), C, S, G, dtype, 3000 + S, True, True, True)
    dy = torch.randn(1, T, C, generator=torch.Generator().manual_seed(1)).to(dtype).cuda()
    kw = dict(D=d["D"], delta_bias=d["bias"], cu_seqlens=torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32).cuda(),
              initial_state=torch.randn(4, C, S, generator=torch.Generator().manual_seed(2)).cuda())
    want = None
    for plain, cut in variants(d, 2):
        if want is None:
            a = (plain["u"], plain["delta"], d["A"], plain["B"], plain["C"])
            want, wg = kda.ssm_scan_fwd(*a, z=plain["z"], **kw), kda.ssm_scan_bwd(*a, dy, z=plain["z"], **kw)
        a = (cut["u"], cut["delta"], d["A"], cut["B"], cut["C"])
        got, g = kda.ssm_scan_fwd(*a, z=cut["z"], **kw), kda.ssm_scan_bwd(*a, dy, z=cut["z"], **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert all(torch.equal(g[k], wg[k]) for k in wg)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("S", [8, 16, 32, 64])
@pytest.mark.parametrize("N,C,G", [(1, 72, 1), (9, 37, 1), (301, 1024, 2)])
def test_scan_step(N, C, G, S, dtype):
    d = make((N,), C, S, G, dtype, 3100 + S, True, True, True)
    g = torch.Generator().manual_seed(3)
    pool, slots = torch.randn(N + 2, C, S, generator=g).cuda(), torch.randperm(N + 2, generator=g)[:N].to(torch.int32).cuda()
    kw = dict(D=d["D"], delta_bias=d["bias"], slots=slots)
    want = None
    for plain, cut in variants(d, 1):
        if want is None:
            wp = pool.clone()
            want = kda.ssm_step(plain["u"], plain["delta"], d["A"], plain["B"], plain["C"], wp, z=plain["z"], **kw)
        p = pool.clone()
        y = kda.ssm_step(cut["u"], cut["delta"], d["A"], cut["B"], cut["C"], p, z=cut["z"], **kw)
        assert torch.equal(y, want) and torch.equal(p, wp)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("W", [2, 3, 4])
@pytest.mark.parametrize("C", [72, 256, 70])
def test_convolution(C, W, dtype):
    lengths = [33, 90, 1, 70]
    T, N = sum(lengths), len(lengths)
    g = torch.Generator().manual_seed(3200 + C)
    x, dy = torch.randn(1, T, C, generator=g).to(dtype).cuda(), torch.randn(1, T, C, generator=g).to(dtype).cuda()
    w, b, h = torch.randn(C, W, generator=g).cuda(), torch.randn(C, generator=g).cuda(), torch.randn(N, W - 1, C, generator=g).to(dtype).cuda()
    kw = dict(bias=b, conv_act=1, initial=h, cu_seqlens=torch.tensor(np.cumsum([0] + lengths), dtype=torch.int32).cuda())
    want, wg = kda.short_conv_fwd(x, w, **kw), kda.short_conv_bwd(x, w, dy, **kw)
    xs, pool = x[0, :40].contiguous(), torch.randn(40, W - 1, C, generator=g).to(dtype).cuda()
    wp = pool.clone()
    ws = kda.short_conv_step(xs, wp, w, bias=b, conv_act=1)
    # sums of T terms below 1.1 |dy| |x| each, in two orders
    apart = 2 * T * 2.0 ** -24 * 1.1 * float(dy.float().abs().sum(1).max()) * max(float(x.abs().max()), float(h.abs().max()), 1.0)
    for before, behind in ((1, 2), (2, 2), (4, 4)):
        cut = odd(x, 2, before, behind)
        got, gg = kda.short_conv_fwd(cut, w, **kw), kda.short_conv_bwd(cut, w, dy, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
        assert torch.equal(gg["dx"], wg["dx"]) and torch.equal(gg["dinitial"], wg["dinitial"])
        # (the runs that the sums over tokens go by depend on how many blocks there are)
        for k in ("dweight", "dbias"):
            torch.testing.assert_close(gg[k], wg[k], rtol=0, atol=apart)
        p = pool.clone()
        y = kda.short_conv_step(odd(xs, 1, before, behind), p, w, bias=b, conv_act=1)
        assert torch.equal(y, ws) and torch.equal(p, wp)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("act", [0, 1])
@pytest.mark.parametrize("N,C,W", [(1, 8, 4), (5, 37, 3), (33, 1032, 4), (256, 264, 2), (70, 13, 4), (9, 2048, 3)])
def test_convolution_steps_are_the_prefill(N, C, W, act, dtype):
    """The same fused multiply-adds in the same order, so the same bits."""
    g = torch.Generator().manual_seed(3300 + N)
    T = 7
    x = torch.randn(N, T, C, generator=g).to(dtype).cuda()
    w, b = torch.randn(C, W, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    whole, last = kda.short_conv_fwd(x, w, bias=b, conv_act=act)
    pool = torch.zeros(N, W - 1, C, dtype=dtype, device="cuda")
    for t in range(T):
        assert torch.equal(kda.short_conv_step(x[:, t], pool, w, bias=b, conv_act=act), whole[:, t])
    assert torch.equal(pool, last)
