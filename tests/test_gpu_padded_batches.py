"""Packed batches whose offsets leave rows at the front and the back that belong to no sequence: the loss does not
depend on them, so their gradients are zero, whatever lies in those rows and in the memory that the gradients are
put into.  Tolerances of the rows in between as in the tests of each operator."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests import test_gpu_short_conv as short_conv, test_gpu_ssm as ssm
from tests.layer_ref import conv, f64, scan

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
# tokens, offsets: short of a tile on either side, whole tiles and runs of nobody, sequences without tokens, no sequence
BATCHES = [(100, [4, 30, 81]), (700, [130, 131, 131, 400]), (300, [0, 5, 7]), (300, [290, 300]), (90, [40, 40, 40]), (64, [64, 64]),
           (70, [9])]


@pytest.fixture
def dirty_memory():
    """Fresh tensors are full of NaN."""
    torch.use_deterministic_algorithms(True, warn_only=True)
    assert torch.utils.deterministic.fill_uninitialized_memory and bool(torch.empty(3, device="cuda").isnan().all())
    yield
    torch.use_deterministic_algorithms(False)


def nobody(T, cu):
    rows = torch.ones(T, dtype=torch.bool)
    rows[cu[0]:cu[-1]] = False
    return rows


def spoiled(t, rows):
    t = t.clone()
    t[0, rows.to(t.device)] = float("nan")
    return t


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("C,W", [(64, 4), (37, 3), (1032, 2)])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_convolution_gradients(batch, C, W, dtype, gdtype, dirty_memory):
    T, cu = BATCHES[batch]
    N, rows = len(cu) - 1, nobody(T, cu)
    g = torch.Generator().manual_seed(2000 + batch)
    x, dy = torch.randn(1, T, C, generator=g).to(dtype).cuda(), torch.randn(1, T, C, generator=g).to(gdtype).cuda()
    w, b = (torch.randn(C, W, generator=g) * 0.5).cuda(), torch.randn(C, generator=g).cuda()
    h, df = torch.randn(N, W - 1, C, generator=g).to(dtype).cuda(), torch.randn(N, W - 1, C, generator=g).to(gdtype).cuda()
    got = kda.short_conv_bwd(spoiled(x, rows), w, spoiled(dy, rows), bias=b, conv_act=1, initial=h, dfinal=df,
                             cu_seqlens=torch.tensor(cu, dtype=torch.int32).cuda())
    assert bool((got["dx"][0, rows.cuda()] == 0).all())
    ref = conv(f64(x[0]), f64(w), f64(b), 1, f64(h), cu, f64(dy[0]), f64(df))
    short_conv.within(got["dx"][0], ref["dx"], 2.0 ** -19 * ref["dx_mag"], gdtype)
    short_conv.within(got["dinitial"], ref["dinitial"], 2.0 ** -19 * ref["di_mag"], gdtype)
    for k, mag in (("dweight", "dw_mag"), ("dbias", "db_mag")):
        short_conv.within(got[k], ref[k], (2.0 ** -19 + T * 2.0 ** -24) * ref[mag], F32)


# channels and groups: chunks of 16, 32 and 64 tokens backwards, and an odd number of channels
@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("C,G,S", [(72, 1, 16), (180, 90, 16), (680, 340, 8), (37, 1, 32), (24, 2, 64)])
@pytest.mark.parametrize("batch", range(len(BATCHES)))
def test_scan_gradients(batch, C, G, S, dtype, gdtype, dirty_memory):
    T, cu = BATCHES[batch]
    N, rows = len(cu) - 1, nobody(T, cu)
    d = ssm.make((1, T), C, S, G, dtype, 2100 + batch, True, True, True)
    g = torch.Generator().manual_seed(2200 + batch)
    for k in ("u", "delta", "z", "B", "C"):
        d[k] = d[k].clone()
        d[k][0, rows.cuda()] = 0          # (the plain form sums over every row)
    dy = torch.randn(1, T, C, generator=g).to(gdtype).cuda()
    dy[0, rows.cuda()] = 0
    s0, df = torch.randn(N, C, S, generator=g).cuda(), torch.randn(N, C, S, generator=g).cuda()
    d.update(sp=True, s0=s0, cu=torch.tensor(cu, dtype=torch.int32).cuda())
    a, kw = ssm.call_args({**d, **{k: spoiled(d[k], rows) for k in ("u", "delta", "z", "B", "C")}})
    got = kda.ssm_scan_bwd(*a, spoiled(dy, rows), dfinal_state=df, **kw)
    for k in ("du", "ddelta", "dz", "dB", "dC"):
        assert bool((got[k][0, rows.cuda()] == 0).all()), k
    r = scan(*ssm.ref_args(d), f64(dy)[0], f64(df))
    for k, dt, n in (("du", gdtype, S), ("ddelta", gdtype, S), ("dz", gdtype, S), ("dB", gdtype, C), ("dC", gdtype, C), ("dA", F32, T),
                     ("dD", F32, T), ("ddelta_bias", F32, T), ("dinitial_state", F32, 1)):
        ssm.within(got[k], r[k], (2.0 ** -19 + n * 2.0 ** -24) * r[k + "_err"], dt)
