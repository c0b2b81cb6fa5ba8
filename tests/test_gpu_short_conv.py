"""The short convolution (forward, backward, single token) against its plain 64-bit form.

Tolerances, element by element.  p is W + 1 fp32 operations, so it is off by at most (W + 1) 2^-24 M with M
the sum of the magnitudes it adds; SiLU's slope is below 1.1, and sigmoid(p) itself is off by 2^-22
(the exponential) + |p| log2(e) 2^-24 (its rounded argument, weighted by 1 - sigmoid) + 2^-23, relative:
together below 2^-20 M.  Gradients: dp has two such factors of dy, below 2^-19 |dy| (1 + M), and dx is
a sum of W of them; dw and dbias are sums over tokens in fp32, off by at most T 2^-24 of the sum of
magnitudes in whatever order they are added.  Rounding to the output type adds half a step."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.layer_ref import conv, f64, half_step

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def within(got, ref, tol, dtype):
    got = f64(got).reshape(ref.shape)
    assert np.isfinite(got).all()
    off = np.abs(got - ref) - (half_step(dtype) * np.abs(ref) + tol * (1 + half_step(dtype)) + 1e-30)
    assert (off <= 0).all(), f"off by up to {off.max():.3e} more than allowed, {int((off > 0).sum())} values"


def make(lengths, C, W, dtype, seed, history, bias, wide=1):
    g = torch.Generator().manual_seed(seed)
    T, N = sum(lengths), len(lengths)
    x = torch.randn(1, T, C * wide, generator=g).to(dtype).cuda()[:, :, (wide - 1) * C:]
    return dict(x=x, w=(torch.randn(C, W, generator=g) * 0.5).cuda(), b=torch.randn(C, generator=g).cuda() if bias else None,
                h=torch.randn(N, W - 1, C, generator=g).to(dtype).cuda() if history else None,
                cu=torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda(),
                dy=torch.randn(1, T, C, generator=g), df=torch.randn(N, W - 1, C, generator=g))


CASES = [
    # lengths, C, W, act, history, bias, wide: one token; runs and tiles met and missed by one; empty and short sequences
    ([1], 8, 4, 1, False, False, 1),
    ([64], 256, 4, 1, True, True, 1),
    ([65, 31, 1], 264, 4, 1, True, False, 2),
    ([0, 3, 0, 0, 2, 1, 90, 0], 40, 4, 0, True, True, 1),
    ([33, 63, 129], 37, 3, 1, True, True, 1),
    ([2, 1, 1, 5, 130], 1032, 2, 1, True, True, 3),
    ([700], 13, 4, 1, False, True, 2),
    ([1] * 40 + [17] * 9, 96, 4, 1, True, False, 1),
    ([1000, 24, 2000], 2048, 4, 1, False, False, 1),
    ([3, 4], 7, 3, 0, False, False, 1),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward(case, dtype):
    lengths, C, W, act, history, bias, wide = CASES[case]
    d = make(lengths, C, W, dtype, 100 + case, history, bias, wide)
    y, final = kda.short_conv_fwd(d["x"], d["w"], bias=d["b"], conv_act=act, initial=d["h"], cu_seqlens=d["cu"])
    ry, rfinal, M = conv(f64(d["x"][0]), f64(d["w"]), f64(d["b"]), act, f64(d["h"]), d["cu"].tolist())
    within(y[0], ry, 2.0 ** -20 * M, dtype)
    assert np.array_equal(f64(final), rfinal)


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_backward(case, dtype, gdtype):
    lengths, C, W, act, history, bias, wide = CASES[case]
    d = make(lengths, C, W, dtype, 200 + case, history, bias, wide)
    dy, df = d["dy"].to(gdtype).cuda(), d["df"].to(gdtype).cuda()
    got = kda.short_conv_bwd(d["x"], d["w"], dy, bias=d["b"], conv_act=act, initial=d["h"], cu_seqlens=d["cu"], dfinal=df)
    ref = conv(f64(d["x"][0]), f64(d["w"]), f64(d["b"]), act, f64(d["h"]), d["cu"].tolist(), f64(dy[0]), f64(df))
    T = sum(lengths)
    within(got["dx"][0], ref["dx"], 2.0 ** -19 * ref["dx_mag"], gdtype)
    within(got["dweight"], ref["dweight"], (2.0 ** -19 + T * 2.0 ** -24) * ref["dw_mag"], F32)
    assert (got["dbias"] is None) == (not bias) and (got["dinitial"] is None) == (not history)
    if bias:
        within(got["dbias"], ref["dbias"], (2.0 ** -19 + T * 2.0 ** -24) * ref["db_mag"], F32)
    if history:
        within(got["dinitial"], ref["dinitial"], 2.0 ** -19 * ref["di_mag"], gdtype)


def test_backward_against_differences():
    # central differences of the 32-bit forward, summed in 64 bits: truncation 1e-6, cancellation 2^-20 / 1e-2
    d = make([5, 9], 16, 4, F32, 300, True, True)
    dy, df = d["dy"].cuda(), d["df"].cuda()
    got = kda.short_conv_bwd(d["x"], d["w"], dy, bias=d["b"], conv_act=1, initial=d["h"], cu_seqlens=d["cu"], dfinal=df)

    def loss(x, w, b, h):
        y, f = kda.short_conv_fwd(x, w, bias=b, conv_act=1, initial=h, cu_seqlens=d["cu"])
        return float((y.double() * dy.double()).sum() + (f.double() * df.double()).sum())
    base = [d["x"].contiguous(), d["w"], d["b"], d["h"]]
    rng = np.random.default_rng(1)
    for i, name in enumerate(("dx", "dweight", "dbias", "dinitial")):
        way = torch.from_numpy(rng.standard_normal(tuple(base[i].shape))).float().cuda()
        plus, minus = ([t + (s * 1e-2 * way if j == i else 0) for j, t in enumerate(base)] for s in (1, -1))
        slope = (loss(*plus) - loss(*minus)) / 2e-2
        want = float((got[name].reshape(way.shape).double() * way.double()).sum())
        scale = float((got[name].reshape(way.shape).double() * way.double()).abs().sum()) + 1.0
        # third derivatives of SiLU are below 0.5 and the steps below 0.05: (0.05)^2 / 6 of the scale
        assert abs(slope - want) <= 2e-3 * scale, name


def test_dense_batch_and_no_final():
    d = make([50, 50, 50], 72, 4, BF16, 310, True, True)
    packed, f1 = kda.short_conv_fwd(d["x"], d["w"], bias=d["b"], conv_act=1, initial=d["h"], cu_seqlens=d["cu"])
    dense, f2 = kda.short_conv_fwd(d["x"].reshape(3, 50, 72), d["w"], bias=d["b"], conv_act=1, initial=d["h"])
    assert torch.equal(packed.view(3, 50, 72), dense) and torch.equal(f1, f2)
    y, none = kda.short_conv_fwd(d["x"], d["w"], bias=d["b"], conv_act=1, initial=d["h"], cu_seqlens=d["cu"], output_final=False)
    assert none is None and torch.equal(y, packed)


def test_no_tokens_hands_the_history_on():
    g = torch.Generator().manual_seed(311)
    h = torch.randn(3, 3, 24, generator=g).to(BF16).cuda()
    x, w = torch.empty(1, 0, 24, dtype=BF16, device="cuda"), torch.ones(24, 4, device="cuda")
    cu = torch.zeros(4, dtype=torch.int32, device="cuda")
    y, final = kda.short_conv_fwd(x, w, initial=h, cu_seqlens=cu)
    assert y.shape == (1, 0, 24) and torch.equal(final, h)
    got = kda.short_conv_bwd(x, w, x, initial=h, cu_seqlens=cu, dfinal=h)
    assert torch.equal(got["dinitial"], h) and not got["dweight"].any()
    y, final = kda.short_conv_fwd(x, w, cu_seqlens=cu)
    assert not final.any()


def test_rows_of_no_sequence_are_left_alone():
    d = make([10, 90], 64, 4, BF16, 312, False, False)
    cu = torch.tensor([4, 30, 81], dtype=torch.int32, device="cuda")   # rows 0-3 and 81-99 belong to nobody
    y = torch.full((1, 100, 64), 7.0, dtype=BF16, device="cuda")
    kda.short_conv_fwd(d["x"], d["w"], conv_act=1, cu_seqlens=cu, y=y)
    ref, _, M = conv(f64(d["x"][0]), f64(d["w"]), None, 1, None, [4, 30, 81])
    within(y[0, 4:81], ref[4:81], 2.0 ** -20 * M[4:81], BF16)
    assert bool((y[0, :4] == 7).all()) and bool((y[0, 81:] == 7).all())


def test_offsets_out_of_order_stay_in_bounds():
    d = make([200], 64, 4, BF16, 313, True, False)
    h = torch.randn(4, 3, 64).to(BF16).cuda()
    for cu in ([0, 150, 50, 180, 200], [0, -5, 900, 20, 200], [200, 0, 200, 0, 7], [2 ** 31 - 1, -2 ** 31, 5, 6, 2 ** 31 - 1]):
        c = torch.tensor(cu, dtype=torch.int32, device="cuda")
        y, f = kda.short_conv_fwd(d["x"], d["w"], conv_act=1, initial=h, cu_seqlens=c)
        kda.short_conv_bwd(d["x"], d["w"], y, conv_act=1, initial=h, cu_seqlens=c, dfinal=h)
    torch.cuda.synchronize()
    ok, _ = kda.short_conv_fwd(d["x"], d["w"], conv_act=1, initial=h[:1], cu_seqlens=torch.tensor([0, 200], dtype=torch.int32).cuda())
    ref, _, M = conv(f64(d["x"][0]), f64(d["w"]), None, 1, f64(h[:1]), [0, 200])
    within(ok[0], ref, 2.0 ** -20 * M, BF16)


def test_infinite_and_nan_inputs_stay_in_their_rows():
    d = make([20, 20], 16, 4, F32, 314, False, False)
    x = d["x"].contiguous()
    clean, _ = kda.short_conv_fwd(x, d["w"], conv_act=1, cu_seqlens=d["cu"])
    x[0, 18, 3], x[0, 5, 7] = float("nan"), float("inf")
    y, _ = kda.short_conv_fwd(x, d["w"], conv_act=1, cu_seqlens=d["cu"])
    touched = torch.zeros(40, 16, dtype=torch.bool, device="cuda")
    touched[18:20, 3] = True      # not into the next sequence
    touched[5:9, 7] = True
    assert torch.equal(y[0][~touched], clean[0][~touched]) and bool(y[0, 18:20, 3].isnan().all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,C,W", [(1, 8, 4), (5, 37, 3), (33, 1032, 4), (256, 264, 2)])
def test_steps_continue_a_prefill(N, C, W, dtype):
    """A prefill of some tokens and steps for the rest give what the whole prefill gives, bit for bit."""
    g = torch.Generator().manual_seed(400 + N)
    T, cut = 7, 3
    x = torch.randn(N, T, C, generator=g).to(dtype).cuda()
    w, b = torch.randn(C, W, generator=g).cuda(), torch.randn(C, generator=g).cuda()
    whole, last = kda.short_conv_fwd(x, w, bias=b, conv_act=1)
    P = N + 3
    pool = torch.full((P, W - 1, C), 5.0, dtype=dtype, device="cuda")
    slots = torch.randperm(P, generator=g)[:N].to(torch.int32).cuda()
    _, h = kda.short_conv_fwd(x[:, :cut].contiguous(), w, bias=b, conv_act=1)
    pool[slots.long()] = h
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    for t in range(cut, T):
        y = kda.short_conv_step(x[:, t], pool, w, bias=b, conv_act=1, slots=slots, status=status)
        if dtype == F32:
            torch.testing.assert_close(y, whole[:, t], rtol=2e-6, atol=2e-6)   # the taps are added in another order
        else:
            torch.testing.assert_close(y.float(), whole[:, t].float(), rtol=2.0 ** -7, atol=2e-6)
    assert torch.equal(pool[slots.long()], last) and int(status) == 0
    others = torch.ones(P, dtype=torch.bool)
    others[slots.cpu().long()] = False
    assert bool((pool[others.cuda()] == 5).all())


def test_step_pads_and_refuses():
    C, P = 40, 4
    x = torch.randn(6, C, device="cuda")
    w = torch.randn(C, 4, device="cuda")
    pool = torch.randn(P, 3, C, device="cuda")
    before = pool.clone()
    y = torch.full((6, C), 9.0, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    # padding, an ordinary row, the same page again, out of range twice, another ordinary row
    slots = torch.tensor([-1, 2, 2, P, -7, 0], dtype=torch.int32, device="cuda")
    kda.short_conv_step(x, pool, w, slots=slots, y=y, status=status)
    assert int(status) == 5
    for i in (0, 2, 3, 4):
        assert bool((y[i] == 9).all())
    for i, p in ((1, 2), (5, 0)):
        line = torch.cat([before[p], x[i:i + 1]]).double()
        ref = (line * w.t().double()).sum(0)
        assert torch.allclose(y[i].double(), ref, rtol=0, atol=2e-5)
        assert torch.equal(pool[p], line[1:].float())
    assert torch.equal(pool[1], before[1]) and torch.equal(pool[3], before[3])
    kda.short_conv_step(x[:1], pool, w, slots=slots[:1], y=y[:1], status=status)
    assert int(status) == 0      # a padded row is no error


def test_captured_and_replayed():
    d = make([40, 60], 128, 4, BF16, 320, True, True)
    want, wf = kda.short_conv_fwd(d["x"], d["w"], bias=d["b"], conv_act=1, initial=d["h"], cu_seqlens=d["cu"])
    dy = d["dy"].to(BF16).cuda()
    wg = kda.short_conv_bwd(d["x"], d["w"], dy, bias=d["b"], conv_act=1, initial=d["h"], cu_seqlens=d["cu"])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, f = kda.short_conv_fwd(d["x"], d["w"], bias=d["b"], conv_act=1, initial=d["h"], cu_seqlens=d["cu"])
        g = kda.short_conv_bwd(d["x"], d["w"], dy, bias=d["b"], conv_act=1, initial=d["h"], cu_seqlens=d["cu"])
    for _ in range(2):
        y.zero_()
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(f, wf) and torch.equal(g["dx"], wg["dx"])
    assert torch.equal(g["dweight"], wg["dweight"])


def test_many_channels_element_by_element():
    """A channel count whose narrow runs are more than its wide ones: the workspace holds either."""
    C, T = 228 * 512 - 1, 700
    g = torch.Generator().manual_seed(330)
    x, dy = torch.randn(1, T, C, generator=g).to(BF16).cuda(), torch.randn(1, T, C, generator=g).to(BF16).cuda()
    w = torch.randn(C, 2, generator=g).cuda()
    got = kda.short_conv_bwd(x, w, dy, conv_act=0)
    prev = torch.cat([torch.zeros_like(x[:, :1]), x[:, :-1]], 1).double()
    want = torch.stack([(dy.double() * prev).sum((0, 1)), (dy.double() * x.double()).sum((0, 1))], 1)
    size = torch.stack([(dy.double() * prev).abs().sum((0, 1)), (dy.double() * x.double()).abs().sum((0, 1))], 1)
    assert bool(((got["dweight"].double() - want).abs() <= T * 2.0 ** -24 * size).all())
