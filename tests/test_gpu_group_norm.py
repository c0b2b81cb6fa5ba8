"""Group norm with an activation, channels last (over tokens and over sequences), and its backward pass against the plain 64-bit
form; the tolerances are derived in gated_norm_ref."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.gated_norm_ref import f64, norm, within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(lead, C, dtype, seed, affine, wide=1, offset=0.5):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
    x = (rn(*lead, wide * C) * (1 + 0.3 * rn(wide * C)) + offset * rn(wide * C)).to(dtype).cuda()[..., :C]
    w, b = ((1 + 0.3 * rn(C)).cuda(), (0.3 * rn(C)).cuda()) if affine else (None, None)
    return x, w, b, rn(*lead, C)


def check(x, G, w, b, dy, act, spans, over, k, dtype, eps=1e-5, inside=slice(None), **kw):
    C = x.shape[-1]
    flat = lambda t: f64(t).reshape(-1, C)  # noqa: E731
    with_stats = {}
    if over == "sequence":
        with_stats["stats"] = torch.full((len(spans), G, 2), 7.0, device="cuda")
    y = kda.group_norm_fwd(x, G, weight=w, bias=b, eps=eps, act=act, over=over, **kw, **with_stats)
    ref = norm(flat(x)[inside], G, f64(w), f64(b), eps, act, spans, over, k)
    within(y.reshape(-1, C)[inside], ref["y"], ref["y_err"], dtype, "y")
    if over == "sequence":
        assert np.allclose(f64(with_stats["stats"]), ref["stats"], rtol=1e-5, atol=1e-5)
    for gdtype in {dtype, F32}:
        dyt = dy.to(gdtype).cuda()
        ref = norm(flat(x)[inside], G, f64(w), f64(b), eps, act, spans, over, k, flat(dyt)[inside])
        for kept in ({}, with_stats):
            out = kda.group_norm_bwd(x, G, dyt, weight=w, bias=b, eps=eps, act=act, over=over, **kw, **kept)
            assert out["dx"].dtype == gdtype
            within(out["dx"].reshape(-1, C)[inside], ref["dx"], ref["dx_err"], gdtype, "dx")
            if w is not None:
                within(out["dweight"], ref["dweight"], ref["dweight_err"], F32, "dweight")
                within(out["dbias"], ref["dbias"], ref["dbias_err"], F32, "dbias")
            else:
                assert out["dweight"] is None and out["dbias"] is None
    return y


# tokens, C, groups: a team of one lane to a whole block, odd group sizes, every number of pieces a lane
TOKENS = [(1, 8, 1), (1, 1, 1), (3, 64, 8), (5, 96, 96), (7, 1530, 30), (1, 4096, 32), (33, 384, 3), (2, 12288, 96), (3, 5000, 1), (2, 12288, 1), (1, 16384, 1),
          (17, 700, 7), (300, 256, 2), (4, 2100, 2), (3, 4200, 1), (2, 4098, 2), (40, 40, 5), (1000, 16, 2), (3, 8192, 2), (2, 9001, 1), (513, 36, 4)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,C,G", TOKENS)
def test_over_tokens(T, C, G, dtype):
    act, affine, wide = (T + G) % 2, T % 3 != 0, 1 + T % 2
    x, w, b, dy = make((1, T), C, dtype, T + C, affine, wide)
    check(x, G, w, b, dy, act, [(0, T)], "token", 32, dtype)
    if T < 4:
        y2 = kda.group_norm_fwd(x[0], G, weight=w, bias=b, act=act)
        assert torch.equal(y2, kda.group_norm_fwd(x, G, weight=w, bias=b, act=act)[0])


SEQS = [([1], 8, 2), ([1, 1, 2], 30, 5), ([64], 64, 1), ([65, 0, 200, 3], 72, 9), ([1] * 90, 16, 4), ([700, 30, 5], 1530, 30), ([2500], 33, 3), ([300, 300], 512, 32),
        ([130], 4096, 32), ([40], 2048, 1), ([3000], 64, 8)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,C,G", SEQS)
def test_over_sequences(lens, C, G, dtype):
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    act, affine = T % 2, T % 3 != 0
    x, w, b, dy = make((1, T), C, dtype, T + C, affine, 1 + T % 2)
    k = 64 + T // 32 + T * C // G // 64 // 64
    check(x, G, w, b, dy, act, list(zip(cu, cu[1:])), "sequence", k, dtype, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("B,T,C,G", [(2, 96, 64, 4), (3, 1, 24, 3), (4, 250, 100, 10)])
def test_batches_of_sequences(B, T, C, G):
    x, w, b, dy = make((B, T), C, BF16, B + C, True)
    y = check(x, G, w, b, dy, 1, [(n * T, n * T + T) for n in range(B)], "sequence", 96, BF16)
    cu = torch.arange(B + 1, dtype=torch.int32, device="cuda") * T
    assert torch.equal(y.view(1, B * T, C), kda.group_norm_fwd(x.view(1, B * T, C), G, weight=w, bias=b, act=1, over="sequence", cu_seqlens=cu))


def test_rows_of_no_sequence():
    C, G, T, lo, hi = 48, 6, 150, 20, 101
    x, w, b, dy = make((1, T), C, F32, 3, True)
    x[:, :lo], x[:, hi:] = float("nan"), float("inf")
    dy[:, hi:] = float("nan")
    cu = torch.tensor([lo, 60, hi], dtype=torch.int32, device="cuda")
    y = torch.full((1, T, C), 3.0, device="cuda")
    check(x, G, w, b, dy, 1, [(0, 60 - lo), (60 - lo, hi - lo)], "sequence", 96, F32, inside=slice(lo, hi), cu_seqlens=cu)
    kda.group_norm_fwd(x, G, weight=w, bias=b, act=1, over="sequence", cu_seqlens=cu, y=y)
    assert bool((y[:, :lo] == 3).all()) and bool((y[:, hi:] == 3).all())
    dx = kda.group_norm_bwd(x, G, dy.cuda(), weight=w, bias=b, act=1, over="sequence", cu_seqlens=cu)["dx"]
    assert not bool(dx[:, :lo].any()) and not bool(dx[:, hi:].any())


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_means_far_from_zero_and_a_first_token_far_from_the_others(over):
    """The variance keeps its digits where the mean is a thousand deviations, and where the first token is."""
    T, C, G = 400, 64, 4
    x, w, b, dy = make((1, T), C, F32, 8, True)
    far = x + 1000.0
    check(far, G, w, b, dy, 0, [(0, T)], over, 96, F32)
    x[:, 0] *= 1000.0
    check(x, G, w, b, dy, 1, [(0, T)], over, 96, F32)


@pytest.mark.parametrize("over", ["token", "sequence"])
def test_constant_groups_and_not_a_number(over):
    """No variance at all: the deviation is eps alone.  A NaN stays in its group (and sequence)."""
    T, C, G = 70, 32, 4
    x = torch.full((1, T, C), 2.5, device="cuda")
    b = torch.randn(C, device="cuda")
    y = kda.group_norm_fwd(x, G, bias=b, over=over)
    assert torch.equal(y, b.expand(1, T, C))
    x, w, b, dy = make((1, T), C, F32, 9, True)
    clean = kda.group_norm_fwd(x, G, weight=w, bias=b, over=over)
    x[0, 10, 9] = float("nan")
    y = kda.group_norm_fwd(x, G, weight=w, bias=b, over=over)
    bad = torch.zeros(1, T, C, dtype=torch.bool)
    bad[0, (slice(10, 11) if over == "token" else slice(None)), 8:16] = True
    bad = bad.cuda()
    assert bool(torch.isnan(y[bad]).all()) and torch.equal(y[~bad], clean[~bad])


def test_differences():
    T, C, G = 12, 20, 4
    cu = [0, 5, 12]
    for over in ("token", "sequence"):
        for act in (0, 1):
            x, w, b, dy = make((1, T), C, F32, 21, True)
            kw = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda")) if over == "sequence" else {}
            out = kda.group_norm_bwd(x, G, dy.cuda(), weight=w, bias=b, act=act, over=over, **kw)
            base = {"x": f64(x)[0], "w": f64(w), "b": f64(b)}
            spans = list(zip(cu, cu[1:])) if over == "sequence" else [(0, T)]
            loss = lambda v: (norm(v["x"], G, v["w"], v["b"], 1e-5, act, spans, over, 1)["y"] * f64(dy)[0]).sum()  # noqa: E731
            ref = norm(base["x"], G, base["w"], base["b"], 1e-5, act, spans, over, 96, f64(dy)[0])
            rng = np.random.default_rng(0)
            for k, name in (("x", "dx"), ("w", "dweight"), ("b", "dbias")):
                way = rng.standard_normal(base[k].shape)
                diff = (loss({**base, k: base[k] + 1e-5 * way}) - loss({**base, k: base[k] - 1e-5 * way})) / 2e-5
                got = (f64(out[name]).reshape(way.shape) * way).sum()
                # the kernel's own error along the way, and the difference's: 1e-10 for its step, 1e-9 for its rounding, of values up to some hundred
                assert abs(got - diff) <= ((ref[name + "_err"] + 2.0 ** -24 * np.abs(ref[name])) * np.abs(way)).sum() + 1e-6, (over, act, name)


def test_same_bits_every_time_captured_and_on_another_stream():
    T, C, G = 500, 264, 11
    x, w, b, dy = make((1, T), C, BF16, 31, True)
    dy = dy.to(BF16).cuda()
    cu = torch.tensor([0, 100, 100, 500], dtype=torch.int32, device="cuda")

    def work():
        got = []
        for over, kw in (("token", {}), ("sequence", {"cu_seqlens": cu})):
            got.append(kda.group_norm_fwd(x, G, weight=w, bias=b, act=1, over=over, **kw))
            got += list(kda.group_norm_bwd(x, G, dy, weight=w, bias=b, act=1, over=over, **kw).values())
        return got
    want = [t.clone() for t in work()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert all(torch.equal(p, q) for p, q in zip(work(), want))
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(2):
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))


def test_nothing_to_do():
    x = torch.empty(0, 4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    assert kda.group_norm_fwd(x, 2).shape == x.shape
    for over in ("token", "sequence"):
        out = kda.group_norm_bwd(x, 2, x, weight=w, bias=w, over=over)
        assert not bool(out["dweight"].any()) and not bool(out["dbias"].any())
    x = torch.empty(2, 0, 8, device="cuda")
    stats = torch.zeros(2, 2, 2, device="cuda")
    kda.group_norm_fwd(x, 2, over="sequence", stats=stats)
    assert torch.allclose(stats[..., 1], torch.full((2, 2), 1e-5 ** -0.5, device="cuda"), rtol=1e-6) and not bool(stats[..., 0].any())
    x = torch.randn(1, 5, 8, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kda.group_norm_bwd(x, 2, x, weight=w, over="sequence", cu_seqlens=cu)
    assert not bool(out["dx"].any()) and not bool(out["dweight"].any())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,C,G", [(700, 6296, 1), (650, 2575, 5), (900, 4096, 1), (700, 4090, 2), (640, 3333, 1), (330, 9002, 1), (330, 12288, 1), (700, 2580, 5),
                                   (1500, 1032, 3), (700, 2451, 1), (700, 1060, 2), (2000, 600, 6)])
def test_many_rows_of_large_groups(T, C, G, dtype):
    """More rows than blocks, so that a block's next rows are under way while it works."""
    x, w, b, dy = make((1, T), C, dtype, T + C, True, 1 + T % 3)
    check(x, G, w, b, dy, 1, [(0, T)], "token", 32, dtype)
