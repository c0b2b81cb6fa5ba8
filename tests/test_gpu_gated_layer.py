"""The convolution, the group norm, the gated recurrence and a second norm as a layer runs them together: forward, backward, a prompt
and its tokens one by one on pages, forks, graphs."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests import gated_norm_ref as R
from tests.layer_ref import conv, f64

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32
C, G, W = 96, 6, 4
# A value passes some 2^6 roundings of 2^-24 on its way through the four operators; the two norms divide by deviations that are 2^-5 of
# what they are of or more.
CHAIN = 2.0 ** -24 * 2 ** 6 * 2 ** 5


def weights(seed):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    return dict(cw=rn(C, W) * 0.5, cb=rn(C) * 0.1, w1=1 + 0.1 * rn(C), b1=0.1 * rn(C), lam=rn(C) * 0.5 - 4.0, w2=1 + 0.1 * rn(C))


def inputs(shape, seed):
    g = torch.Generator().manual_seed(seed)
    return {k: torch.randn(*shape, C, generator=g) * s for k, s in (("x", 1.0), ("r", 1.5), ("i", 1.0), ("z", 1.5))}


def cuda(d, dtype=None):
    return {k: v.cuda() if dtype is None else v.to(dtype).cuda() for k, v in d.items()}


def forward(d, p, cu, **more):
    u, hist = kda.short_conv_fwd(d["x"], p["cw"], p["cb"], conv_act=1, cu_seqlens=cu)
    v = kda.group_norm_fwd(u, G, p["w1"], p["b1"], act=1)
    y, state = kda.gated_scan_fwd(v, d["r"], d["i"], p["lam"], z=d["z"], cu_seqlens=cu, **more)
    return u, v, y, kda.group_norm_fwd(y, G, p["w2"]), hist, state


def backward(d, p, cu, u, v, y, do, states=None):
    n2 = kda.group_norm_bwd(y, G, do, p["w2"])
    s = kda.gated_scan_bwd(v, d["r"], d["i"], p["lam"], n2["dx"], z=d["z"], cu_seqlens=cu, states=states)
    n1 = kda.group_norm_bwd(u, G, s["dx"], p["w1"], p["b1"], act=1)
    c = kda.short_conv_bwd(d["x"], p["cw"], n1["dx"], p["cb"], conv_act=1, cu_seqlens=cu)
    return dict(x=c["dx"], r=s["dr"], i=s["di"], z=s["dz"], cw=c["dweight"], cb=c["dbias"], w1=n1["dweight"], b1=n1["dbias"], lam=s["dlam"], w2=n2["dweight"])


def plain(d, p, cu):
    """The layer in 64 bits; d, p: numpy."""
    rows = {k: v.reshape(-1, C) for k, v in d.items()}
    T = rows["x"].shape[0]
    u = conv(rows["x"], p["cw"], p["cb"], 1, None, cu)[0]
    v = R.norm(u, G, p["w1"], p["b1"], 1e-5, 1, [(0, T)], "token", 0)["y"].reshape(T, C)
    y = R.gated(v, rows["r"], rows["i"], p["lam"], 8.0, rows["z"], None, cu)["y"]
    return R.norm(y, G, p["w2"], None, 1e-5, 0, [(0, T)], "token", 0)["y"].reshape(T, C)


def test_forward_and_backward():
    lens = [70, 1, 130]
    cu = [0, 70, 71, 201]
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    p, d = cuda(weights(1)), cuda(inputs((1, cu[-1]), 2))
    states = torch.empty(kda.gated_scan_states(d["x"]), device="cuda")
    u, v, y, o, _, _ = forward(d, p, off, states=states)
    p64, d64 = {k: f64(t) for k, t in p.items()}, {k: f64(t) for k, t in d.items()}
    want = plain(d64, p64, cu)
    assert (np.abs(f64(o).reshape(-1, C) - want) <= CHAIN * (1 + np.abs(want))).all()
    do = torch.randn(o.shape, generator=torch.Generator().manual_seed(3)).cuda()
    grads = backward(d, p, off, u, v, y, do, states)
    # every gradient against differences of the 64-bit form, along itself and along a line at random
    rng = np.random.default_rng(4)
    loss = lambda d, p: float((plain(d, p, cu) * f64(do).reshape(-1, C)).sum())  # noqa: E731
    for k, g in grads.items():
        g = f64(g)
        for line in (g / np.sqrt((g * g).sum()), rng.standard_normal(g.shape) / np.sqrt(g.size)):
            h = 1e-5
            side = lambda s: loss({**d64, k: d64[k] + s * line}, p64) if k in d64 else loss(d64, {**p64, k: p64[k] + s * line})  # noqa: E731,B023
            diff = (side(h) - side(-h)) / (2 * h)
            got = float((g * line).sum())
            # CHAIN of the gradient's length; the differences are off by h^2 times a third derivative, and by 2^-53 of the loss' terms over h
            assert abs(got - diff) <= 2 * CHAIN * np.sqrt((g * g).sum()) + 1e-7 * (1 + abs(diff)), (k, got, diff)
    again = backward(d, p, off, u, v, y, do, states)
    assert all(torch.equal(grads[k], again[k]) for k in grads) and len(lens) == 3


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_each_stage_in_its_type(dtype):
    """A batch in bf16 and fp32, a norm over sequences before the recurrence: every stage on what the one before gave."""
    B, T = 3, 65
    p, d = cuda(weights(5)), cuda(inputs((B, T), 6), dtype)
    cu = [0, T, 2 * T, 3 * T]
    u, _ = kda.short_conv_fwd(d["x"], p["cw"], p["cb"], conv_act=1)
    stats = torch.empty(B, G, 2, device="cuda")
    v = kda.group_norm_fwd(u, G, p["w1"], p["b1"], act=1, over="sequence", stats=stats)
    states = torch.empty(kda.gated_scan_states(v), device="cuda")
    y, state = kda.gated_scan_fwd(v, d["r"], d["i"], p["lam"], z=d["z"], states=states)
    do = torch.randn(y.shape, generator=torch.Generator().manual_seed(7)).to(dtype).cuda()
    s = kda.gated_scan_bwd(v, d["r"], d["i"], p["lam"], do, z=d["z"], states=states)
    n = kda.group_norm_bwd(u, G, s["dx"], p["w1"], p["b1"], act=1, over="sequence", stats=stats)
    rows = lambda t: f64(t).reshape(-1, C)  # noqa: E731
    spans = [(T * b, T * b + T) for b in range(B)]
    k = 60 + T * C // G // 64  # as sums over a sequence are taken: in parts of 64 rows and more
    ref = R.norm(rows(u), G, f64(p["w1"]), f64(p["b1"]), 1e-5, 1, spans, "sequence", k)
    R.within(v.reshape(-1, C), ref["y"], ref["y_err"], dtype, "v")
    ref = R.gated(rows(v), rows(d["r"]), rows(d["i"]), f64(p["lam"]), 8.0, rows(d["z"]), None, cu, rows(do))
    R.within(y.reshape(-1, C), ref["y"], ref["y_err"], dtype, "y")
    R.within(state, ref["state"], ref["state_err"], F32, "state")
    for name in ("dx", "dr", "di", "dz"):
        R.within(s[name].reshape(-1, C), ref[name], ref[name + "_err"], dtype, name)
    R.within(s["dlam"], ref["dlam"], ref["dlam_err"], F32, "dlam")
    ref = R.norm(rows(u), G, f64(p["w1"]), f64(p["b1"]), 1e-5, 1, spans, "sequence", k, rows(s["dx"]))
    R.within(n["dx"].reshape(-1, C), ref["dx"], ref["dx_err"], dtype, "norm dx")


def step(d, p, hist, state, slots):
    u = kda.short_conv_step(d["x"], hist, p["cw"], p["cb"], conv_act=1, slots=slots)
    v = kda.group_norm_fwd(u, G, p["w1"], p["b1"], act=1)
    y = kda.gated_step(v, d["r"], d["i"], p["lam"], state, z=d["z"], slots=slots)
    return kda.group_norm_fwd(y, G, p["w2"])


def test_prompts_then_tokens_on_pages():
    """Three prompts packed, then single tokens on pages taken from a pool, a padded row among them; one sequence forks."""
    lens, more, P = [20, 1, 33], 6, 9
    p = cuda(weights(8))
    seqs = [cuda(inputs((1, n + more), 9 + k)) for k, n in enumerate(lens)]
    packed = {k: torch.cat([s[k][:, :n] for s, n in zip(seqs, lens)], 1) for k in "xriz"}
    off = torch.tensor([0, 20, 21, 54], dtype=torch.int32, device="cuda")
    _, _, _, o, hist, state = forward(packed, p, off)
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    kda.pages_alloc(refs, 2)  # (somebody else's)
    pages = kda.pages_alloc(refs, 3)
    hists, pool = torch.full((P, W - 1, C), float("nan"), device="cuda"), torch.full((P, C), float("nan"), device="cuda")
    hists[pages.long()], pool[pages.long()] = hist, state
    outs = [[o[0, a:b]] for a, b in ((0, 20), (20, 21), (21, 54))]
    slots = torch.cat([pages, torch.tensor([-1], dtype=torch.int32, device="cuda")])
    rows = lambda t: {k: torch.cat([s[k][0, n + t:n + t + 1] for s, n in zip(seqs, lens)] + [torch.zeros(1, C, device="cuda")]) for k in "xriz"}  # noqa: E731
    for t in range(more):
        if t == 3:  # the third sequence's twin from here on
            twin = kda.pages_alloc(refs, 1)
            for cache in (hists, pool):
                kda.pages_copy(cache, pages[2:], twin)
            slots[3:] = twin
        d = rows(t)
        if t >= 3:
            d = {k: torch.cat([v[:3], v[2:3]]) for k, v in d.items()}
        got = step(d, p, hists, pool, slots)
        for k in range(3):
            outs[k].append(got[k:k + 1])
        if t >= 3:
            assert torch.equal(got[2], got[3])
    assert torch.equal(pool[twin.long()], pool[pages[2:].long()]) and torch.equal(hists[twin.long()], hists[pages[2:].long()])
    p64 = {k: f64(t) for k, t in p.items()}
    for s, out, n in zip(seqs, outs, lens):
        want = plain({k: f64(t) for k, t in s.items()}, p64, [0, n + more])
        got = f64(torch.cat(out))
        assert (np.abs(got - want) <= CHAIN * (1 + np.abs(want))).all()
    others = [k for k in range(P) if k not in pages.tolist() + twin.tolist()]
    assert bool(torch.isnan(pool[others]).all()) and bool(torch.isnan(hists[others]).all())


def test_captured_while_an_eager_one_runs():
    """A training step of the layer captured on one stream, replayed with new inputs while an eager step runs on another: the bits of
    steps by themselves."""
    cu = [0, 100, 164, 300]
    off = torch.tensor(cu, dtype=torch.int32, device="cuda")
    p = cuda(weights(20))
    sets = [cuda(inputs((1, 300), 21 + k), BF16) for k in range(3)]
    dos = [torch.randn(1, 300, C, generator=torch.Generator().manual_seed(k)).to(BF16).cuda() for k in range(3)]

    def train(d, do):
        states = torch.empty(kda.gated_scan_states(d["x"]), device="cuda")
        u, v, y, o, _, _ = forward(d, p, off, states=states)
        return {"o": o, **backward(d, p, off, u, v, y, do, states)}

    want = [train(d, do) for d, do in zip(sets, dos)]
    torch.cuda.synchronize()
    held, hdo = {k: v.clone() for k, v in sets[0].items()}, dos[0].clone()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        train(held, hdo)
        side.synchronize()
        with torch.cuda.graph(graph, stream=side):
            out = train(held, hdo)
    torch.cuda.synchronize()
    for k in (1, 2):
        with torch.cuda.stream(side):
            for name in held:
                held[name].copy_(sets[k][name])
            hdo.copy_(dos[k])
            graph.replay()
        with torch.cuda.stream(other):
            eager = [train(sets[0], dos[0]) for _ in range(3)]
        torch.cuda.synchronize()
        assert all(torch.equal(out[n], want[k][n]) for n in out)
        assert all(torch.equal(e[n], want[0][n]) for e in eager for n in e)
