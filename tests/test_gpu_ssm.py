"""The selective state space scan (prompts, their backward pass, single tokens) against its plain
64-bit form.

Tolerances, element by element.  The step size d is off by 2^-21 relative (softplus: one exponential,
2^-22, and a series), and the decay's exponent d A by as much of itself plus a rounding, so the decay is off
by |d A| 2^-20 + 2^-22 relative; with the products' roundings a state is off by
2^-19 (|a h| (1 + |d A|) + |d u B|) per step.  y adds S products and D u, each rounded, and the gate's
relative 2^-20 |z| + 2^-21.

Over a prompt these errors follow the recurrences: `layer_ref.scan` carries along, for every state,
gradient and sum, the sum of the magnitudes that a relative error of 2^-19 of each part is taken of (the
decay's part 1 + |d A| times).  Cutting the tokens into runs adds one rounded decay product a run, below what
the per-token parts already count.  Sums over n terms in fp32 add n 2^-24 of the sum of magnitudes."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.layer_ref import f64, half_step, scan, silu, softplus

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


LARGEST = 3.3e38   # below the largest fp32 and bf16 numbers


def within(got, ref, tol, dtype, largest=None):
    """largest: the largest magnitude among what each value is computed from.  One beyond fp32's range (a
    growing state: step sizes below zero, without softplus) has no result to be compared."""
    got = f64(got).reshape(ref.shape)
    if largest is not None:
        has = largest < LARGEST
        got, ref, tol = got[has], ref[has], tol[has]
    assert np.isfinite(got).all()
    off = np.abs(got - ref) - (half_step(dtype) * np.abs(ref) + tol * (1 + half_step(dtype)) + 1e-30)
    assert (off <= 0).all(), f"off by up to {off.max():.3e} more than allowed, {int((off > 0).sum())} values"


def make(lead, C, S, G, dtype, seed, gate, D, bias):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
    bc = rn(*lead, 2, G, S).to(dtype).cuda()
    return dict(u=rn(*lead, C).to(dtype).cuda(), delta=(rn(*lead, C) * 2 - 2).to(dtype).cuda(), A=-torch.exp(rn(C, S)).cuda(),
                B=bc[..., 0, :, :], C=bc[..., 1, :, :], D=rn(C).cuda() if D else None, z=(rn(*lead, C) * 2).to(dtype).cuda() if gate else None,
                bias=(rn(C) - 1).cuda() if bias else None)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,C,S,G,gate,D,bias,sp", [(1, 1, 8, 1, True, True, True, True), (3, 37, 16, 1, True, False, True, True),
                                                    (2, 130, 64, 2, False, True, False, True), (5, 66, 32, 3, True, True, True, False),
                                                    (40, 4096, 16, 1, True, True, True, True), (300, 1030, 8, 5, True, True, True, True)])
def test_step(N, C, S, G, gate, D, bias, sp, dtype):
    d = make((N,), C, S, G, dtype, 800 + N, gate, D, bias)
    if not sp:
        d["delta"] = d["delta"].abs()
    P = N + 3
    g = torch.Generator().manual_seed(N)
    slots = torch.randperm(P, generator=g)[:N].to(torch.int32).cuda()
    pool = torch.randn(P, C, S, generator=g).cuda()
    before = f64(pool)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    y = kda.ssm_step(d["u"], d["delta"], d["A"], d["B"], d["C"], pool, D=d["D"], z=d["z"], delta_bias=d["bias"], softplus=sp, slots=slots,
                     status=status)
    u, raw, A = f64(d["u"]), f64(d["delta"]) + (f64(d["bias"]) if bias else 0), f64(d["A"])
    dl = softplus(raw) if sp else raw
    grp = np.arange(C) // (C // G)
    Bx, Cx = f64(d["B"])[:, grp], f64(d["C"])[:, grp]
    dA = dl[..., None] * A
    at = slots.cpu().numpy()
    ah, b = np.exp(dA) * before[at], (dl * u)[..., None] * Bx
    h = ah + b
    th = 2.0 ** -19 * (np.abs(ah) * (1 + np.abs(dA)) + np.abs(b))
    lin = (Cx * h).sum(-1) + (f64(d["D"]) * u if D else 0)
    mag = (np.abs(Cx * h)).sum(-1) + (np.abs(f64(d["D"]) * u) if D else 0)
    tol = (np.abs(Cx) * th).sum(-1) + (S + 3) * 2.0 ** -24 * mag
    ref = lin
    if gate:
        z = f64(d["z"])
        ref = lin * silu(z)
        tol = tol * np.abs(silu(z)) + np.abs(ref) * (2.0 ** -20 * np.abs(z) + 2.0 ** -21)
    grown = np.maximum(np.exp(dA), np.abs(ah) + np.abs(b))
    within(y, ref, tol, dtype, np.maximum(mag, grown.max(-1)) * np.maximum(1, np.abs(silu(f64(d["z"])) if gate else 1)))
    within(pool[slots.long()], h, th, F32, grown)
    assert int(status) == 0
    rest = np.setdiff1d(np.arange(P), at)
    assert np.array_equal(f64(pool)[rest], before[rest])


def test_step_without_slots_equals_with():
    d = make((6,), 96, 16, 1, BF16, 830, True, True, True)
    a = torch.randn(6, 96, 16, device="cuda")
    b = a.clone()
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["bias"])
    y1 = kda.ssm_step(d["u"], d["delta"], d["A"], d["B"], d["C"], a, **kw)
    y2 = kda.ssm_step(d["u"], d["delta"], d["A"], d["B"], d["C"], b, slots=torch.arange(6, dtype=torch.int32, device="cuda"), **kw)
    assert torch.equal(y1, y2) and torch.equal(a, b)


def test_step_pads_and_refuses():
    d = make((6,), 40, 8, 1, F32, 831, False, False, False)
    pool = torch.randn(4, 40, 8, device="cuda")
    before = pool.clone()
    y = torch.full((6, 40), 9.0, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([-1, 2, 2, 4, -7, 0], dtype=torch.int32, device="cuda")
    kda.ssm_step(d["u"], d["delta"], d["A"], d["B"], d["C"], pool, slots=slots, y=y, status=status)
    want = before[[2, 0]].clone()
    rows = [1, 5]
    wy = kda.ssm_step(d["u"][rows], d["delta"][rows], d["A"], d["B"][rows], d["C"][rows], want)
    assert int(status) == 5 and torch.equal(y[rows], wy) and bool((y[[0, 2, 3, 4]] == 9).all())
    before[[2, 0]] = want
    assert torch.equal(pool, before)


def test_step_sizes_at_the_ends():
    """softplus far below, around and far above zero, and a decay that underflows."""
    raw = torch.tensor([-200.0, -90.0, -30.0, -10.0, -1e-6, 0.0, 1e-6, 15.0, 30.0, 1e4, 3e38, float("-inf")], device="cuda")
    C = raw.numel()
    A = torch.full((C, 8), -1.0, device="cuda")
    one = torch.ones(1, 1, 8, device="cuda")
    pool = torch.full((1, C, 8), 2.0, device="cuda")
    kda.ssm_step(torch.ones(1, C, device="cuda"), raw[None], A, one, one, pool)
    dl = softplus(f64(raw))
    want = np.exp(-dl) * 2 + dl
    assert np.allclose(f64(pool)[0, :, 0], want, rtol=2e-6, atol=0)


# lengths, C, S, G, gate, D, bias, softplus, state, wide
SCANS = [
    ([1], 8, 16, 1, True, True, True, True, False),
    ([64], 40, 16, 1, True, True, True, True, True),
    ([65, 1, 63], 130, 16, 1, False, True, True, True, True),
    ([0, 3, 0, 0, 9, 1, 90, 0], 36, 8, 2, True, False, True, True, True),
    ([31, 33, 129], 70, 32, 2, True, True, False, True, True),
    ([200], 24, 64, 3, True, True, True, True, False),
    ([1] * 30 + [17] * 6, 129, 16, 1, True, True, True, True, True),
    ([300, 5], 260, 16, 1, False, False, False, False, True),
    ([130], 1, 64, 1, True, True, True, True, True),
    # blocks enough that the backward pass takes chunks of 64 tokens (above, 16), and of 32
    ([130, 70, 1, 64, 35], 600, 16, 300, True, True, True, True, True),
    ([400], 330, 8, 330, False, True, False, True, False),
    ([31, 65, 0, 40, 128, 3], 270, 32, 90, True, False, True, True, True),
    ([200, 64], 1300, 64, 1, True, True, True, True, False),
]


def scan_inputs(case, dtype, seed):
    lengths, C, S, G, gate, D, bias, sp, state = SCANS[case]
    d = make((1, sum(lengths)), C, S, G, dtype, seed, gate, D, bias)
    if not sp:
        d["delta"] = (d["delta"].float().abs() * 0.3).to(dtype)
    g = torch.Generator().manual_seed(seed + 1)
    N = len(lengths)
    d["s0"] = torch.randn(N, C, S, generator=g).cuda() if state else None
    d["cu"] = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    d["dy"] = torch.randn(1, sum(lengths), C, generator=g)
    d["df"] = torch.randn(N, C, S, generator=g).cuda() if state else None
    d["sp"] = sp
    return d


def call_args(d):
    return (d["u"], d["delta"], d["A"], d["B"], d["C"]), dict(D=d["D"], z=d["z"], delta_bias=d["bias"], softplus=d["sp"],
                                                             initial_state=d["s0"], cu_seqlens=d["cu"])


def ref_args(d):
    one = lambda t: None if t is None else f64(t)[0]  # noqa: E731
    return (one(d["u"]), one(d["delta"]), f64(d["A"]), one(d["B"]), one(d["C"]), f64(d["D"]), one(d["z"]), f64(d["bias"]), d["sp"],
            f64(d["s0"]), d["cu"].tolist())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("case", range(len(SCANS)))
def test_scan(case, dtype):
    d = scan_inputs(case, dtype, 900 + case)
    a, kw = call_args(d)
    y, state = kda.ssm_scan_fwd(*a, **kw)
    r = scan(*ref_args(d))
    S = d["A"].shape[1]
    within(y[0], r["y"], (2.0 ** -19 + S * 2.0 ** -24) * r["y_err"], dtype)
    within(state, r["state"], 2.0 ** -19 * r["state_err"], F32)


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("case", range(len(SCANS)))
def test_scan_backward(case, dtype, gdtype):
    d = scan_inputs(case, dtype, 950 + case)
    a, kw = call_args(d)
    dy = d["dy"].to(gdtype).cuda()
    got = kda.ssm_scan_bwd(*a, dy, dfinal_state=d["df"], **kw)
    r = scan(*ref_args(d), f64(dy)[0], f64(d["df"]))
    T, C = dy.shape[1:]
    S = d["A"].shape[1]
    for k, dt, n in (("du", gdtype, S), ("ddelta", gdtype, S), ("dz", gdtype, S), ("dB", gdtype, C), ("dC", gdtype, C), ("dA", F32, T),
                     ("dD", F32, T), ("ddelta_bias", F32, T), ("dinitial_state", F32, 1)):
        given = {"dz": d["z"], "dD": d["D"], "ddelta_bias": d["bias"], "dinitial_state": d["s0"]}.get(k, d["u"]) is not None
        assert (got[k] is not None) == given, k
        if given:
            within(got[k], r[k], (2.0 ** -19 + n * 2.0 ** -24) * r[k + "_err"], dt)


def test_scan_backward_against_differences():
    """Along random directions of every argument: the loss is smooth, steps of 1e-2 leave a relative truncation
    of 1e-4 of the magnitudes, and the forward's rounding 2^-18 / 1e-2."""
    d = scan_inputs(1, F32, 990)
    a, kw = call_args(d)
    dy = d["dy"].cuda()
    got = kda.ssm_scan_bwd(*a, dy, dfinal_state=d["df"], **kw)
    names = ["u", "delta", "A", "B", "C", "D", "z", "bias", "s0"]
    grads = ["du", "ddelta", "dA", "dB", "dC", "dD", "dz", "ddelta_bias", "dinitial_state"]

    def loss(v):
        y, s = kda.ssm_scan_fwd(v["u"], v["delta"], v["A"], v["B"], v["C"], D=v["D"], z=v["z"], delta_bias=v["bias"],
                                initial_state=v["s0"], cu_seqlens=d["cu"])
        return float((y.double() * dy.double()).sum() + (s.double() * d["df"].double()).sum())
    g = torch.Generator().manual_seed(991)
    for name, grad in zip(names, grads):
        way = torch.randn(d[name].shape, generator=g).cuda()
        slope = (loss({**d, name: (d[name] + 1e-2 * way).contiguous()}) - loss({**d, name: (d[name] - 1e-2 * way).contiguous()})) / 2e-2
        terms = got[grad].reshape(way.shape).double() * way.double()
        assert abs(slope - float(terms.sum())) <= 2e-3 * (float(terms.abs().sum()) + 1.0), name


def test_long_run_of_slow_decay():
    """Several runs of one sequence, channels that hardly forget: the state in 64 bits on the device."""
    T, C, S = 5000, 40, 16
    g = torch.Generator().manual_seed(992)
    u, delta = torch.randn(1, T, C, generator=g).cuda(), (torch.rand(1, T, C, generator=g) * 0.01).cuda()
    A = -(torch.arange(S).float() * 0.1).repeat(C, 1).cuda()          # a rate of zero among them
    B, Cm = torch.randn(1, T, 1, S, generator=g).cuda(), torch.randn(1, T, 1, S, generator=g).cuda()
    y, state = kda.ssm_scan_fwd(u, delta, A, B, Cm, softplus=False)
    h = torch.zeros(C, S, dtype=torch.float64, device="cuda")
    ys, mag, peak = [], torch.zeros_like(h), 0.0
    for t in range(T):
        x = delta[0, t].double()[:, None] * A.double()
        b = (delta[0, t] .double() * u[0, t].double())[:, None] * B[0, t].double()
        h = torch.exp(x) * h + b
        mag = torch.exp(x) * mag + b.abs() + h.abs()
        ys.append((h * Cm[0, t].double()).sum(-1))
    want = torch.stack(ys)
    off = (state[0].double() - h).abs() / mag
    assert float(off.max()) <= 2.0 ** -22      # each step rounds the state once and its decay by 2^-22 of a small exponent
    assert float((y[0].double() - want).abs().max()) <= 1e-4 * float(want.abs().max())


def test_scan_dense_equals_packed_and_leaves_other_rows():
    d = make((3, 50), 72, 16, 1, BF16, 993, True, True, True)
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["bias"])
    y, s = kda.ssm_scan_fwd(d["u"], d["delta"], d["A"], d["B"].contiguous(), d["C"].contiguous(), **kw)
    flat = lambda t: t.contiguous().reshape(1, 150, *t.shape[2:])  # noqa: E731
    cu = torch.tensor([0, 50, 100, 150], dtype=torch.int32, device="cuda")
    args = [flat(d["u"]), flat(d["delta"]), d["A"], flat(d["B"]), flat(d["C"])]
    y2, s2 = kda.ssm_scan_fwd(*args, D=d["D"], z=flat(d["z"]), delta_bias=d["bias"], cu_seqlens=cu)
    assert torch.equal(y.view(1, 150, 72), y2) and torch.equal(s, s2)
    cu = torch.tensor([7, 50, 140], dtype=torch.int32, device="cuda")
    y3 = torch.full_like(y2, 5.0)
    kda.ssm_scan_fwd(*args, D=d["D"], z=flat(d["z"]), delta_bias=d["bias"], cu_seqlens=cu, y=y3)
    assert bool((y3[0, :7] == 5).all()) and bool((y3[0, 140:] == 5).all())
    assert torch.equal(y3[0, 50:100], y2[0, 50:100])       # a sequence of the same start
    got = kda.ssm_scan_bwd(*args, y2, D=d["D"], z=flat(d["z"]), delta_bias=d["bias"], cu_seqlens=cu)
    assert all(bool(got[k].isfinite().all()) for k in ("dA", "dD", "ddelta_bias"))


def test_scan_without_tokens():
    e = torch.empty(1, 0, 24, device="cuda")
    v = torch.empty(1, 0, 1, 16, device="cuda")
    A = -torch.ones(24, 16, device="cuda")
    s0 = torch.randn(2, 24, 16, device="cuda")
    cu = torch.zeros(3, dtype=torch.int32, device="cuda")
    y, s = kda.ssm_scan_fwd(e, e, A, v, v, initial_state=s0, cu_seqlens=cu)
    assert torch.equal(s, s0) and y.numel() == 0
    got = kda.ssm_scan_bwd(e, e, A, v, v, e, initial_state=s0, cu_seqlens=cu, dfinal_state=s0)
    assert torch.equal(got["dinitial_state"], s0) and not got["dA"].any()


@pytest.mark.parametrize("case", [5, 9, 11])
def test_scan_offsets_out_of_order_stay_in_bounds(case):
    d = scan_inputs(case, BF16, 994)
    s0 = torch.randn(4, *d["A"].shape, device="cuda")
    a, kw = call_args(d)
    for cu in ([0, 150, 50, 180, 200], [0, -5, 900, 20, 200], [200, 0, 200, 0, 7], [2 ** 31 - 1, -2 ** 31, 5, 6, 2 ** 31 - 1]):
        kw["initial_state"], kw["cu_seqlens"] = s0, torch.tensor(cu, dtype=torch.int32, device="cuda")
        y, _ = kda.ssm_scan_fwd(*a, **kw)
        kda.ssm_scan_bwd(*a, y, dfinal_state=s0, **kw)
    torch.cuda.synchronize()


def test_steps_continue_a_scan():
    """Prefill into a pool and single tokens from there, as the whole prompt."""
    d = make((4, 20), 200, 16, 1, F32, 995, True, True, True)
    kw = dict(D=d["D"], delta_bias=d["bias"])
    args = lambda sl: [x[:, sl].contiguous() for x in (d["u"], d["delta"], d["B"], d["C"], d["z"])]  # noqa: E731
    u, dl, B, C, z = args(slice(None))
    whole, last = kda.ssm_scan_fwd(u, dl, d["A"], B, C, z=z, **kw)
    u, dl, B, C, z = args(slice(0, 12))
    _, state = kda.ssm_scan_fwd(u, dl, d["A"], B, C, z=z, **kw)
    pool = torch.zeros(7, 200, 16, device="cuda")
    slots = torch.tensor([5, 0, 3, 6], dtype=torch.int32, device="cuda")
    pool[slots.long()] = state
    for t in range(12, 20):
        y = kda.ssm_step(d["u"][:, t], d["delta"][:, t], d["A"], d["B"][:, t], d["C"][:, t], pool, z=d["z"][:, t], slots=slots, **kw)
        torch.testing.assert_close(y, whole[:, t], rtol=1e-5, atol=1e-5)
    torch.testing.assert_close(pool[slots.long()], last, rtol=1e-5, atol=1e-5)


def test_layer_of_convolution_and_scan():
    """The convolution's output into the scan and their gradients back through both, packed, against the plain
    forms chained: bf16 between them, so within the steps of its roundings."""
    from tests.layer_ref import conv
    lengths, C = [40, 70, 1], 64
    d = make((1, 111), C, 16, 1, F32, 996, True, True, True)
    w = (torch.randn(C, 4, generator=torch.Generator().manual_seed(3)) * 0.5).cuda()
    cu = torch.tensor([0, 40, 110, 111], dtype=torch.int32, device="cuda")
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["bias"], cu_seqlens=cu)
    x, _ = kda.short_conv_fwd(d["u"], w, conv_act=1, cu_seqlens=cu)
    y, _ = kda.ssm_scan_fwd(x, d["delta"], d["A"], d["B"], d["C"], **kw)
    dy = torch.randn(1, 111, C, generator=torch.Generator().manual_seed(4)).cuda()
    back = kda.ssm_scan_bwd(x, d["delta"], d["A"], d["B"], d["C"], dy, **kw)
    got = kda.short_conv_bwd(d["u"], w, back["du"], conv_act=1, cu_seqlens=cu)
    rx, _, _ = conv(f64(d["u"])[0], f64(w), None, 1, None, cu.tolist())
    d2 = dict(d, sp=True, s0=None, cu=cu)
    args = list(ref_args(d2))
    args[0] = rx
    r = scan(*args, f64(dy)[0], None)
    rg = conv(f64(d["u"])[0], f64(w), None, 1, None, cu.tolist(), r["du"], None)
    within(y[0], r["y"], 2.0 ** -17 * r["y_err"], F32)
    scale = np.abs(r["du_err"]).max() * np.abs(f64(w)).sum(1).max()
    assert np.abs(f64(got["dx"])[0] - rg["dx"]).max() <= 2.0 ** -17 * scale * 2
    assert np.abs(f64(got["dweight"]) - rg["dweight"]).max() <= 2.0 ** -17 * scale * 111


@pytest.mark.parametrize("case", [6, 9])
def test_scan_captured_and_replayed_on_another_stream(case):
    d = scan_inputs(case, BF16, 997)
    a, kw = call_args(d)
    dy = d["dy"].to(BF16).cuda()
    want, ws = kda.ssm_scan_fwd(*a, **kw)
    wg = kda.ssm_scan_bwd(*a, dy, dfinal_state=d["df"], **kw)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        y, s = kda.ssm_scan_fwd(*a, **kw)
        g = kda.ssm_scan_bwd(*a, dy, dfinal_state=d["df"], **kw)
    side.synchronize()
    assert torch.equal(y, want) and torch.equal(s, ws) and all(torch.equal(g[k], wg[k]) for k in wg if wg[k] is not None)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, s = kda.ssm_scan_fwd(*a, **kw)
        g = kda.ssm_scan_bwd(*a, dy, dfinal_state=d["df"], **kw)
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(y, want) and torch.equal(s, ws) and all(torch.equal(g[k], wg[k]) for k in wg if wg[k] is not None)


@pytest.mark.parametrize("C,G", [(72, 1), (180, 90), (680, 340)])     # chunks of 16, 32 and 64 tokens backwards
def test_scan_nan_and_infinity_stay_in_their_sequence(C, G):
    """A sequence with NaN and infinite inputs in one chunk with others: theirs are as without it, bit for bit,
    forwards and backwards (the sums over everything apart)."""
    lengths = [40, 9, 50, 64, 37]
    d = make((1, 200), C, 16, G, F32, 998, True, True, True)
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32, device="cuda")
    s0 = torch.randn(5, C, 16, generator=torch.Generator().manual_seed(5)).cuda()
    dy = torch.randn(1, 200, C, generator=torch.Generator().manual_seed(6)).cuda()
    kw = dict(D=d["D"], z=d["z"], delta_bias=d["bias"], initial_state=s0, cu_seqlens=cu)

    def run(u, delta, grad):
        y, s = kda.ssm_scan_fwd(u, delta, d["A"], d["B"], d["C"], **kw)
        g = kda.ssm_scan_bwd(u, delta, d["A"], d["B"], d["C"], grad, dfinal_state=s0, **kw)
        return y, s, g
    y, s, g = run(d["u"], d["delta"], dy)
    for at in (range(0, 40), range(40, 49), range(99, 163)):
        u, delta, grad = d["u"].clone(), d["delta"].clone(), dy.clone()
        t = at[len(at) // 2]
        u[0, t, 3], delta[0, t, 4], grad[0, t, 5], delta[0, t, 6], u[0, t, 7] = (float("nan"),) * 3 + (float("inf"),) * 2
        y2, s2, g2 = run(u, delta, grad)
        n = [0, 40, 49, 99, 163].index(at[0])
        others = torch.ones(200, dtype=torch.bool)
        others[list(at)] = False
        rest = [i for i in range(5) if i != n]
        assert torch.equal(y[0, others], y2[0, others]) and torch.equal(s[rest], s2[rest])
        for k in ("du", "ddelta", "dz", "dB", "dC"):
            assert torch.equal(g[k][0, others], g2[k][0, others]), k
        assert torch.equal(g["dinitial_state"][rest], g2["dinitial_state"][rest])
        clean = [c for c in range(C) if c not in (3, 4, 5, 6, 7)]
        assert torch.equal(y[0][:, clean], y2[0][:, clean]) and torch.equal(g["du"][0][:, clean], g2["du"][0][:, clean])


def test_scan_many_short_sequences():
    """More sequences than one round of the search for boundaries looks at."""
    rng = np.random.default_rng(9)
    lengths = rng.integers(0, 4, 3000)
    T, C = int(lengths.sum()), 24
    d = make((1, T), C, 8, 1, F32, 999, False, True, True)
    cu = np.concatenate([[0], np.cumsum(lengths)])
    s0 = torch.randn(3000, C, 8, generator=torch.Generator().manual_seed(7)).cuda()
    dy = torch.randn(1, T, C, generator=torch.Generator().manual_seed(8)).cuda()
    kw = dict(D=d["D"], delta_bias=d["bias"], initial_state=s0, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    y, s = kda.ssm_scan_fwd(d["u"], d["delta"], d["A"], d["B"], d["C"], **kw)
    got = kda.ssm_scan_bwd(d["u"], d["delta"], d["A"], d["B"], d["C"], dy, **kw)
    args = ref_args(dict(d, sp=True, s0=s0, cu=torch.tensor(cu)))
    r = scan(*args, f64(dy)[0], None)
    within(y[0], r["y"], 2.0 ** -18 * r["y_err"], F32)
    within(s, r["state"], 2.0 ** -19 * r["state_err"], F32)
    for k, n in (("du", 8), ("ddelta", 8), ("dB", C), ("dC", C), ("dinitial_state", 1), ("dA", T)):
        within(got[k], r[k], (2.0 ** -19 + n * 2.0 ** -24) * r[k + "_err"], F32)


def test_rows_far_apart():
    """Rows whose offsets pass 2^31 elements, as slices of one wide buffer."""
    T, C, wide = 2100, 40, (1 << 20) + 8
    buf = torch.zeros(1, T, wide, dtype=BF16, device="cuda")
    d = make((1, T), C, 8, 1, BF16, 1000, True, True, True)
    v = lambda i: buf[:, :, i * 64:i * 64 + C]  # noqa: E731
    for i, k in enumerate(("u", "delta", "z")):
        v(i).copy_(d[k])
    bc = buf[:, :, 512:528].unflatten(2, (2, 1, 8))
    bc[:, :, 0].copy_(d["B"])
    bc[:, :, 1].copy_(d["C"])
    kw = dict(D=d["D"], delta_bias=d["bias"])
    want, ws = kda.ssm_scan_fwd(d["u"], d["delta"], d["A"], d["B"].contiguous(), d["C"].contiguous(), z=d["z"], **kw)
    y, s = kda.ssm_scan_fwd(v(0), v(1), d["A"], bc[:, :, 0], bc[:, :, 1], z=v(2), **kw)
    assert torch.equal(y, want) and torch.equal(s, ws)
    wg = kda.ssm_scan_bwd(d["u"], d["delta"], d["A"], d["B"].contiguous(), d["C"].contiguous(), want, z=d["z"], **kw)
    g = kda.ssm_scan_bwd(v(0), v(1), d["A"], bc[:, :, 0], bc[:, :, 1], want, z=v(2), **kw)
    assert all(torch.equal(g[k], wg[k]) for k in wg if wg[k] is not None)
    w = torch.randn(C, 4, device="cuda")
    assert torch.equal(kda.short_conv_fwd(v(0), w, conv_act=1)[0], kda.short_conv_fwd(d["u"], w, conv_act=1)[0])
    a, b = kda.short_conv_bwd(v(0), w, want, conv_act=1), kda.short_conv_bwd(d["u"], w, want, conv_act=1)
    assert torch.equal(a["dx"], b["dx"]) and torch.equal(a["dweight"], b["dweight"])
