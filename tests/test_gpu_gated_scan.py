"""The gated linear recurrence (prompts, their backward pass, single tokens) against its plain 64-bit form; the tolerances are
derived in gated_norm_ref."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.gated_norm_ref import f64, gated, within

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def make(lead, C, dtype, seed, gate, wide=1):
    g = torch.Generator().manual_seed(seed)
    rn = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
    rows = lambda std: (rn(*lead, wide * C) * std).to(dtype).cuda()[..., :C]  # noqa: E731
    a = 0.5 + 0.499 * torch.rand(C, generator=g)
    return dict(x=rows(1.0), r=rows(2.0), i=rows(1.5), z=rows(2.0) if gate else None, lam=torch.log(torch.expm1(-torch.log(a) / 8.0)).cuda())


def offsets(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def flat(t, C):
    return None if t is None else f64(t).reshape(-1, C)


def ref_of(d, C, initial, cu, dy=None, dfinal=None, decay=8.0):
    return gated(flat(d["x"], C), flat(d["r"], C), flat(d["i"], C), f64(d["lam"]), decay, flat(d["z"], C), f64(initial), cu,
                 flat(dy, C), f64(dfinal))


def args(d):
    return d["x"], d["r"], d["i"], d["lam"]


FORMS = [  # lens, C, gate, initial states, rows of wider ones
    ([1], 1, True, True, 1), ([1], 64, False, False, 1), ([2, 1], 66, True, True, 1), ([31, 33], 7, False, True, 1), ([64], 128, True, False, 1),
    ([65, 0, 127, 1, 3], 72, True, True, 1), ([1] * 70, 34, True, True, 1), ([300, 5, 260], 200, True, True, 2), ([700], 1530, True, True, 1),
    ([2000], 70, False, True, 1), ([513, 40, 600], 264, True, True, 3),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,C,gate,state,wide", FORMS)
def test_packed(lens, C, gate, state, wide, dtype):
    T, N = sum(lens), len(lens)
    d = make((1, T), C, dtype, 100 + T + C, gate, wide)
    g = torch.Generator().manual_seed(T)
    initial = torch.randn(N, C, generator=g).cuda() if state else None
    cu = offsets(lens)
    states = torch.full(kda.gated_scan_states(d["x"]), 7.0, device="cuda")
    y, final = kda.gated_scan_fwd(*args(d), z=d["z"], initial_state=initial, cu_seqlens=cu, states=states)
    dy = torch.randn(1, T, C, generator=g).to(dtype).cuda()
    dfinal = torch.randn(N, C, generator=g).cuda() if state else None
    ref = ref_of(d, C, initial, cu.tolist(), dy, dfinal)
    within(y, ref["y"], ref["y_err"], dtype, "y")
    within(final, ref["state"], ref["state_err"], F32, "state")
    within(states, ref["before"][::32], ref["before_err"][::32], F32, "states")
    for kept in (states, None):
        out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], initial_state=initial, cu_seqlens=cu, dfinal_state=dfinal, states=kept)
        for k in ("dx", "dr", "di") + (("dz",) if gate else ()):
            within(out[k], ref[k], ref[k + "_err"], dtype, k)
        within(out["dlam"], ref["dlam"], ref["dlam_err"], F32, "dlam")
        if state:
            within(out["dinitial_state"], ref["dinitial_state"], ref["dinitial_state_err"], F32, "dinitial")
        assert (out["dz"] is None) == (not gate) and (out["dinitial_state"] is None) == (not state)


@pytest.mark.parametrize("dtype,gdtype", [(BF16, BF16), (BF16, F32), (F32, F32)])
@pytest.mark.parametrize("B,T,C,gate,state", [(1, 1, 16, True, False), (3, 1, 130, False, True), (2, 96, 64, True, True), (2, 250, 100, True, False),
                                              (5, 33, 9, False, True), (1, 1100, 320, True, True)])
def test_batches(B, T, C, gate, state, dtype, gdtype):
    d = make((B, T), C, dtype, 900 + T + C, gate)
    g = torch.Generator().manual_seed(C)
    initial = torch.randn(B, C, generator=g).cuda() if state else None
    dfinal = torch.randn(B, C, generator=g).cuda() if state else None
    dy = torch.randn(B, T, C, generator=g).to(gdtype).cuda()
    cu = [b * T for b in range(B + 1)]
    ref = ref_of(d, C, initial, cu, dy, dfinal)
    states = torch.empty(kda.gated_scan_states(d["x"]), device="cuda")
    y, final = kda.gated_scan_fwd(*args(d), z=d["z"], initial_state=initial, states=states)
    within(y, ref["y"], ref["y_err"], dtype, "y")
    within(final, ref["state"], ref["state_err"], F32, "state")
    within(states, ref["before"].reshape(B, T, C)[:, ::32], ref["before_err"].reshape(B, T, C)[:, ::32], F32, "states")
    for kept in (states, None):
        out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], initial_state=initial, dfinal_state=dfinal, states=kept)
        for k in ("dx", "dr", "di") + (("dz",) if gate else ()):
            assert out[k].dtype == gdtype
            within(out[k], ref[k], ref[k + "_err"], gdtype, k)
        within(out["dlam"], ref["dlam"], ref["dlam_err"], F32, "dlam")
        if state:
            within(out["dinitial_state"], ref["dinitial_state"], ref["dinitial_state_err"], F32, "dinitial")


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,C,gate", [(1, 1, True), (3, 37, False), (5, 64, True), (40, 4096, True), (300, 1030, True), (2, 130, False)])
def test_step(N, C, gate, dtype):
    d = make((N,), C, dtype, 50 + N, gate)
    P = N + 3
    g = torch.Generator().manual_seed(N)
    slots = torch.randperm(P, generator=g)[:N].to(torch.int32).cuda()
    pool = torch.randn(P, C, generator=g).cuda()
    before = pool.clone()
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    y = kda.gated_step(*args(d), pool, z=d["z"], slots=slots, status=status)
    ref = ref_of(d, C, before[slots.long()], list(range(N + 1)))
    within(y, ref["y"], ref["y_err"], dtype, "y")
    within(pool[slots.long()], ref["state"], ref["state_err"], F32, "state")
    assert int(status) == 0
    before[slots.long()] = pool[slots.long()]
    assert torch.equal(pool, before)
    again = before[slots.long()].contiguous()
    rows = kda.gated_step(*args(d), again, z=d["z"])
    pool2 = before.clone()
    assert torch.equal(rows, kda.gated_step(*args(d), pool2, z=d["z"], slots=slots)) and torch.equal(again, pool2[slots.long()])


def test_step_pads_and_refuses():
    C = 40
    d = make((6,), C, F32, 831, True)
    pool = torch.randn(4, C, device="cuda")
    before = pool.clone()
    y = torch.full((6, C), 9.0, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    slots = torch.tensor([-1, 2, 2, 4, -7, 0], dtype=torch.int32, device="cuda")
    kda.gated_step(*args(d), pool, z=d["z"], slots=slots, y=y, status=status)
    rows = [1, 5]
    want = before[[2, 0]].clone()
    wy = kda.gated_step(d["x"][rows], d["r"][rows], d["i"][rows], d["lam"], want, z=d["z"][rows])
    assert int(status) == 5 and torch.equal(y[rows], wy) and bool((y[[0, 2, 3, 4]] == 9).all())
    before[[2, 0]] = want
    assert torch.equal(pool, before)


def test_steps_continue_a_prompt():
    """A prompt's end state and the tokens behind it, one at a time, against the whole sequence."""
    C, T = 96, 70
    d = make((1, T), C, F32, 5, True)
    ref = ref_of(d, C, None, [0, T])
    part = {k: v if k == "lam" else v[:, :40].contiguous() for k, v in d.items()}
    _, state = kda.gated_scan_fwd(*args(part), z=part["z"])
    for t in range(40, T):
        y = kda.gated_step(d["x"][:, t], d["r"][:, t], d["i"][:, t], d["lam"], state, z=d["z"][:, t])
        within(y, ref["y"][t:t + 1], ref["y_err"][t:t + 1], F32, t)
    within(state, ref["state"], ref["state_err"], F32, "state")
    # and in pieces by prompts
    _, s2 = kda.gated_scan_fwd(*args(part), z=part["z"])
    rest = {k: v if k == "lam" else v[:, 40:] for k, v in d.items()}
    y2, s2 = kda.gated_scan_fwd(*args(rest), z=rest["z"], initial_state=s2)
    within(y2, ref["y"][40:], ref["y_err"][40:], F32, "piece")
    within(s2, ref["state"], ref["state_err"], F32, "state")


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_of_no_sequence(dtype):
    """Rows before the first offset and behind the last one: outputs left as they are, gradients zero, whatever they hold."""
    C, T = 72, 200
    d = make((1, T), C, dtype, 6, True)
    lo, hi = 37, 150
    for k in ("x", "r", "i", "z"):
        d[k][:, :lo] = float("nan")
        d[k][:, hi:] = float("inf")
    cu = torch.tensor([lo, 90, hi], dtype=torch.int32, device="cuda")
    y = torch.full((1, T, C), 3.0, dtype=dtype, device="cuda")
    _, final = kda.gated_scan_fwd(*args(d), z=d["z"], cu_seqlens=cu, y=y)
    inner = {k: v if k == "lam" else v[:, lo:hi].contiguous() for k, v in d.items()}
    dy = torch.randn(1, T, C, device="cuda").to(dtype)
    dy[:, :lo] = float("nan")
    ref = ref_of(inner, C, None, [0, 90 - lo, hi - lo], dy[:, lo:hi])
    assert bool((y[:, :lo] == 3).all()) and bool((y[:, hi:] == 3).all())
    within(y[:, lo:hi], ref["y"], ref["y_err"], dtype, "y")
    within(final, ref["state"], ref["state_err"], F32, "state")
    out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], cu_seqlens=cu)
    for k in ("dx", "dr", "di", "dz"):
        assert not bool(out[k][:, :lo].any()) and not bool(out[k][:, hi:].any())
        within(out[k][:, lo:hi], ref[k], ref[k + "_err"], dtype, k)
    within(out["dlam"], ref["dlam"], ref["dlam_err"], F32, "dlam")


def test_not_a_number_stays_in_its_sequence():
    C, lens = 64, [50, 70, 3, 400]
    T = sum(lens)
    cu = offsets(lens)
    for bad in (float("nan"), float("inf")):
        d = make((1, T), C, F32, 7, True)
        clean = {k: v if v is None else v.clone() for k, v in d.items()}
        d["x"][:, 60] = bad
        dy = torch.randn(1, T, C, device="cuda")
        a, fa = kda.gated_scan_fwd(*args(d), z=d["z"], cu_seqlens=cu)
        b, fb = kda.gated_scan_fwd(*args(clean), z=clean["z"], cu_seqlens=cu)
        keep = [t for t in range(T) if not 50 <= t < 120]
        assert torch.equal(a[:, keep], b[:, keep]) and torch.equal(fa[[0, 2, 3]], fb[[0, 2, 3]])
        ga = kda.gated_scan_bwd(*args(d), dy, z=d["z"], cu_seqlens=cu)
        gb = kda.gated_scan_bwd(*args(clean), dy, z=clean["z"], cu_seqlens=cu)
        dyn = dy.clone()
        dyn[:, 60] = bad
        gn = kda.gated_scan_bwd(*args(clean), dyn, z=clean["z"], cu_seqlens=cu)
        for k in ("dx", "dr", "di", "dz"):
            assert torch.equal(ga[k][:, keep], gb[k][:, keep]) and torch.equal(gn[k][:, keep], gb[k][:, keep])


def test_gates_at_their_ends():
    """Closed and open gates (an infinite logit too), decays of one and of zero: values and gradients stay finite and right."""
    r = torch.tensor([-float("inf"), -200.0, -60.0, -20.0, 0.0, 20.0, 60.0, 200.0, float("inf")])
    lam = torch.tensor([-200.0, -60.0, -20.0, -5.0, 0.0, 5.0, 40.0])
    n, C = r.numel(), lam.numel()
    T = n * n
    g = torch.Generator().manual_seed(1)
    d = dict(x=torch.randn(1, T, C, generator=g).cuda(), lam=lam.cuda(), z=None,
             r=r.repeat_interleave(n)[None, :, None].expand(1, T, C).contiguous().cuda(), i=r.repeat(n)[None, :, None].expand(1, T, C).contiguous().cuda())
    dy = torch.randn(1, T, C, generator=g).cuda()
    y, final = kda.gated_scan_fwd(*args(d))
    out = kda.gated_scan_bwd(*args(d), dy)
    cap = lambda v: torch.nan_to_num(v, posinf=300.0, neginf=-300.0)  # noqa: E731
    ref = ref_of(dict(d, r=cap(d["r"]), i=cap(d["i"])), C, None, [0, T], dy)
    # a closed gate's 2^-60 instead of less, and 1 / m where m^2 < 1e-36
    within(y, ref["y"], ref["y_err"] + 1e-15, F32, "y")
    within(final, ref["state"], ref["state_err"] + 1e-15, F32, "state")
    for k in ("dx", "di", "dr"):
        within(out[k], ref[k], ref[k + "_err"] + 1e-12, F32, k)
    assert torch.isfinite(out["dlam"]).all()


def test_differences():
    """Gradients against central differences of the 64-bit form."""
    C, lens = 6, [5, 1, 40]
    T = sum(lens)
    d = make((1, T), C, F32, 12, True)
    cu = offsets(lens)
    g = torch.Generator().manual_seed(3)
    initial, dy, dfinal = torch.randn(3, C, generator=g).cuda(), torch.randn(1, T, C, generator=g).cuda(), torch.randn(3, C, generator=g).cuda()
    out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], initial_state=initial, cu_seqlens=cu, dfinal_state=dfinal)
    base = {k: flat(d[k], C) for k in ("x", "r", "i", "z")}
    base.update(lam=f64(d["lam"]), initial=f64(initial))

    def loss(v):
        o = gated(v["x"], v["r"], v["i"], v["lam"], 8.0, v["z"], v["initial"], cu.tolist())
        return (o["y"] * flat(dy, C)).sum() + (o["state"] * f64(dfinal)).sum()
    names = {"x": "dx", "r": "dr", "i": "di", "z": "dz", "lam": "dlam", "initial": "dinitial_state"}
    ref = ref_of(d, C, initial, cu.tolist(), dy, dfinal)
    rng = np.random.default_rng(0)
    for k, name in names.items():
        way = rng.standard_normal(base[k].shape)
        step = 1e-5
        diff = (loss({**base, k: base[k] + step * way}) - loss({**base, k: base[k] - step * way})) / (2 * step)
        got = (f64(out[name]).reshape(way.shape) * way).sum()
        # the kernel's own error along the way, and the difference's: 1e-10 for its step, 1e-9 for its rounding, of values up to some hundred
        assert abs(got - diff) <= ((ref[name + "_err"] + 2.0 ** -24 * np.abs(ref[name])) * np.abs(way)).sum() + 1e-6, name


def test_same_bits_every_time_and_from_slices():
    for C, dtype in ((264, BF16), (70, F32), (33, BF16)):
        T = 900
        d = make((1, T), C, dtype, 77, True, wide=3)
        cu = offsets([400, 1, 499])
        dy = torch.randn(1, T, C, device="cuda").to(dtype)
        whole = {k: v if k == "lam" else v.contiguous() for k, v in d.items()}
        first = None
        for e in (d, whole, d, whole):
            y, final = kda.gated_scan_fwd(*args(e), z=e["z"], cu_seqlens=cu)
            out = kda.gated_scan_bwd(*args(e), dy, z=e["z"], cu_seqlens=cu)
            got = [y, final, out["dx"], out["dr"], out["di"], out["dz"], out["dlam"]]
            first = first or got
            assert all(torch.equal(p, q) for p, q in zip(first, got))


def test_captured_and_on_another_stream():
    C, T = 128, 333
    d = make((1, T), C, BF16, 9, True)
    cu = offsets([200, 133])
    dy = torch.randn(1, T, C, device="cuda").to(BF16)
    states = torch.empty(kda.gated_scan_states(d["x"]), device="cuda")
    pool = torch.randn(4, C, device="cuda")
    slots = torch.tensor([2], dtype=torch.int32, device="cuda")
    one = {k: v if k == "lam" else v[:, 0] for k, v in d.items()}

    def work():
        y, final = kda.gated_scan_fwd(*args(d), z=d["z"], cu_seqlens=cu, states=states)
        out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], cu_seqlens=cu, states=states)
        return [y, final, *[out[k] for k in ("dx", "dr", "di", "dz", "dlam")], kda.gated_step(*args(one), pool, z=one["z"], slots=slots)]
    before = pool.clone()
    want = [t.clone() for t in work()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        pool.copy_(before)
        assert all(torch.equal(a, b) for a, b in zip(work(), want))
        pool.copy_(before)
    side.synchronize()
    with torch.cuda.graph(graph):
        got = work()
    for _ in range(2):
        pool.copy_(before)
        for t in got:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_nothing_to_do():
    C = 8
    e = lambda *s: torch.empty(*s, C, device="cuda")  # noqa: E731
    lam = torch.zeros(C, device="cuda")
    y, final = kda.gated_scan_fwd(e(0, 5), e(0, 5), e(0, 5), lam)
    assert y.shape == (0, 5, C) and final.shape == (0, C)
    initial = torch.randn(2, C, device="cuda")
    y, final = kda.gated_scan_fwd(e(2, 0), e(2, 0), e(2, 0), lam, initial_state=initial)
    assert torch.equal(final, initial)
    out = kda.gated_scan_bwd(e(2, 0), e(2, 0), e(2, 0), lam, e(2, 0), initial_state=initial, dfinal_state=initial)
    assert torch.equal(out["dinitial_state"], initial) and not bool(out["dlam"].any())
    x = torch.randn(1, 4, C, device="cuda")
    cu = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = kda.gated_scan_bwd(x, x, x, lam, x, cu_seqlens=cu)
    assert not bool(out["dx"].any()) and not bool(out["dlam"].any())
    assert kda.gated_step(e(0), e(0), e(0), lam, e(3)).shape == (0, C)
