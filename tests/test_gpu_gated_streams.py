"""The gated linear recurrence where its kernels divide the work in other ways: sequences with blocks of their own and as one stream,
blocks of 64, 32 and 16 channels, alone and in clusters, many sequences, offsets that leave rows out."""
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.gated_norm_ref import within
from tests.test_gpu_gated_scan import BF16, F32, args, make, ref_of

pytestmark = pytest.mark.gpu


def cumulative(lens, lead=0):
    out = [lead]
    for n in lens:
        out.append(out[-1] + n)
    return out


def check(d, C, dtype, cu, T, seed, gate, kept=(True, False)):
    """Everything a call gives against the 64-bit form, rows of no sequence among it."""
    N = len(cu) - 1
    g = torch.Generator().manual_seed(seed)
    initial, dfinal = torch.randn(N, C, generator=g).cuda(), torch.randn(N, C, generator=g).cuda()
    dy = torch.randn(1, T, C, generator=g).to(dtype).cuda()
    offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
    lo, hi = cu[0], cu[-1]
    y = torch.full((1, T, C), 5.0, dtype=dtype, device="cuda")
    states = torch.full(kda.gated_scan_states(d["x"]), 7.0, device="cuda")
    _, final = kda.gated_scan_fwd(*args(d), z=d["z"], initial_state=initial, cu_seqlens=offsets, states=states, y=y)
    inner = {k: v if k == "lam" or v is None else v[:, lo:hi] for k, v in d.items()}
    ref = ref_of(inner, C, initial, [c - lo for c in cu], dy[:, lo:hi], dfinal)
    within(y[:, lo:hi], ref["y"], ref["y_err"], dtype, "y")
    within(final, ref["state"], ref["state_err"], F32, "state")
    assert bool((y[:, :lo] == 5).all()) and bool((y[:, hi:] == 5).all())
    for keep in kept:
        out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], initial_state=initial, cu_seqlens=offsets, dfinal_state=dfinal,
                                 states=states if keep else None)
        for k in ("dx", "dr", "di") + (("dz",) if gate else ()):
            within(out[k][:, lo:hi], ref[k], ref[k + "_err"], dtype, k)
            assert not bool(out[k][:, :lo].any()) and not bool(out[k][:, hi:].any())
        within(out["dlam"], ref["dlam"], ref["dlam_err"], F32, "dlam")
        within(out["dinitial_state"], ref["dinitial_state"], ref["dinitial_state_err"], F32, "dinitial")


PACKED = [  # lens, rows before and behind, C
    ([64] * 40, 0, 0, 1024), ([40] * 30, 0, 0, 264), ([130] * 20, 0, 0, 72), ([1] * 10 + [2500] + [3] * 9, 0, 0, 72), ([100] * 300, 0, 0, 16),
    ([10] * 300, 0, 0, 34), ([0, 363, 0, 501], 37, 99, 200), ([0, 363, 0, 501, 0], 37, 99, 2048), ([0, 500, 0], 0, 0, 2048), ([0], 400, 13, 136),
    ([0, 0, 0], 200, 300, 1600), ([97, 200, 1], 31, 1, 33), ([320, 96, 33], 32, 64, 1536),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,lead,tail,C", PACKED)
def test_packed(lens, lead, tail, C, dtype):
    T = lead + sum(lens) + tail
    d = make((1, T), C, dtype, T + C, True)
    for k in ("x", "r", "i", "z"):
        d[k][:, :lead] = float("nan")
        d[k][:, lead + sum(lens):] = float("inf")
    check(d, C, dtype, cumulative(lens, lead), T, T, True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("B,T,C", [(1, 1500, 2048), (2, 300, 4096), (4, 150, 4096), (1, 700, 16), (3, 513, 48), (1, 1030, 1030), (2, 260, 96)])
def test_widths(B, T, C, dtype):
    d = make((B, T), C, dtype, T, True)
    g = torch.Generator().manual_seed(C)
    dy, dfinal = torch.randn(B, T, C, generator=g).to(dtype).cuda(), torch.randn(B, C, generator=g).cuda()
    states = torch.empty(kda.gated_scan_states(d["x"]), device="cuda")
    y, final = kda.gated_scan_fwd(*args(d), z=d["z"], states=states)
    ref = ref_of(d, C, None, [T * b for b in range(B + 1)], dy, dfinal)
    within(y.reshape(-1, C), ref["y"], ref["y_err"], dtype, "y")
    within(final, ref["state"], ref["state_err"], F32, "state")
    within(states, ref["before"].reshape(B, T, C)[:, ::32], ref["before_err"].reshape(B, T, C)[:, ::32], F32, "states")
    out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], dfinal_state=dfinal, states=states)
    for k in ("dx", "dr", "di", "dz"):
        within(out[k].reshape(-1, C), ref[k], ref[k + "_err"], dtype, k)
    within(out["dlam"], ref["dlam"], ref["dlam_err"], F32, "dlam")


def test_large_rates():
    """Decays far from 1: logits and rates that take s from far below a quarter to far above it."""
    C, T = 136, 400
    for dtype in (BF16, F32):
        d = make((1, T), C, dtype, 77, True)
        d["lam"] = torch.linspace(-12.0, 6.0, C).cuda()
        d["r"] = (d["r"].float() * 3.0).to(dtype)
        check(d, C, dtype, [0, 150, 400], T, 3, True)


def test_offsets_that_are_not_sorted():
    """Results are then undefined, but nothing outside the tensors is touched and the call ends."""
    C, T = 72, 600
    d = make((1, T), C, BF16, 78, True)
    guard = torch.full((3, T, C), 2.0, dtype=BF16, device="cuda")
    for cu in ([0, 400, 100, 600], [600, 0, 300, 0], [-5, 700, 90, 1000], [600, 600, 0, 0]):
        offsets = torch.tensor(cu, dtype=torch.int32, device="cuda")
        kda.gated_scan_fwd(*args(d), z=d["z"], cu_seqlens=offsets, y=guard[1:2])
        kda.gated_scan_bwd(*args(d), guard[:1], z=d["z"], cu_seqlens=offsets)
        torch.cuda.synchronize()
        assert bool((guard[0] == 2).all()) and bool((guard[2] == 2).all())


def test_bits_do_not_depend_on_the_others():
    """A sequence with blocks of its own has the bits of the same sequence by itself, wherever it begins at a whole block."""
    C = 4096
    lens = [256, 96, 320, 160]
    cu = cumulative(lens)
    d = make((1, cu[-1]), C, BF16, 79, True)
    y, final = kda.gated_scan_fwd(*args(d), z=d["z"], cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    again, _ = kda.gated_scan_fwd(*args(d), z=d["z"], cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert torch.equal(y, again)
    batch = {k: v if k == "lam" else v[:, :256].expand(4, 256, C).contiguous() for k, v in d.items()}
    yb, fb = kda.gated_scan_fwd(*args(batch), z=batch["z"])
    assert torch.equal(yb[0], y[0, :256]) and torch.equal(yb[3], yb[0]) and torch.equal(fb[0], final[0])


@pytest.mark.parametrize("lens,lead,tail,C", [([0, 363, 0, 501], 100, 99, 200), ([150, 200], 70, 90, 2048), ([3] * 20, 40, 70, 72)])
def test_states_before_tokens_of_no_sequence_are_not_used(lens, lead, tail, C):
    """They are left as they are, whatever was there."""
    T = lead + sum(lens) + tail
    cu = torch.tensor(cumulative(lens, lead), dtype=torch.int32, device="cuda")
    d = make((1, T), C, BF16, T, True)
    dy = torch.randn(1, T, C, generator=torch.Generator().manual_seed(C)).to(BF16).cuda()
    out = []
    for filled in (0.0, float("nan")):
        states = torch.full(kda.gated_scan_states(d["x"]), filled, device="cuda")
        kda.gated_scan_fwd(*args(d), z=d["z"], cu_seqlens=cu, states=states)
        out.append(kda.gated_scan_bwd(*args(d), dy, z=d["z"], cu_seqlens=cu, states=states))
    assert all(torch.equal(out[0][k], out[1][k]) for k in ("dx", "dr", "di", "dz", "dlam"))
