"""The selective state space scan (single token) against its plain 64-bit form.

Tolerances, element by element.  The step size d is off by 2^-21 relative (softplus: one exponential,
2^-22, and a series), and the decay's exponent d A by as much of itself plus a rounding, so the decay is off
by |d A| 2^-20 + 2^-22 relative; with the products' roundings a state is off by
2^-19 (|a h| (1 + |d A|) + |d u B|) per step.  y adds S products and D u, each rounded, and the gate's
relative 2^-20 |z| + 2^-21."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.layer_ref import f64, half_step, silu, softplus

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
