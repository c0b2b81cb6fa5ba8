"""The gated recurrence and the group norm where offsets pass 32 bits: many tokens, and rows of very wide ones."""
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


def rows(T, C, seed):
    return torch.empty(1, T, C, dtype=BF16, device="cuda").normal_(generator=torch.Generator("cuda").manual_seed(seed))


def test_more_elements_than_32_bits_count():
    """The last sequences of a stream of 2.2e9 elements against the same by themselves, up to roundings."""
    C, T, n = 8192, 270016, 64
    assert T * C > 2 ** 31
    x, r, i, dy = (rows(T, C, k) for k in range(4))
    lam = torch.linspace(-6.0, -2.0, C, device="cuda")
    cu = torch.arange(0, T + 1, n, dtype=torch.int32, device="cuda")
    y, final = kda.gated_scan_fwd(x, r, i, lam, cu_seqlens=cu)
    few = 3 * n
    tail = [t[:, -few:].contiguous() for t in (x, r, i)]
    ends = torch.arange(0, few + 1, n, dtype=torch.int32, device="cuda")
    y1, final1 = kda.gated_scan_fwd(*tail, lam, cu_seqlens=ends)
    assert torch.allclose(y[:, -few:].float(), y1.float(), rtol=2 ** -7, atol=1e-5) and torch.allclose(final[-3:], final1, rtol=2 ** -14, atol=1e-6)
    out = kda.gated_scan_bwd(x, r, i, lam, dy, cu_seqlens=cu)
    out1 = kda.gated_scan_bwd(*tail, lam, dy[:, -few:].contiguous(), cu_seqlens=ends)
    for k in ("dx", "dr", "di"):
        assert torch.allclose(out[k][:, -few:].float(), out1[k].float(), rtol=2 ** -7, atol=1e-5), k
    del out, y
    y = kda.group_norm_fwd(x, 64, act=1)
    assert torch.equal(y[:, -few:], kda.group_norm_fwd(tail[0], 64, act=1))
    dx = kda.group_norm_bwd(x, 64, dy, act=1)["dx"]
    assert torch.equal(dx[:, -few:], kda.group_norm_bwd(tail[0], 64, dy[:, -few:].contiguous(), act=1)["dx"])
    y = kda.group_norm_fwd(x, 64, act=1, over="sequence", cu_seqlens=cu)
    y1 = kda.group_norm_fwd(tail[0], 64, act=1, over="sequence", cu_seqlens=ends)
    assert torch.allclose(y[:, -few:].float(), y1.float(), rtol=2 ** -7, atol=2 ** -12)


def test_rows_of_very_wide_ones():
    """Rows 2^25 elements apart: the last is 2^31 and more behind the first."""
    C, T, ld = 136, 70, 2 ** 25 + 8
    wide = torch.empty(T * ld, dtype=BF16, device="cuda").view(1, T, ld)
    part = [wide[..., k * C:(k + 1) * C] for k in range(4)]
    for k, p in enumerate(part):
        p.copy_(rows(T, C, 10 + k))
    lam = torch.linspace(-6.0, -2.0, C, device="cuda")
    near = [p.contiguous() for p in part]
    y, final = kda.gated_scan_fwd(*part[:3], lam, z=part[3])
    y1, final1 = kda.gated_scan_fwd(*near[:3], lam, z=near[3])
    assert torch.equal(y, y1) and torch.equal(final, final1)
    a = kda.gated_scan_bwd(*part[:3], lam, y, z=part[3])
    b = kda.gated_scan_bwd(*near[:3], lam, y, z=near[3])
    assert all(torch.equal(a[k], b[k]) for k in ("dx", "dr", "di", "dz", "dlam"))
    for over in ("token", "sequence"):
        assert torch.equal(kda.group_norm_fwd(part[0], 8, act=1, over=over), kda.group_norm_fwd(near[0], 8, act=1, over=over))
        a, b = (kda.group_norm_bwd(t, 8, y, act=1, over=over)["dx"] for t in (part[0], near[0]))
        assert torch.equal(a, b)
    s, s1 = torch.zeros(T, C, device="cuda"), torch.zeros(T, C, device="cuda")
    assert torch.equal(kda.gated_step(*(t[0] for t in part[:3]), lam, s, z=part[3][0]), kda.gated_step(*(t[0] for t in near[:3]), lam, s1, z=near[3][0]))
    assert torch.equal(s, s1)


def test_most_tokens():
    """One channel of as many tokens as a call takes: its end against the same tokens by themselves (a state lives for a few tokens)."""
    T, few = 2 ** 31 - 65536 - 1, 4096
    x, r, i, dy = (rows(T, 1, 20 + k) for k in range(4))
    lam = torch.ones(1, device="cuda")
    y, final = kda.gated_scan_fwd(x, r, i, lam)
    # 64 tokens in, the start is forgotten: a <= exp(-8 softplus(1) sigmoid(-6)) = 0.974 a token, and 0.005 for most
    tail = [t[:, -few:].contiguous() for t in (x, r, i, dy)]
    y1, final1 = kda.gated_scan_fwd(*tail[:3], lam)
    assert torch.allclose(y[:, -few + 512:].float(), y1[:, 512:].float(), rtol=2 ** -7, atol=1e-5) and torch.allclose(final, final1, rtol=2 ** -14, atol=1e-6)
    del y
    out, out1 = kda.gated_scan_bwd(x, r, i, lam, dy), kda.gated_scan_bwd(*tail[:3], lam, tail[3])
    for k in ("dx", "dr", "di"):
        assert torch.allclose(out[k][:, -few + 512:].float(), out1[k][:, 512:].float(), rtol=2 ** -7, atol=1e-5), k
    del out
    w, b = torch.full((1,), 2.0, device="cuda"), torch.full((1,), 0.5, device="cuda")
    assert bool((kda.group_norm_fwd(x, 1, w, b) == 0.5).all())  # of one channel each token is its own mean
    y = kda.group_norm_fwd(x, 1, w, b, over="sequence")  # (mean 0 and deviation 1 up to some 2e-5)
    assert torch.allclose(y[:, -few:].float(), 2 * tail[0].float() + 0.5, rtol=2 ** -7, atol=1e-3)
