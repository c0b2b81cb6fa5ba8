"""Batches of single tokens in which padded rows and rows without a page stand at every place among the others, and the
first page, which has no meaning for them, is somebody's: outputs and pages equal those of the other rows alone, bit
for bit, from the smallest batches to those whose blocks take several rows."""
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda

pytestmark = pytest.mark.gpu

BF16, F32 = torch.bfloat16, torch.float32


def batch(N, seed):
    """Slots of N rows (a third of them padded, some out of range), and the rows that have a page."""
    g = torch.Generator().manual_seed(seed)
    P = N + 1
    slots = torch.randperm(P, generator=g)[:N].to(torch.int32)
    slots[torch.rand(N, generator=g) < 0.35] = -1
    slots[N // 2] = 0 if not (slots == 0).any() else slots[N // 2]       # the first page is in use
    if N > 4:
        slots[1], slots[-2] = P, -9
    return g, P, slots, torch.nonzero((slots >= 0) & (slots < P)).view(-1).cuda()


def check(N, live, slots, P, pool, run):
    """run(rows, pool, slots or None, y, status): one step of those rows."""
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = pool.clone()
    y = run(None, got, slots.cuda(), status)
    at = slots.cuda()[live].long()
    mine = pool[at].clone()
    want = run(live, mine, None, None)
    rest = torch.ones(N, dtype=torch.bool, device="cuda")
    rest[live] = False
    pool[at] = mine
    assert torch.equal(y[live], want) and torch.equal(got, pool) and bool((y[rest] == 3).all())
    assert int(status) == (5 if bool(((slots < -1) | (slots >= P)).any()) else 0)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,H,K,V", [(1, 2, 128, 128), (7, 3, 64, 64), (150, 4, 128, 64)])
def test_recurrent_step(N, H, K, V, dtype):
    g, P, slots, live = batch(N, 4000 + N)
    pool = torch.randn(P, H, K, V, generator=g).cuda()
    q, k, v = (torch.randn(N, H, d, generator=g).to(dtype).cuda() for d in (K, K, V))
    gate, beta = (-torch.rand(N, H, K, generator=g)).to(dtype).cuda(), torch.rand(N, H, generator=g).to(dtype).cuda()

    def run(rows, pages, slots, status):
        args = [a if rows is None else a[rows].contiguous() for a in (q, k, v, gate, beta)]
        o = torch.full((args[0].shape[0], H, V), 3.0, device="cuda")
        return kda.recurrent_step(*args, pages, o=o, slots=slots, status=status)
    check(N, live, slots, P, pool, run)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,C,S", [(1, 40, 8), (6, 40, 16), (7, 130, 64), (301, 1024, 16), (300, 600, 32)])
def test_scan_step(N, C, S, dtype):
    g, P, slots, live = batch(N, 4100 + N)
    pool = torch.randn(P, C, S, generator=g).cuda()
    u, delta, z = (torch.randn(N, C, generator=g).to(dtype).cuda() for _ in range(3))
    B, Cm = (torch.randn(N, 1, S, generator=g).to(dtype).cuda() for _ in range(2))
    A, D = -torch.rand(C, S, generator=g).cuda(), torch.randn(C, generator=g).cuda()

    def run(rows, pages, slots, status):
        x = [a if rows is None else a[rows].contiguous() for a in (u, delta, B, Cm, z)]
        y = torch.full(x[0].shape, 3.0, dtype=dtype, device="cuda")
        return kda.ssm_step(x[0], x[1], A, x[2], x[3], pages, D=D, z=x[4], slots=slots, status=status, y=y)
    check(N, live, slots, P, pool, run)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N,C,W", [(1, 40, 4), (6, 37, 3), (301, 2048, 4), (998, 600, 2)])
def test_convolution_step(N, C, W, dtype):
    g, P, slots, live = batch(N, 4200 + N)
    pool, x = torch.randn(P, W - 1, C, generator=g).to(dtype).cuda(), torch.randn(N, C, generator=g).to(dtype).cuda()
    w = torch.randn(C, W, generator=g).cuda()

    def run(rows, pages, slots, status):
        a = x if rows is None else x[rows].contiguous()
        y = torch.full(a.shape, 3.0, dtype=dtype, device="cuda")
        return kda.short_conv_step(a, pages, w, conv_act=1, slots=slots, status=status, y=y)
    check(N, live, slots, P, pool, run)
