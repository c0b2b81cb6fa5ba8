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
