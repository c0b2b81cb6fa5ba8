"""KDA decode by slot: what recurrent_step gives on the pages gathered together, bit for bit, and a
serving run of prefill, fork, decode, leave, close up, decode on a pool of states."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
import oracle
from kimi_delta_attention_chunk_gb300 import synth
from tests.kda_testutil import TOL_BF16, rel_err

pytestmark = pytest.mark.gpu


def inputs(N, H, K, V, dtype, seed, steps=1):
    d = synth.decode_inputs(N, H, K, V, steps, dtype, seed)
    return {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in d.items()}


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("N,H,K,V", [(1, 1, 64, 64), (5, 3, 128, 64), (33, 2, 64, 128), (300, 4, 128, 128)])
def test_equals_the_dense_step(N, H, K, V, dtype):
    d = inputs(N, H, K, V, dtype, 700 + N)
    P = N + 9
    g = torch.Generator().manual_seed(N)
    slots = torch.randperm(P, generator=g)[:N].to(torch.int32).cuda()
    pool = torch.randn(P, H, K, V, generator=g).cuda()
    before = pool.clone()
    dense = pool[slots.long()].clone()
    args = [d[k][0] for k in ("q", "k", "v", "g", "beta")]
    want = kda.recurrent_step(*args, dense)
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    got = kda.recurrent_step(*args, pool, slots=slots, status=status)
    before[slots.long()] = dense
    assert torch.equal(got, want) and torch.equal(pool, before) and int(status) == 0


def test_pads_and_refuses():
    N, H, K, V, P = 7, 2, 128, 128, 5
    d = inputs(N, H, K, V, torch.bfloat16, 720)
    args = [d[k][0] for k in ("q", "k", "v", "g", "beta")]
    pool = torch.randn(P, H, K, V, device="cuda")
    before = pool.clone()
    slots = torch.tensor([3, -1, 3, P, 0, -2, 3], dtype=torch.int32, device="cuda")
    status = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    o = torch.full((N, H, V), 4.0, device="cuda")
    kda.recurrent_step(*args, pool, slots=slots, o=o, status=status)
    rows = [0, 4]
    dense = before[[3, 0]].clone()
    want = kda.recurrent_step(*[a[rows].contiguous() for a in args], dense)
    assert int(status) == 5 and torch.equal(o[rows], want)
    assert bool((o[[1, 2, 3, 5, 6]] == 4).all())
    before[[3, 0]] = dense
    assert torch.equal(pool, before)
    kda.recurrent_step(*[a[:0].contiguous() for a in args], pool, slots=slots[:0], status=status)
    assert int(status) == 0


def test_a_serving_run():
    """Three prompts prefilled into pages, one forked, all decoded, one leaves, the pool closes up, the rest
    go on: every output equals the oracle's on the sequence's own tokens."""
    H, K, V, P = 2, 128, 128, 8
    lengths, steps = [70, 3, 129], 4
    inp = synth.direct_inputs(0, H, K, V, torch.bfloat16, seed=730, lengths=lengths)
    d = {k: v.cuda() if isinstance(v, torch.Tensor) else v for k, v in inp.items()}
    _, states = kda.chunk_fwd(d["q"], d["k"], d["v"], d["g"], d["beta"], cu_seqlens=d["cu_seqlens"])
    refs = torch.zeros(P, dtype=torch.int32, device="cuda")
    tables = torch.full((4, 1), -1, dtype=torch.int32, device="cuda")
    lens = torch.tensor(lengths + [0], dtype=torch.int32, device="cuda")
    hold = kda.pages_alloc(refs, 1)          # something else sits on the first page
    pool = torch.full((P, H, K, V), float("nan"), device="cuda")
    tables[:3, 0] = kda.pages_alloc(refs, 3)
    pool[tables[:3, 0].long()] = states
    src, dst = kda.pages_fork(tables, lens, refs, torch.tensor([1], dtype=torch.int32).cuda(), torch.tensor([3], dtype=torch.int32).cuda(), 1 << 30)
    kda.pages_copy(pool, src, dst)
    kda.pages_free(refs, hold)
    cu = inp["cu_seqlens"].tolist()
    of = [0, 1, 2, 1]
    tok = {s: [[inp[n][0, cu[of[s]]:cu[of[s] + 1]] for n in ("q", "k", "v", "g", "beta")]] for s in range(4)}
    new = synth.decode_inputs(4, H, K, V, 2 * steps, torch.bfloat16, 731)
    alive, outs = [0, 1, 2, 3], {s: [] for s in range(4)}
    for t in range(2 * steps):
        if t == steps:
            kda.pages_free(refs, tables[0])
            tables[0] = -1
            alive = [1, 2, 3]
            src, dst = kda.pages_compact(refs, tables)
            kda.pages_copy(pool, src, dst)
            assert sorted(tables[1:, 0].tolist()) == [0, 1, 2]
        rows = alive + [0] * (4 - len(alive))
        slots = tables[rows, 0].contiguous()
        args = [new[n][t][rows].contiguous().cuda() for n in ("q", "k", "v", "g", "beta")]
        o = kda.recurrent_step(*args, pool, slots=slots)
        for i, s in enumerate(alive):
            outs[s].append(o[i])
            tok[s].append([new[n][t][s:s + 1] for n in ("q", "k", "v", "g", "beta")])
    for s in range(4):
        q, k, v, g, b = (torch.cat([part[i] for part in tok[s]])[None] for i in range(5))
        ro, rs = oracle.kda_forward(q, k, v, g, b, scale=K ** -0.5)
        n = len(outs[s])
        assert rel_err(torch.stack(outs[s]), ro[0, -n:]) <= TOL_BF16
        if s in alive:
            assert rel_err(pool[int(tables[s, 0])], rs[0]) <= TOL_BF16


def test_a_state_space_layer_served_from_two_pools():
    """Convolution and scan, prompts and single tokens, their histories and states in two pools that go by one set
    of books: prompts come in, one is forked, one leaves, the pools are closed up; every sequence's outputs equal
    those of its whole prompt."""
    C, S, W, P = 72, 16, 4, 9
    g = torch.Generator().manual_seed(740)
    rn = lambda *shape: torch.randn(*shape, generator=g).cuda()  # noqa: E731
    w, A, D, bias = rn(C, W) * 0.5, -torch.exp(rn(C, S)), rn(C), rn(C) - 2
    lengths, steps = [33, 1, 90], 6
    T = max(lengths) + 2 * steps
    x, delta, z, B, Cm = rn(4, T, C), rn(4, T, C), rn(4, T, C), rn(4, T, 1, S), rn(4, T, 1, S)
    of = [0, 1, 2, 2]                      # sequence 3 is forked from 2 and goes on with tokens of its own
    for s in (x, delta, z, B, Cm):
        s[3, :lengths[2]] = s[2, :lengths[2]]

    def whole(s, n):
        cut = lambda v: v[s:s + 1, :n].contiguous()  # noqa: E731
        u, _ = kda.short_conv_fwd(cut(x), w, conv_act=1)
        return kda.ssm_scan_fwd(u, cut(delta), A, cut(B), cut(Cm), D=D, z=cut(z), delta_bias=bias)[0][0]
    # the prompts, packed
    cat = lambda v: torch.cat([v[i, :n] for i, n in enumerate(lengths)])[None].contiguous()  # noqa: E731
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lengths)]), dtype=torch.int32).cuda()
    u, h = kda.short_conv_fwd(cat(x), w, conv_act=1, cu_seqlens=cu)
    _, st = kda.ssm_scan_fwd(u, cat(delta), A, cat(B), cat(Cm), D=D, z=cat(z), delta_bias=bias, cu_seqlens=cu)
    hist, state = torch.full((P, W - 1, C), float("nan"), device="cuda"), torch.full((P, C, S), float("nan"), device="cuda")
    refs, lens = torch.zeros(P, dtype=torch.int32).cuda(), torch.tensor(lengths + [0], dtype=torch.int32).cuda()
    tables = torch.full((4, 1), -1, dtype=torch.int32).cuda()
    hold = kda.pages_alloc(refs, 2)
    tables[:3, 0] = kda.pages_alloc(refs, 3)
    kda.pages_free(refs, hold)
    hist[tables[:3, 0].long()], state[tables[:3, 0].long()] = h, st
    one = lambda v: torch.tensor([v], dtype=torch.int32).cuda()  # noqa: E731
    src, dst = kda.pages_fork(tables, lens, refs, one(2), one(3), 1 << 30)
    assert dst.tolist() == [0]
    for pool in (hist, state):
        kda.pages_copy(pool, src, dst)
    alive, at, outs = [0, 1, 2, 3], [lengths[i] for i in of], {s: [] for s in range(4)}
    for t in range(2 * steps):
        if t == steps:
            kda.pages_free(refs, tables[1])
            tables[1] = -1
            alive = [0, 2, 3]
            src, dst = kda.pages_compact(refs, tables)
            for pool in (hist, state):
                kda.pages_copy(pool, src, dst)
        rows = alive + [1] * (4 - len(alive))          # the gone sequence's row is padding
        slots = tables[rows, 0].contiguous()
        pick = lambda v: torch.stack([v[s, at[s]] for s in rows])  # noqa: E731
        u = kda.short_conv_step(pick(x), hist, w, conv_act=1, slots=slots)
        y = kda.ssm_step(u, pick(delta), A, pick(B), pick(Cm), state, D=D, z=pick(z), delta_bias=bias, slots=slots)
        for i, s in enumerate(alive):
            outs[s].append(y[i])
            at[s] += 1
    for s in range(4):
        want = whole(s, at[s])[-len(outs[s]):]
        # the same 32-bit recurrences, cut elsewhere
        torch.testing.assert_close(torch.stack(outs[s]), want, rtol=2e-5, atol=2e-5)


def test_pools_past_two_to_the_31_elements():
    C, S, P = 4096, 64, 8400                          # 2.2e9 states, 8.8 GB
    pool = torch.zeros(P, C, S, device="cuda")
    g = torch.Generator().manual_seed(741)
    u = torch.randn(2, C, generator=g).cuda()
    A, B = -torch.ones(C, S, device="cuda"), torch.randn(2, 1, S, generator=g).cuda()
    slots = torch.tensor([P - 1, 3], dtype=torch.int32, device="cuda")
    small = torch.zeros(2, C, S, device="cuda")
    y = kda.ssm_step(u, u, A, B, B, pool, slots=slots)
    assert torch.equal(y, kda.ssm_step(u, u, A, B, B, small)) and torch.equal(pool[[P - 1, 3]], small)
    assert not pool[4:P - 1].any()
    del pool
    q = torch.randn(2, 4, 128, generator=g).cuda()
    b = torch.rand(2, 4, generator=g).cuda()
    pool = torch.zeros(33000, 4, 128, 128, device="cuda")   # 2.2e9
    small = torch.zeros(2, 4, 128, 128, device="cuda")
    slots = torch.tensor([32999, 0], dtype=torch.int32, device="cuda")
    o = kda.recurrent_step(q, q, q, -b[..., None].expand(2, 4, 128).contiguous(), b, pool, slots=slots)
    assert torch.equal(o, kda.recurrent_step(q, q, q, -b[..., None].expand(2, 4, 128).contiguous(), b, small))
    assert torch.equal(pool[[32999, 0]], small)
    del pool
    hist = torch.zeros(180000, 3, 4096, dtype=torch.bfloat16, device="cuda")   # 2.2e9
    slots = torch.tensor([179999, 1], dtype=torch.int32, device="cuda")
    xb, w = u.to(torch.bfloat16), torch.randn(C, 4, generator=g).cuda()
    small = torch.zeros(2, 3, 4096, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(kda.short_conv_step(xb, hist, w, slots=slots), kda.short_conv_step(xb, small, w))
    assert torch.equal(hist[[179999, 1]], small)
