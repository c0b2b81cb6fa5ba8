"""The pages of a cache against the same books kept in Python lists: every number equal."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.layer_ref import Books, copy_pages

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def word():
    return torch.full((1,), -1, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("P,n,used", [(1, 1, 0.0), (1, 2, 1.0), (7, 3, 0.5), (1024, 100, 0.5), (1025, 700, 0.4), (8192, 5000, 0.3),
                                      (8193, 9000, 0.1), (100003, 60000, 0.5), (40000, 1, 1.0), (9000, 9000, 0.0)])
def test_alloc(P, n, used):
    rng = np.random.default_rng(P + n)
    refs = (rng.random(P) < used) * rng.integers(1, 4, P)
    books, r, st = Books(refs), dev(refs), word()
    want, short = books.alloc(n)
    got = kda.pages_alloc(r, n, status=st)
    assert got.tolist() == want and r.tolist() == books.refs and int(st) == (5 if short else 0)


def test_free():
    rng = np.random.default_rng(3)
    P = 500
    refs = rng.integers(0, 4, P)
    # every page as often as it has references, in a scrambled order, with padding: all come free
    pages = np.concatenate([np.repeat(np.arange(P), refs), np.full(77, -1)])
    rng.shuffle(pages)
    r, st = dev(refs), word()
    kda.pages_free(r, dev(pages), status=st)
    assert not r.any() and int(st) == 0
    # too often, out of range
    bad = np.concatenate([pages, [0, 1, 2, P, -2, 2 ** 31 - 1]])
    rng.shuffle(bad)
    r, books = dev(refs), Books(refs)
    assert books.free(bad)
    kda.pages_free(r, dev(bad).view(-1, 1), status=st)
    assert r.tolist() == books.refs and int(st) == 5
    kda.pages_free(r, dev([]), status=st)
    assert int(st) == 0


def sequences(rng, S, width, tokens, P, busy):
    """Books of S sequences of which `busy` hold pages."""
    order = rng.permutation(P)
    tables, lens, refs, k = np.full((S, width), -1), np.zeros(S, int), np.zeros(P, int), 0
    for s in rng.permutation(S)[:busy]:
        lens[s] = rng.integers(0, width * tokens + 1)
        held = -(-lens[s] // tokens)
        tables[s, :held] = order[k:k + held]
        refs[order[k:k + held]] = 1
        k += held
    return tables, lens, refs


@pytest.mark.parametrize("S,width,tokens,P,busy,n", [(2, 1, 1 << 30, 3, 1, 1), (12, 5, 16, 60, 6, 6), (40, 1, 1 << 20, 64, 20, 18),
                                                     (300, 33, 64, 9000, 200, 100), (700, 3, 128, 1100, 350, 300)])
def test_fork(S, width, tokens, P, busy, n):
    rng = np.random.default_rng(S + n)
    tables, lens, refs = sequences(rng, S, width, tokens, P, busy)
    idle = [s for s in range(S) if (tables[s] == -1).all()]
    have = [s for s in range(S) if lens[s] > 0] or [0]
    children = np.asarray(idle)[rng.permutation(len(idle))[:n]]
    parents = rng.choice([h for h in have if h not in set(children)] or [s for s in range(S) if s not in set(children)], len(children))
    parents[rng.random(len(parents)) < 0.05] = -1
    books = Books(refs, tables, lens)
    t, l, r, st = dev(tables), dev(lens), dev(refs), word()
    src, dst = kda.pages_fork(t, l, r, dev(parents), dev(children), tokens, status=st)
    ws, wd, refused = books.fork([int(p) for p in parents], [int(c) for c in children], tokens)
    assert src.tolist() == ws and dst.tolist() == wd
    assert t.tolist() == books.tables and l.tolist() == books.lens and r.tolist() == books.refs
    assert int(st) == (5 if refused else 0)


@pytest.mark.parametrize("n", [64, 65, 256, 257, 900])
@pytest.mark.parametrize("same", [False, True])
def test_forks_in_conflict(n, same):
    """Children listed twice, children that are parents, skipped requests and rows out of range among many; `same`: one
    child for most requests."""
    rng = np.random.default_rng(n)
    S, width, tokens, P = 1200, 3, 16, 2000
    tables, lens, refs = sequences(rng, S, width, tokens, P, 500)
    order = np.argsort(lens == 0, kind="stable")
    parents, children = order[rng.integers(0, 500, n)], order[500 + rng.permutation(S - 500)[:n] if n <= S - 500 else 500 + rng.integers(0, S - 500, n)]
    children[rng.random(n) < (0.6 if same else 0.0)] = order[700]
    for what, at in (("twice", rng.random(n) < 0.1), ("parent", rng.random(n) < 0.05), ("child", rng.random(n) < 0.05)):
        other = rng.integers(0, n, n)
        if what == "twice":
            children[at] = children[other[at]]
        elif what == "parent":
            children[at] = parents[other[at]]
        else:
            parents[at] = children[other[at]]
    parents[rng.random(n) < 0.05], children[rng.random(n) < 0.05] = -1, -1
    parents[rng.random(n) < 0.02], children[rng.random(n) < 0.02] = S, -7
    books = Books(refs, tables, lens)
    t, l, r, st = dev(tables), dev(lens), dev(refs), word()
    src, dst = kda.pages_fork(t, l, r, dev(parents), dev(children), tokens, status=st)
    ws, wd, refused = books.fork([int(p) for p in parents], [int(c) for c in children], tokens)
    assert refused and src.tolist() == ws and dst.tolist() == wd
    assert t.tolist() == books.tables and l.tolist() == books.lens and r.tolist() == books.refs and int(st) == 5


def test_fork_refuses():
    tokens, P = 16, 12
    tables = np.full((8, 3), -1)
    tables[0, :2], tables[1, :3], tables[2, :1] = [3, 4], [0, 1, 2], [7]
    lens = np.array([20, 48, 16, 0, 0, 0, 49, -1])
    refs = np.zeros(P, int)
    refs[[0, 1, 2, 3, 4]] = 1       # page 7 of sequence 2 is not in use
    for parents, children in [([0], [3]), ([0, 0], [3, 3]), ([0, 1], [1, 3]), ([0], [0]), ([8], [3]), ([0], [-3]), ([2], [3]), ([6], [3]),
                              ([7], [3]), ([3], [4]), ([0, 2, 1, 0], [3, 4, 5, 7]), ([-1, 0], [3, 3]), ([0, 0, 0], [3, 4, 5]),
                              ([0] * 4, [3, 4, 5, 9])]:
        books = Books(refs, tables, lens)
        t, l, r, st = dev(tables), dev(lens), dev(refs), word()
        src, dst = kda.pages_fork(t, l, r, dev(parents), dev(children), tokens, status=st)
        ws, wd, refused = books.fork(parents, children, tokens)
        assert (src.tolist(), dst.tolist()) == (ws, wd), (parents, children)
        assert t.tolist() == books.tables and l.tolist() == books.lens and r.tolist() == books.refs, (parents, children)
        assert int(st) == (5 if refused else 0), (parents, children)


def test_fork_without_pages_left():
    tables, lens = np.full((6, 2), -1), np.array([17, 16, 0, 0, 0, 0])
    tables[0], tables[1, 0] = [0, 1], 2
    refs = np.array([1, 1, 1, 0])
    books = Books(refs, tables, lens)
    t, l, r, st = dev(tables), dev(lens), dev(refs), word()
    # one free page: the first request gets it, the second is refused, the third needs none
    src, dst = kda.pages_fork(t, l, r, dev([0, 0, 1]), dev([2, 3, 4]), 16, status=st)
    assert (src.tolist(), dst.tolist(), True) == books.fork([0, 0, 1], [2, 3, 4], 16)
    assert t.tolist() == books.tables and l.tolist() == books.lens and r.tolist() == books.refs and int(st) == 5


@pytest.mark.parametrize("P,rows,width,used", [(1, 1, 1, 1.0), (2, 1, 1, 0.5), (16, 5, 4, 0.5), (1000, 40, 30, 0.6), (8200, 64, 100, 0.7),
                                               (30001, 100, 200, 0.5), (512, 8, 64, 1.0), (512, 8, 64, 0.0)])
def test_compact(P, rows, width, used):
    rng = np.random.default_rng(P)
    refs = np.zeros(P, int)
    tables = np.full((rows, width), -1)
    held = rng.permutation(P)[:min(int(round(P * used)), rows * width)]
    tables.reshape(-1)[rng.permutation(rows * width)[:len(held)]] = held
    refs[held] = rng.integers(1, 5, len(held))
    books = Books(refs, tables)
    t, r, st = dev(tables), dev(refs), word()
    src, dst = kda.pages_compact(r, t, status=st)
    ws, wd, refused = books.compact()
    assert src.tolist() == ws and dst.tolist() == wd and not refused
    assert t.tolist() == books.tables and r.tolist() == books.refs and int(st) == 0
    again, _ = kda.pages_compact(r, t)
    assert bool((again == -1).all())


def test_compact_without_tables_and_with_stale_entries():
    refs = np.array([0, 2, 0, 1, 0, 1])
    books, r = Books(refs), dev(refs)
    src, dst = kda.pages_compact(r)
    assert (src.tolist(), dst.tolist()) == books.compact()[:2] and r.tolist() == books.refs
    tables = np.array([[5, 4, -1], [3, 9, -8]])       # 4 is free, 9 and -8 are no pages
    books, r, t, st = Books(refs, tables), dev(refs), dev(tables), word()
    kda.pages_compact(r, t, status=st)
    assert books.compact()[2] and t.tolist() == books.tables and int(st) == 5


@pytest.mark.parametrize("dtype,page", [(torch.float32, (4,)), (torch.bfloat16, (3, 8)), (torch.float32, (2, 64, 66)), (torch.uint8, (48,)),
                                        (torch.bfloat16, (5, 4100, 2))])
@pytest.mark.parametrize("P,n", [(2, 1), (40, 25), (200, 300), (150, 128), (150, 129), (400, 127)])
def test_copy(P, n, dtype, page):
    rng = np.random.default_rng(P + n)
    pool = torch.randint(0, 100, (P,) + page, generator=torch.Generator().manual_seed(P)).to(dtype)
    order = rng.permutation(P)
    half = max(1, P // 2)
    src, dst = order[rng.integers(0, half, n)], order[half + rng.integers(0, P - half, n)] if P > half else order[:n]
    src[rng.random(n) < 0.1] = -1
    if n > 100:
        src[7], dst[11], dst[13], src[17] = P, -2, -1, dst[20]      # out of range, skipped, and one read that another pair writes
    want = pool.float().numpy().copy()
    bad = copy_pages(want, src.tolist(), dst.tolist())
    got, st = pool.cuda(), word()
    kda.pages_copy(got, dev(src), dev(dst), status=st)
    assert np.array_equal(got.float().cpu().numpy(), want) and int(st) == (5 if bad else 0)


def test_copy_refuses_a_page_that_is_read_and_written():
    pool = torch.arange(6, dtype=torch.float32, device="cuda")[:, None].repeat(1, 4)
    st = word()
    kda.pages_copy(pool, dev([0, 1, 2, 3, 3]), dev([1, 2, 0, 4, 4]), status=st)       # a ring, and one page twice
    assert pool[:, 0].tolist() == [0, 1, 2, 3, 3, 5] and int(st) == 5
    kda.pages_copy(pool, dev([5, 2]), dev([5, 0]), status=st)                         # onto itself: nothing
    assert pool[:, 0].tolist() == [2, 1, 2, 3, 3, 5] and int(st) == 0


def test_pages_past_four_gigabytes():
    pool = torch.empty(72, 16 * 1024 * 1024, dtype=torch.float32, device="cuda")      # 64 MiB a page, 4.5 GiB
    pool[70], pool[1] = 3.0, 1.0
    kda.pages_copy(pool, dev([70, 1]), dev([69, 71]))
    assert bool((pool[69] == 3).all()) and bool((pool[71] == 1).all())


def test_copy_in_the_largest_pool():
    """The last pages of 2^30 pages of 16 bytes, by few pairs and by marks."""
    P = 2 ** 30
    pool = torch.empty(P, 4, dtype=torch.int32, device="cuda")
    for n in (3, 200):
        pool[-n - 2:] = torch.arange(n + 2, dtype=torch.int32, device="cuda")[:, None]
        src, dst, st = dev([P - 1] * n), dev(range(P - n - 2, P - 2)), word()
        kda.pages_copy(pool, src, dst, status=st)
        assert int(st) == 0 and bool((pool[-n - 2:-2] == n + 1).all()) and int(pool[-2, 0]) == n
        kda.pages_copy(pool, dev([0] * (n - 1) + [P - 1]), dev([P - 1] * n), status=st)     # written again and again, and onto itself
        assert int(st) == 5 and bool((pool[-1] == pool[0]).all())          # the last that writes it (its own pair is none)


def test_many_forks():
    """More requests than one block looks over, of a small pool's full pages."""
    for n in (300, 9000, 65536):
        tables = torch.full((n + 1, 3), -1, dtype=torch.int32, device="cuda")
        tables[0] = dev([2, 1, 3])
        lens, refs, st = torch.zeros(n + 1, dtype=torch.int32, device="cuda"), dev([0, 1, 1, 1]), word()
        lens[0] = 48
        children = torch.randperm(n, generator=torch.Generator().manual_seed(n)).to(torch.int32).cuda() + 1
        children[n // 2] = children[n // 3]
        src, dst = kda.pages_fork(tables, lens, refs, torch.zeros_like(children), children, 16, status=st)
        assert int(st) == 5 and bool((src == -1).all()) and bool((dst == -1).all())
        made = (tables[1:] == tables[0]).all(1)
        assert int(made.sum()) == n - 2 and refs.tolist() == [0] + [n - 1] * 3 and int((lens == 48).sum()) == n - 1


def test_books_in_a_graph():
    """A captured turn (free, close up, copy, take) replayed on moving books equals the lists'."""
    rng = np.random.default_rng(8)
    P, rows = 64, 40
    tables, refs = rng.permutation(P)[:rows].reshape(rows, 1), np.zeros(P, int)
    refs[tables] = 1
    pool0 = rng.integers(0, 1000, (P, 8)).astype(np.float32)
    gone = dev(rng.permutation(rows)[:10])
    t, r, pool = dev(tables), dev(refs), torch.from_numpy(pool0).cuda()

    def turn():
        kda.pages_free(r, t[gone.long()])
        t.index_fill_(0, gone.long(), -1)      # (an assigned scalar would be copied from the host)
        src, dst = kda.pages_compact(r, t)
        kda.pages_copy(pool, src, dst)
        t[gone.long()] = kda.pages_alloc(r, 10).view(-1, 1)
    turn()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        turn()
    graph.replay()
    gone.copy_(dev(rng.permutation(rows)[:10]))
    graph.replay()
    torch.cuda.synchronize()
    assert sorted(t.view(-1).tolist()) == [p for p in range(P) if r[p] == 1] and int(r.sum()) == rows
    assert max(t.view(-1).tolist()) < rows
