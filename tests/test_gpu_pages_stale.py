"""Closing up pools while table entries still name pages that were given back: such an entry is reported wherever
its page lies, also where another page moves into that place and the entry would name it without a word."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.layer_ref import Books

pytestmark = pytest.mark.gpu


def dev(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def word():
    return torch.full((1,), -1, dtype=torch.int32, device="cuda")


def test_an_entry_that_names_a_hole():
    # pages 0, 2 and 5 are in use; 1 is free and page 5 moves there: the old entry 1 now names another row's page
    r, t, st = dev([1, 0, 1, 0, 0, 1]), dev([[0, 2], [5, -1], [1, -1]]), word()
    src, dst = kda.pages_compact(r, t, status=st)
    assert src.tolist() == [5, -1, -1] and dst.tolist() == [1, -1, -1] and r.tolist() == [1, 1, 1, 0, 0, 0]
    assert t.tolist() == [[0, 2], [1, -1], [1, -1]] and int(st) == 5
    kda.pages_compact(dev([1, 0, 1, 0, 0, 1]), dev([[0, 2], [5, -1], [-1, -1]]), status=st)
    assert int(st) == 0


# one block, a cluster, and entries enough for a launch of their own
@pytest.mark.parametrize("P,rows,width", [(64, 9, 7), (8192, 100, 80), (30001, 100, 300), (30001, 100, 700)])
@pytest.mark.parametrize("stale", [0, 1, 50])
def test_stale_entries_among_many(P, rows, width, stale):
    rng = np.random.default_rng(P + width + stale)
    order = rng.permutation(P)
    held = order[:min(P // 2, rows * width - 50)]
    refs = np.zeros(P, int)
    refs[held] = 1
    tables = np.full(rows * width, -1)
    at = rng.permutation(rows * width)
    tables[at[:len(held)]] = held
    holes = np.flatnonzero(refs[:len(held)] == 0)
    tables[at[len(held):len(held) + stale]] = rng.choice(holes, stale)
    tables = tables.reshape(rows, width)
    books, r, t, st = Books(refs, tables), dev(refs), dev(tables), word()
    # a workspace full of what an earlier call could have left: every number that an entry could be taken for
    ws = torch.arange(-1, P, dtype=torch.int32, device="cuda")
    src, dst = kda.pages_compact(r, t, workspace=ws, status=st)
    ws_, wd, _ = books.compact()
    assert src.tolist() == ws_ and dst.tolist() == wd and r.tolist() == books.refs
    assert t.tolist() == books.tables and int(st) == (5 if stale else 0)
