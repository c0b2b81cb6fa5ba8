"""Workspaces of the group norm over sequences: what they hold and no more.  Nothing here reaches a launch."""
import pytest

import kimi_delta_attention_chunk_gb300 as kda
from kimi_delta_attention_chunk_gb300 import build as kbuild


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


@pytest.mark.parametrize("T,C,G", [(65536, 12288, 1), (4096, 4979, 13), (100, 512, 32), (64, 8, 8)])
def test_a_sequence_more(lib, T, C, G):
    """costs one place of sums a channel (two of them, fp32), and two numbers a group for each of the means and the statistics."""
    for name, stats, means in (("kda_group_norm_fwd_workspace_size", 1, 0), ("kda_group_norm_bwd_workspace_size", 1, 1)):
        size = getattr(lib, name)
        for kept in (0, 1):
            few, many = 1, 65536
            more = size(1, T, C, G, many, 1, 1, kept) - size(1, T, C, G, few, 1, 1, kept)
            want = (many - few) * (2 * C * 4 + (stats * (1 - kept) + means) * G * 8)
            assert abs(more - want) <= 4 * 256, name  # (every part is rounded up to 256 bytes)


@pytest.mark.parametrize("T,C,G", [(65536, 12288, 1), (700, 4979, 13), (700, 3333, 33), (100, 512, 32), (64, 8, 8)])
def test_runs(lib, T, C, G):
    """Backwards as many places again for the sums a run, and the sequence's means: with no sequences, twice the forward pass's."""
    bwd, fwd = (getattr(lib, f"kda_group_norm_{k}_workspace_size") for k in ("bwd", "fwd"))
    places = fwd(1, T, C, G, 0, 1, 1, 1)
    assert places >= 2 * C * 4 and bwd(1, T, C, G, 0, 1, 1, 1) == 2 * places
