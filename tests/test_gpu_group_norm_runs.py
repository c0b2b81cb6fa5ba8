"""Group norm over sequences where channels alone nearly fill the machine and tokens are cut in runs by whole fillings of it, and
with offsets that are out of order."""
import numpy as np
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.test_gpu_group_norm import BF16, F32, check, make

pytestmark = pytest.mark.gpu


# (odd channel counts go one by one, 32 to a block: 105, 156 and 182 blocks for 456 places forwards and 304 backwards)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("C,G", [(3333, 33), (3333, 1), (4979, 13), (4979, 1), (5797, 11)])
@pytest.mark.parametrize("lens", [[700], [65, 0, 200, 3, 1, 431], [64, 64, 257]])
def test_runs_by_whole_fillings(lens, C, G, dtype):
    T = sum(lens)
    cu = np.concatenate([[0], np.cumsum(lens)])
    x, w, b, dy = make((1, T), C, dtype, T + C, True)
    k = 64 + T // 32 + T * C // G // 64 // 64
    check(x, G, w, b, dy, 1, list(zip(cu, cu[1:])), "sequence", k, dtype, cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("C,G", [(72, 9), (33, 3), (512, 1), (4979, 13)])
def test_offsets_that_are_not_sorted(C, G):
    """Results are then undefined, but nothing outside the tensors is touched and the call ends."""
    T = 600
    x, w, b, dy = make((1, T), C, BF16, 78, True)
    dy = dy.to(BF16).cuda()
    for cu in ([0, 400, 100, 600], [600, 0, 300, 0], [-5, 700, 90, 1000], [600, 600, 0, 0], [0, 2 ** 31 - 1, -2 ** 31, 5]):
        N = len(cu) - 1
        kw = dict(over="sequence", cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        y = torch.full((3, T, C), 2.0, dtype=BF16, device="cuda")
        stats = torch.full((3, N, G, 2), 2.0, device="cuda")
        need = kda.load_library().kda_group_norm_bwd_workspace_size(1, T, C, G, N, 1, 1, 1)
        room = torch.full((need + 8192,), 7, dtype=torch.uint8, device="cuda")
        kda.group_norm_fwd(x, G, weight=w, bias=b, act=1, y=y[1:2], stats=stats[1], workspace=room[4096:4096 + need], **kw)
        kda.group_norm_bwd(x, G, dy, weight=w, bias=b, act=1, stats=stats[1], workspace=room[4096:4096 + need], **kw)
        torch.cuda.synchronize()
        assert bool((y[::2] == 2).all()) and bool((stats[::2] == 2).all())
        assert bool((room[:4096] == 7).all()) and bool((room[4096 + need:] == 7).all())
