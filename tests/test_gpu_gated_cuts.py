"""The gated linear recurrence over sequences that are walked as one stream: what is not a number or infinite stays in its
sequence, and gradients in fp32 beside bf16 rows."""
import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from tests.gated_norm_ref import within
from tests.test_gpu_gated_scan import BF16, F32, args, make, ref_of
from tests.test_gpu_gated_streams import cumulative

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
# sequences too short for blocks of their own: one tile, several of a cluster, blocks of 64, 32 and 16 channels
SHORT = [([8] * 60, 64), ([8] * 300, 64), ([3, 20, 1, 0, 7, 16] * 12, 1024), ([8] * 60, 2048), ([5] * 90, 33)]


def calls(d, dy, cu, initial, dfinal, kept):
    states = torch.zeros(kda.gated_scan_states(d["x"]), device="cuda")
    y, final = kda.gated_scan_fwd(*args(d), z=d["z"], initial_state=initial, cu_seqlens=cu, states=states)
    out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], initial_state=initial, cu_seqlens=cu, dfinal_state=dfinal, states=states if kept else None)
    rows = {"y": y, **{k: out[k] for k in ("dx", "dr", "di", "dz")}}
    return rows, {"final": final, "dinitial": out["dinitial_state"]}


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("lens,C", SHORT)
def test_not_a_number_or_infinite_stays_in_its_sequence(lens, C, dtype):
    T, N = sum(lens), len(lens)
    offsets = cumulative(lens)
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    d = make((1, T), C, dtype, 41, True)
    g = torch.Generator().manual_seed(T)
    rn = lambda *shape: torch.randn(*shape, generator=g)  # noqa: E731
    dy, initial, dfinal = rn(1, T, C).to(dtype).cuda(), rn(N, C).cuda(), rn(N, C).cuda()
    want = {kept: calls(d, dy, cu, initial, dfinal, kept) for kept in (True, False)}
    for n in (1, N // 2 - N // 2 % 6 + 1, N - 1):  # (one with tokens)
        first, last = offsets[n], offsets[n + 1]
        at = (first + last) // 2
        others = torch.tensor([not first <= t < last for t in range(T)], device="cuda")
        rest = torch.arange(N, device="cuda") != n
        for what, bad in (("x", NAN), ("x", INF), ("x", -INF), ("r", NAN), ("r", INF), ("i", NAN), ("z", INF), ("dy", NAN), ("dy", -INF), ("initial", NAN),
                          ("initial", INF), ("dfinal", NAN), ("dfinal", -INF)):
            e, given = dict(d), {"dy": dy, "initial": initial, "dfinal": dfinal}
            at_row = (0, at) if what not in ("initial", "dfinal") else (n,)
            to = e if what in e else given
            to[what] = to[what].clone()
            to[what][at_row] = bad
            for kept in (True, False):
                rows, states = calls(e, given["dy"], cu, given["initial"], given["dfinal"], kept)
                for k, v in rows.items():
                    assert torch.equal(v[:, others], want[kept][0][k][:, others]), (what, bad, n, kept, k)
                for k, v in states.items():
                    assert torch.equal(v[rest], want[kept][1][k][rest]), (what, bad, n, kept, k)
                if what == "x":
                    assert not bool(torch.isfinite(rows["y"][:, at:last]).any()) and not bool(torch.isfinite(states["final"][n]).any())
                    assert torch.equal(rows["y"][:, first:at], want[kept][0]["y"][:, first:at])
                if what == "dy":
                    assert not bool(torch.isfinite(rows["dx"][:, first:at + 1]).any()) and not bool(torch.isfinite(states["dinitial"][n]).any())
                    assert torch.equal(rows["dx"][:, at + 1:last], want[kept][0]["dx"][:, at + 1:last])


@pytest.mark.parametrize("lens,C", [([8] * 60, 64), ([130] * 20, 72), ([320, 96, 33], 1536), ([1] * 10 + [2500] + [3] * 9, 72), ([65, 0, 127, 1, 3], 33)])
def test_gradients_in_fp32_beside_bf16_rows(lens, C):
    T, N = sum(lens), len(lens)
    offsets = cumulative(lens)
    d = make((1, T), C, BF16, T + C, True)
    g = torch.Generator().manual_seed(T)
    dy, initial, dfinal = (torch.randn(*s, generator=g).cuda() for s in ((1, T, C), (N, C), (N, C)))
    cu = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    states = torch.empty(kda.gated_scan_states(d["x"]), device="cuda")
    kda.gated_scan_fwd(*args(d), z=d["z"], initial_state=initial, cu_seqlens=cu, states=states)
    ref = ref_of(d, C, initial, offsets, dy, dfinal)
    for kept in (states, None):
        out = kda.gated_scan_bwd(*args(d), dy, z=d["z"], initial_state=initial, cu_seqlens=cu, dfinal_state=dfinal, states=kept)
        for k in ("dx", "dr", "di", "dz"):
            assert out[k].dtype == F32
            within(out[k], ref[k], ref[k + "_err"], F32, k)
        within(out["dlam"], ref["dlam"], ref["dlam_err"], F32, "dlam")
        within(out["dinitial_state"], ref["dinitial_state"], ref["dinitial_state_err"], F32, "dinitial")
