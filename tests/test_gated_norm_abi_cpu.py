"""Refusals of the gated recurrence and the group norm: bad calls return on the host before anything is launched; and what the
binding refuses (the library replaced by a recorder, tensors without memory)."""
import pytest

import kimi_delta_attention_chunk_gb300 as kda
from kimi_delta_attention_chunk_gb300 import build as kbuild
from tests.test_layer_abi_cpu import INVALID_ARG, UNSUPPORTED, WORKSPACE, at
from tests.test_layer_binding_cpu import MANY, f, i, lib as recorder, t  # noqa: F401  (a fixture)

MOST_TOKENS = 2 ** 31 - 65536 - 1
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def fwd(lib, **kw):
    a = dict(x=at(1), ldx=256, r=at(2), ldr=256, i=at(3), ldi=256, lam=at(4), z=None, ldz=0, decay=8.0, dt=1, s0=None, cu=None, B=1, T=64, C=256,
             N=1, y=at(5), fs=None, st=None)
    a.update(kw)
    return lib.kda_gated_scan_fwd(a["x"], a["ldx"], a["r"], a["ldr"], a["i"], a["ldi"], a["lam"], a["z"], a["ldz"], a["decay"], a["dt"], a["s0"],
                                  a["cu"], a["B"], a["T"], a["C"], a["N"], a["y"], a["fs"], a["st"], None)


def test_gated_scan_fwd(lib):
    assert fwd(lib, dt=2) == UNSUPPORTED and fwd(lib, C=(1 << 20) + 1, ldx=1 << 21, ldr=1 << 21, ldi=1 << 21) == UNSUPPORTED
    for d in (0.0, -1.0, NAN, INF):
        assert fwd(lib, decay=d) == INVALID_ARG
    assert fwd(lib, C=0) == INVALID_ARG and fwd(lib, B=-1, N=-1) == INVALID_ARG and fwd(lib, T=-1) == INVALID_ARG
    for k in ("ldx", "ldr", "ldi"):
        assert fwd(lib, **{k: 255}) == INVALID_ARG
    assert fwd(lib, z=at(6), ldz=255) == INVALID_ARG
    for k, n in (("x", 1), ("r", 2), ("i", 3), ("lam", 4), ("y", 5)):
        assert fwd(lib, **{k: None}) == INVALID_ARG and fwd(lib, **{k: at(n, 1)}) == INVALID_ARG
    for k in ("s0", "fs", "st"):
        assert fwd(lib, **{k: at(7, 2)}) == INVALID_ARG
    assert fwd(lib, N=2) == INVALID_ARG and fwd(lib, B=2, N=3, cu=at(8)) == INVALID_ARG and fwd(lib, cu=at(8, 2)) == INVALID_ARG
    assert fwd(lib, y=at(1, 512)) == INVALID_ARG and fwd(lib, s0=at(7), fs=at(7)) == INVALID_ARG and fwd(lib, st=at(5, 64)) == INVALID_ARG
    assert fwd(lib, T=MOST_TOKENS + 1) == INVALID_ARG
    assert fwd(lib, B=1 << 24, N=1 << 24, T=1, C=64 * 17, ldx=1088, ldr=1088, ldi=1088) == UNSUPPORTED      # blocks of one launch
    assert fwd(lib, B=0, N=0, x=None, r=None, i=None, y=None) == 0


def test_gated_scan_bwd(lib):
    need = lib.kda_gated_scan_bwd_workspace_size(1, 64, 256, 1, 0, 1)
    assert need >= 256 * 4 and lib.kda_gated_scan_bwd_workspace_size(1, 64, 256, 1, 0, 0) >= need + 2 * 256 * 4
    assert lib.kda_gated_scan_bwd_workspace_size(1, -1, 256, 1, 0, 0) == 0

    def call(**kw):
        a = dict(x=at(1), ldx=256, r=at(2), ldr=256, i=at(3), ldi=256, lam=at(4), z=None, ldz=0, decay=8.0, dt=1, s0=None, cu=None, B=1, T=64, C=256,
                 N=1, dy=at(5), dfs=None, gdt=1, st=at(6), dx=at(7), dr=at(8), di=at(9), dlam=at(10), dz=None, d0=None, ws=at(11), wsb=need)
        a.update(kw)
        return lib.kda_gated_scan_bwd(a["x"], a["ldx"], a["r"], a["ldr"], a["i"], a["ldi"], a["lam"], a["z"], a["ldz"], a["decay"], a["dt"], a["s0"],
                                      a["cu"], a["B"], a["T"], a["C"], a["N"], a["dy"], a["dfs"], a["gdt"], a["st"], a["dx"], a["dr"], a["di"],
                                      a["dlam"], a["dz"], a["d0"], a["ws"], a["wsb"], None)
    assert call(dt=0, gdt=1) == UNSUPPORTED and call(gdt=5) == UNSUPPORTED and call(dt=5) == UNSUPPORTED
    for k in ("dy", "dx", "dr", "di", "dlam"):
        assert call(**{k: None}) == INVALID_ARG
    assert call(z=at(12), ldz=256) == INVALID_ARG and call(dz=at(12)) == INVALID_ARG        # dz exactly with z
    assert call(dx=at(5)) == INVALID_ARG and call(dr=at(1)) == INVALID_ARG and call(ws=at(6)) == INVALID_ARG
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE and call(st=None) == WORKSPACE
    assert call(ws=at(11, 8)) == INVALID_ARG and call(dlam=at(10, 2)) == INVALID_ARG and call(d0=at(12, 2)) == INVALID_ARG


def test_gated_step(lib):
    def call(**kw):
        a = dict(x=at(1), ldx=256, r=at(2), ldr=256, i=at(3), ldi=256, lam=at(4), z=None, ldz=0, decay=8.0, dt=1, s=at(5), sl=at(6), P=8, N=4, C=256,
                 y=at(7), st=None)
        a.update(kw)
        return lib.kda_gated_step(a["x"], a["ldx"], a["r"], a["ldr"], a["i"], a["ldi"], a["lam"], a["z"], a["ldz"], a["decay"], a["dt"], a["s"],
                                  a["sl"], a["P"], a["N"], a["C"], a["y"], a["st"], None)
    assert call(dt=7) == UNSUPPORTED and call(N=(1 << 18) + 1) == UNSUPPORTED and call(sl=None, N=(1 << 30) + 1, P=(1 << 30) + 2) == UNSUPPORTED
    assert call(sl=None, N=1 << 30, P=1 << 30) == UNSUPPORTED                # more blocks than one launch has
    assert call(N=-1) == INVALID_ARG and call(P=0) == INVALID_ARG and call(C=-4) == INVALID_ARG and call(decay=NAN) == INVALID_ARG
    assert call(sl=None, N=9) == INVALID_ARG and call(sl=at(6, 1)) == INVALID_ARG and call(st=at(8, 3)) == INVALID_ARG
    for k in ("x", "r", "i", "lam", "s", "y"):
        assert call(**{k: None}) == INVALID_ARG
    assert call(ldr=255) == INVALID_ARG and call(z=at(9), ldz=8) == INVALID_ARG and call(y=at(5)) == INVALID_ARG and call(y=at(1)) == INVALID_ARG
    assert call(N=0, P=0, x=None, r=None, i=None, s=None, y=None) == 0


def norm(lib, bwd=False, **kw):
    a = dict(x=at(1), ldx=256, w=at(2), b=at(3), eps=1e-5, act=1, seq=0, dt=1, cu=None, B=1, T=64, C=256, G=8, N=1, y=at(4), st=None, ws=at(5), wsb=1 << 24,
             dy=at(6), gdt=1, dx=at(7), dw=at(8), db=at(9))
    a.update(kw)
    head = (a["x"], a["ldx"], a["w"], a["b"], a["eps"], a["act"], a["seq"], a["dt"], a["cu"], a["B"], a["T"], a["C"], a["G"], a["N"])
    if bwd:
        return lib.kda_group_norm_bwd(*head, a["dy"], a["gdt"], a["st"], a["dx"], a["dw"], a["db"], a["ws"], a["wsb"], None)
    return lib.kda_group_norm_fwd(*head, a["y"], a["st"], a["ws"], a["wsb"], None)


@pytest.mark.parametrize("bwd", [False, True])
def test_group_norm(lib, bwd):
    size = lib.kda_group_norm_bwd_workspace_size if bwd else lib.kda_group_norm_fwd_workspace_size
    call = lambda **kw: norm(lib, bwd, **kw)  # noqa: E731
    assert call(dt=3) == UNSUPPORTED and call(C=16385, ldx=16385, G=1) == UNSUPPORTED
    for e in (0.0, -1e-5, NAN, INF):
        assert call(eps=e) == INVALID_ARG
    assert call(G=0) == INVALID_ARG and call(G=7) == INVALID_ARG and call(act=2) == INVALID_ARG and call(seq=2) == INVALID_ARG
    assert call(ldx=255) == INVALID_ARG and call(x=None) == INVALID_ARG and call(x=at(1, 1)) == INVALID_ARG and call(w=at(2, 2)) == INVALID_ARG
    assert call(cu=at(10)) == INVALID_ARG                       # over tokens there are no sequences
    assert call(st=at(10)) == INVALID_ARG                       # and no statistics to keep
    assert call(seq=1, st=at(10, 4)) == INVALID_ARG and call(seq=1, N=2) == INVALID_ARG and call(seq=1, cu=at(10, 2)) == INVALID_ARG
    need = size(1, 64, 256, 8, 1, 1, 0, 0)
    assert need > size(1, 64, 256, 8, 1, 1, 0, 1) > 0
    assert call(seq=1, wsb=need - 1) == WORKSPACE and call(seq=1, ws=None) == WORKSPACE and call(seq=1, ws=at(5, 8)) == INVALID_ARG
    assert size(1, 64, 256, 7, 1, 1, 0, 0) == 0 and size(1, -1, 256, 8, 1, 1, 0, 0) == 0
    if bwd:
        assert call(dt=0, gdt=1) == UNSUPPORTED and call(dy=None) == INVALID_ARG and call(dx=None) == INVALID_ARG
        assert call(dx=at(6)) == INVALID_ARG and call(dw=at(8, 2)) == INVALID_ARG and call(db=at(8)) == INVALID_ARG and call(ws=at(1)) == INVALID_ARG
        assert call(wsb=size(1, 64, 256, 8, 1, 0, 0, 0) - 1) == WORKSPACE
    else:
        assert size(1, 64, 256, 8, 1, 0, 0, 0) == 0
        assert call(y=None) == INVALID_ARG and call(y=at(1)) == INVALID_ARG and call(y=at(4, 1)) == INVALID_ARG
        assert call(B=0, N=0, x=None, y=None) == 0


def test_binding(recorder):  # noqa: F811
    C = 16
    x = t(1, 5, C)
    for bad in (t(5, C), t(1, 5, 2, C)):
        with pytest.raises(ValueError):
            kda.gated_scan_fwd(bad, bad, bad, f(C))
        with pytest.raises(ValueError):
            kda.gated_scan_bwd(bad, bad, bad, f(C), bad)
    for bad in (t(1, 5, C), t(C)):
        with pytest.raises(ValueError, match=r"\[N, 16\]"):
            kda.gated_step(bad, bad, bad, f(C), f(4, C))
    with pytest.raises(ValueError):
        kda.gated_scan_fwd(x, x, t(1, 5, C + 1), f(C))
    with pytest.raises(TypeError):
        kda.gated_scan_fwd(x, x, f(1, 5, C), f(C))
    with pytest.raises(TypeError):
        kda.gated_scan_fwd(x, x, x, t(C))
    with pytest.raises(ValueError):
        kda.gated_scan_fwd(x, x, x, f(C), states=f(1, 2, C))
    with pytest.raises(TypeError):
        kda.gated_scan_fwd(x, x, x, f(C), initial_state=t(1, C))
    with pytest.raises(ValueError):
        kda.gated_step(t(2, C), t(2, C), t(2, C), f(C), f(4, C + 1))
    with pytest.raises(ValueError, match="over"):
        kda.group_norm_fwd(x, 4, over="batch")
    with pytest.raises(ValueError):
        kda.group_norm_fwd(x, 4, cu_seqlens=i(2))
    with pytest.raises(ValueError):
        kda.group_norm_fwd(t(5, C), 4, over="sequence")
    with pytest.raises(ValueError):
        kda.group_norm_fwd(x, 4, weight=f(C + 1))
    with pytest.raises(TypeError):
        kda.group_norm_bwd(x, 4, x, bias=t(C))
    with pytest.raises(ValueError):
        kda.group_norm_bwd(x, 4, t(1, 4, C))
    with pytest.raises(ValueError):
        kda.group_norm_fwd(x, 4, over="sequence", stats=f(1, 4))
    big, one = t(1, MANY, 1), f(1)
    for call in (lambda: kda.gated_scan_fwd(big, big, big, one), lambda: kda.gated_scan_bwd(big, big, big, one, big),
                 lambda: kda.gated_step(big[0], big[0], big[0], one, f(MANY, 1)), lambda: kda.group_norm_fwd(big, 1),
                 lambda: kda.group_norm_bwd(big, 1, big), lambda: kda.group_norm_fwd(x, MANY)):
        with pytest.raises(ValueError, match="2\\*\\*31"):
            call()
    assert recorder.calls == []
    kda.gated_scan_fwd(x, x, x, f(C), z=x, states=f(1, 1, C))
    kda.group_norm_fwd(t(3, C), 4)
    assert recorder.names() == ["kda_gated_scan_fwd", "kda_group_norm_fwd"]
