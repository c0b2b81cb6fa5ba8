"""Refusals of the recurrent layer's operators (short convolution, selective scan, decode by slot,
pages of a cache): bad calls return on the host before anything is launched."""
import ctypes

import pytest
import torch

import kimi_delta_attention_chunk_gb300 as kda
from kimi_delta_attention_chunk_gb300 import build as kbuild

INVALID_ARG, UNSUPPORTED, WORKSPACE = 1, 2, 3


def at(i, off=0):
    """Fake, far apart, never dereferenced addresses."""
    return ctypes.c_void_p((i << 36) + off)


@pytest.fixture(scope="module")
def lib():
    kbuild.build()
    return kda.load_library()


def test_conv_fwd(lib):
    def call(**kw):
        a = dict(x=at(1), ldx=256, w=at(2), b=None, act=1, dt=1, h=None, cu=None, B=1, T=64, C=256, W=4, N=1, y=at(3), f=None)
        a.update(kw)
        return lib.kda_short_conv_fwd(a["x"], a["ldx"], a["w"], a["b"], a["act"], a["dt"], a["h"], a["cu"], a["B"], a["T"],
                                      a["C"], a["W"], a["N"], a["y"], a["f"], None)
    assert call(dt=2) == UNSUPPORTED
    assert call(W=1) == UNSUPPORTED and call(W=5) == UNSUPPORTED
    assert call(C=(1 << 20) + 1, ldx=1 << 21) == UNSUPPORTED
    assert call(C=0) == INVALID_ARG and call(B=-1) == INVALID_ARG and call(T=-1) == INVALID_ARG and call(N=-1) == INVALID_ARG
    assert call(ldx=255) == INVALID_ARG
    assert call(act=2) == INVALID_ARG
    assert call(x=None) == INVALID_ARG and call(y=None) == INVALID_ARG and call(w=None) == INVALID_ARG
    assert call(x=at(1, 1)) == INVALID_ARG and call(w=at(2, 2)) == INVALID_ARG
    assert call(N=2) == INVALID_ARG                          # N must equal B without cu_seqlens
    assert call(B=2, N=3, cu=at(4)) == INVALID_ARG           # packed sequences need B == 1
    assert call(cu=at(4, 2)) == INVALID_ARG
    assert call(B=1 << 15, T=1 << 16, N=1 << 15) == INVALID_ARG
    assert call(y=at(1, 512)) == INVALID_ARG                 # y over x
    assert call(h=at(5), f=at(5)) == INVALID_ARG             # the final history over the initial one
    assert call(y=at(3), f=at(3, 64)) == INVALID_ARG         # two outputs over each other
    assert call(B=0, N=0, x=None, y=None) == 0               # nothing to do


def test_conv_bwd(lib):
    need = lib.kda_short_conv_bwd_workspace_size(1, 64, 256, 4)
    # two runs of 32 tokens: W + 1 sums a channel each
    assert need == 2 * 256 * 5 * 4
    assert lib.kda_short_conv_bwd_workspace_size(1, 64, 256, 5) == 0
    # rows in 16-byte pieces: two runs; element by element: three, the more
    assert lib.kda_short_conv_bwd_workspace_size(1, 700, 228 * 512, 4) == 3 * 228 * 512 * 5 * 4
    assert lib.kda_short_conv_bwd_workspace_size(1, -1, 256, 4) == 0

    def call(**kw):
        a = dict(x=at(1), ldx=256, w=at(2), b=None, act=1, dt=1, h=None, cu=None, B=1, T=64, C=256, W=4, N=1, dy=at(3), df=None,
                 gdt=1, dx=at(4), dw=at(5), db=None, di=None, ws=at(6), wsb=need)
        a.update(kw)
        return lib.kda_short_conv_bwd(a["x"], a["ldx"], a["w"], a["b"], a["act"], a["dt"], a["h"], a["cu"], a["B"], a["T"],
                                      a["C"], a["W"], a["N"], a["dy"], a["df"], a["gdt"], a["dx"], a["dw"], a["db"], a["di"],
                                      a["ws"], a["wsb"], None)
    assert call(dt=0, gdt=1) == UNSUPPORTED                  # bf16 gradients of fp32 inputs
    assert call(gdt=3) == UNSUPPORTED and call(W=6) == UNSUPPORTED
    assert call(dy=None) == INVALID_ARG and call(dx=None) == INVALID_ARG and call(dw=None) == INVALID_ARG
    assert call(dw=at(5, 2)) == INVALID_ARG and call(df=at(7, 1)) == INVALID_ARG
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(ws=at(6, 8)) == INVALID_ARG
    assert call(dx=at(3)) == INVALID_ARG                     # in place over dy
    assert call(ws=at(1)) == INVALID_ARG


def test_conv_step(lib):
    def call(**kw):
        a = dict(x=at(1), ldx=256, w=at(2), b=None, act=1, dt=1, h=at(3), sl=at(4), P=8, N=4, C=256, W=4, y=at(5), st=None)
        a.update(kw)
        return lib.kda_short_conv_step(a["x"], a["ldx"], a["w"], a["b"], a["act"], a["dt"], a["h"], a["sl"], a["P"], a["N"],
                                       a["C"], a["W"], a["y"], a["st"], None)
    assert call(dt=7) == UNSUPPORTED and call(W=8) == UNSUPPORTED
    assert call(N=-1) == INVALID_ARG and call(P=0) == INVALID_ARG and call(C=-4) == INVALID_ARG
    assert call(N=(1 << 30) + 1) == UNSUPPORTED
    assert call(sl=None, N=9) == INVALID_ARG                 # more rows than pages
    assert call(sl=at(4, 1)) == INVALID_ARG and call(st=at(6, 3)) == INVALID_ARG
    assert call(h=None) == INVALID_ARG and call(y=at(3)) == INVALID_ARG
    assert call(N=0, x=None, h=None, y=None, P=0) == 0


def test_ssm_step(lib):
    def call(**kw):
        a = dict(u=at(1), ldu=256, d=at(2), ldd=256, A=at(3), B=at(4), ldb=32, C=at(5), ldc=32, D=None, z=None, ldz=0, b=None,
                 sp=1, dt=1, s=at(6), sl=at(7), P=8, N=4, c=256, G=2, S=16, y=at(8), st=None)
        a.update(kw)
        return lib.kda_ssm_step(a["u"], a["ldu"], a["d"], a["ldd"], a["A"], a["B"], a["ldb"], a["C"], a["ldc"], a["D"], a["z"],
                                a["ldz"], a["b"], a["sp"], a["dt"], a["s"], a["sl"], a["P"], a["N"], a["c"], a["G"], a["S"],
                                a["y"], a["st"], None)
    assert call(S=12) == UNSUPPORTED and call(S=128, ldb=256, ldc=256) == UNSUPPORTED and call(dt=5) == UNSUPPORTED
    assert call(G=3) == INVALID_ARG and call(G=0) == INVALID_ARG
    assert call(N=1 << 30, P=1 << 30) == UNSUPPORTED         # more blocks than one launch has
    assert call(N=(1 << 31) - 1, c=1, G=1) == UNSUPPORTED
    assert call(sp=2) == INVALID_ARG
    assert call(ldu=255) == INVALID_ARG and call(ldb=31) == INVALID_ARG and call(z=at(9), ldz=100) == INVALID_ARG
    assert call(A=at(3, 4)) == INVALID_ARG and call(s=at(6, 16)) == INVALID_ARG
    assert call(s=None) == INVALID_ARG and call(A=None) == INVALID_ARG
    assert call(sl=None, N=9) == INVALID_ARG
    assert call(y=at(1)) == INVALID_ARG and call(y=at(6)) == INVALID_ARG
    assert call(N=0, P=0, u=None, s=None) == 0


def scan(lib, **kw):
    a = dict(u=at(1), ldu=256, d=at(2), ldd=256, A=at(3), B=at(4), ldb=32, C=at(5), ldc=32, D=None, z=None, ldz=0, b=None, sp=1, dt=1,
             s0=None, cu=None, nb=1, T=64, c=256, G=2, S=16, N=1, y=at(8), sT=None, ws=at(9), wsb=1 << 30)
    a.update(kw)
    return lib.kda_ssm_scan_fwd(a["u"], a["ldu"], a["d"], a["ldd"], a["A"], a["B"], a["ldb"], a["C"], a["ldc"], a["D"], a["z"],
                                a["ldz"], a["b"], a["sp"], a["dt"], a["s0"], a["cu"], a["nb"], a["T"], a["c"], a["G"], a["S"],
                                a["N"], a["y"], a["sT"], a["ws"], a["wsb"], None)


def test_scan_fwd(lib):
    assert scan(lib, S=4) == UNSUPPORTED and scan(lib, dt=9) == UNSUPPORTED and scan(lib, c=(1 << 20) + 2) == UNSUPPORTED
    assert scan(lib, G=3) == INVALID_ARG and scan(lib, T=-1) == INVALID_ARG and scan(lib, N=2) == INVALID_ARG
    assert scan(lib, nb=2, N=2, cu=at(7)) == INVALID_ARG
    assert scan(lib, ldu=255) == INVALID_ARG and scan(lib, ldc=31) == INVALID_ARG and scan(lib, z=at(6), ldz=9) == INVALID_ARG
    assert scan(lib, A=at(3, 4)) == INVALID_ARG and scan(lib, s0=at(6, 4)) == INVALID_ARG and scan(lib, sT=at(6, 4)) == INVALID_ARG
    assert scan(lib, A=None) == INVALID_ARG and scan(lib, y=None) == INVALID_ARG and scan(lib, sp=3) == INVALID_ARG
    assert scan(lib, s0=at(6), sT=at(6)) == INVALID_ARG      # the final state over the initial one
    assert scan(lib, y=at(1)) == INVALID_ARG
    need = lib.kda_ssm_scan_fwd_workspace_size(1, 4096, 256, 2, 16, 1, 0)
    assert need > 0 and scan(lib, T=4096, wsb=need - 1) == WORKSPACE and scan(lib, T=4096, ws=None) == WORKSPACE
    assert scan(lib, T=4096, ws=at(9, 8)) == INVALID_ARG
    # one run, or sequences enough: none
    assert lib.kda_ssm_scan_fwd_workspace_size(1, 64, 256, 2, 16, 1, 0) == 0
    assert lib.kda_ssm_scan_fwd_workspace_size(1000, 512, 256, 2, 16, 1000, 0) == 0
    assert lib.kda_ssm_scan_fwd_workspace_size(1, 4096, 256, 3, 16, 1, 0) == 0
    assert scan(lib, nb=0, N=0, u=None, d=None, B=None, C=None, y=None, ws=None, wsb=0) == 0


def test_scan_bwd(lib):
    need = lib.kda_ssm_scan_bwd_workspace_size(1, 64, 256, 2, 16, 1, 0)
    # four chunks: states, gradients and middle states, two sums of d, dD and dbias, four channel blocks' dB and dC, flags
    assert need == 4 * (3 * 256 * 16 * 4 + 4 * 256 * 4) + 4 * 64 * 32 * 4 + 256

    def call(**kw):
        a = dict(u=at(1), A=at(3), z=None, ldz=0, dt=1, T=64, c=256, G=2, S=16, N=1, dy=at(10), df=None, gdt=1, du=at(11), dd=at(12),
                 dA=at(13), dB=at(14), dC=at(15), dD=None, dz=None, db=None, d0=None, ws=at(16), wsb=need)
        a.update(kw)
        return lib.kda_ssm_scan_bwd(a["u"], 256, at(2), 256, a["A"], at(4), 32, at(5), 32, None, a["z"], a["ldz"], None, 1, a["dt"],
                                    None, None, 1, a["T"], a["c"], a["G"], a["S"], a["N"], a["dy"], a["df"], a["gdt"], a["du"],
                                    a["dd"], a["dA"], a["dB"], a["dC"], a["dD"], a["dz"], a["db"], a["d0"], a["ws"], a["wsb"], None)
    assert call(S=20) == UNSUPPORTED and call(dt=0, gdt=1) == UNSUPPORTED and call(gdt=2) == UNSUPPORTED
    assert call(T=65535 * 64 + 1) == UNSUPPORTED
    assert call(dA=None) == INVALID_ARG and call(du=None) == INVALID_ARG and call(dB=None) == INVALID_ARG
    assert call(z=at(6), ldz=256) == INVALID_ARG             # z without dz
    assert call(dz=at(6)) == INVALID_ARG                     # dz without z
    assert call(d0=at(17, 4)) == INVALID_ARG and call(df=at(17, 8)) == INVALID_ARG
    assert call(wsb=need - 1) == WORKSPACE and call(ws=None) == WORKSPACE
    assert call(du=at(10)) == INVALID_ARG and call(dB=at(14), dC=at(14)) == INVALID_ARG


def test_recurrent_step_slots(lib):
    def call(**kw):
        a = dict(q=at(1), pool=at(2), sl=at(3), P=8, N=4, H=2, K=128, V=128, dt=1, st=None)
        a.update(kw)
        return lib.kda_recurrent_step_slots(a["q"], at(4), at(5), at(6), at(7), a["dt"], 0.0, a["pool"], a["sl"], a["P"], a["N"],
                                            a["H"], a["K"], a["V"], at(8), 0, a["st"], None)
    assert call(K=96) == UNSUPPORTED and call(dt=4) == UNSUPPORTED
    assert call(q=None) == INVALID_ARG and call(pool=at(2, 8)) == INVALID_ARG
    assert call(sl=None) == INVALID_ARG and call(sl=at(3, 2)) == INVALID_ARG and call(st=at(9, 1)) == INVALID_ARG
    assert call(P=0) == INVALID_ARG and call(P=-1) == INVALID_ARG
    assert call(N=1 << 30, H=4) == INVALID_ARG
    assert call(N=0, sl=None, P=0) == 0


def test_pages(lib):
    assert lib.kda_pages_alloc(at(1), -1, 4, at(2), None, None) == INVALID_ARG
    assert lib.kda_pages_alloc(None, 8, 4, at(2), None, None) == INVALID_ARG
    assert lib.kda_pages_alloc(at(1), 8, 4, None, None, None) == INVALID_ARG
    assert lib.kda_pages_alloc(at(1), 8, 4, at(1), None, None) == INVALID_ARG
    assert lib.kda_pages_alloc(at(1), 8, 4, at(2, 2), None, None) == INVALID_ARG
    assert lib.kda_pages_alloc(at(1), 8, 0, None, None, None) == 0
    many = (1 << 30) + 1
    assert lib.kda_pages_alloc(at(1), many, 4, at(9), None, None) == UNSUPPORTED
    assert lib.kda_pages_alloc(at(1), 8, many, at(9), None, None) == UNSUPPORTED
    assert lib.kda_pages_free(at(1), many, at(9), 3, None, None) == UNSUPPORTED
    assert lib.kda_pages_free(at(1), 8, None, 3, None, None) == INVALID_ARG
    assert lib.kda_pages_free(at(1), 8, at(1), 3, None, None) == INVALID_ARG
    assert lib.kda_pages_free(at(1), 8, at(2), 3, at(3, 2), None) == INVALID_ARG
    assert lib.kda_pages_free(at(1), 8, None, 0, None, None) == 0

    def fork(**kw):
        a = dict(t=at(1), l=at(2), S=4, w=3, pt=16, r=at(3), P=16, p=at(4), c=at(5), n=2, s=at(6), d=at(7), st=None)
        a.update(kw)
        return lib.kda_pages_fork(a["t"], a["l"], a["S"], a["w"], a["pt"], a["r"], a["P"], a["p"], a["c"], a["n"], a["s"], a["d"],
                                  a["st"], None)
    assert fork(w=0) == INVALID_ARG and fork(pt=0) == INVALID_ARG and fork(n=-1) == INVALID_ARG
    assert fork(n=65537) == UNSUPPORTED and fork(P=many, r=at(20)) == UNSUPPORTED
    assert fork(t=None) == INVALID_ARG and fork(r=None) == INVALID_ARG and fork(p=None) == INVALID_ARG
    assert fork(s=at(7)) == INVALID_ARG and fork(l=at(2, 1)) == INVALID_ARG
    assert fork(n=0) == 0

    need = lib.kda_pages_compact_workspace_size(100)
    assert need == 404 and lib.kda_pages_compact_workspace_size(0) == 0

    def compact(**kw):
        a = dict(r=at(1), P=100, t=at(2), e=12, s=at(3), d=at(4), ws=at(5), wsb=need, st=None)
        a.update(kw)
        return lib.kda_pages_compact(a["r"], a["P"], a["t"], a["e"], a["s"], a["d"], a["ws"], a["wsb"], a["st"], None)
    assert compact(t=None) == INVALID_ARG and compact(r=None) == INVALID_ARG and compact(s=None) == INVALID_ARG
    assert compact(e=-1) == INVALID_ARG and compact(P=many) == UNSUPPORTED
    assert compact(wsb=need - 1) == WORKSPACE and compact(ws=None) == WORKSPACE
    assert compact(ws=at(5, 4)) == INVALID_ARG and compact(ws=at(1)) == INVALID_ARG
    assert compact(P=0, r=None, s=None, d=None, ws=None, wsb=0) == 0

    need = lib.kda_pages_copy_workspace_size(100, 300)
    assert need == (1 + 200 + 300) * 4 and lib.kda_pages_copy_workspace_size(100, 0) == 0
    assert lib.kda_pages_copy_workspace_size(100, 128) == 0      # few pairs need none

    def copy(**kw):
        a = dict(p=at(1), P=100, b=64, s=at(2), d=at(3), n=300, ws=at(4), wsb=need, st=None)
        a.update(kw)
        return lib.kda_pages_copy(a["p"], a["P"], a["b"], a["s"], a["d"], a["n"], a["ws"], a["wsb"], a["st"], None)
    assert copy(b=24) == UNSUPPORTED and copy(n=many) == UNSUPPORTED and copy(P=many) == UNSUPPORTED
    assert copy(b=0) == INVALID_ARG and copy(p=None) == INVALID_ARG and copy(p=at(1, 8)) == INVALID_ARG
    assert copy(s=None) == INVALID_ARG and copy(d=at(3, 1)) == INVALID_ARG
    assert copy(wsb=need - 1) == WORKSPACE and copy(ws=at(2)) == INVALID_ARG
    assert copy(n=0, s=None, d=None, ws=None, wsb=0) == 0


def test_binding_refuses_what_it_cannot_pass_on(lib):
    x, w = torch.zeros(1, 8, 32), torch.zeros(32, 4)
    with pytest.raises(ValueError):
        kda.short_conv_fwd(x, w)                             # not on a device
    with pytest.raises(TypeError):
        kda.short_conv_fwd(x, w.double())
    with pytest.raises(ValueError):
        kda.short_conv_fwd(x, torch.zeros(31, 4))
    with pytest.raises(ValueError):
        kda.pages_free(torch.zeros(4, dtype=torch.int32), torch.zeros(4, dtype=torch.int32))
    q, s = torch.zeros(2, 3, 64), torch.zeros(2, 3, 64, 64)
    with pytest.raises(ValueError):
        kda.recurrent_step(q, q, q, q, q[..., 0], s, status=torch.zeros(1, dtype=torch.int32))


def test_rows_of_a_slice():
    from kimi_delta_attention_chunk_gb300.kda import _rows
    wide = torch.zeros(2, 5, 12)
    assert _rows("x", wide[:, :, 4:8], 2)[1] == 12
    assert _rows("x", wide[:, :1, 4:8], 2)[1] == 60          # one row a batch
    assert _rows("x", wide[:1, :1, :4], 2)[1] == 4
    assert _rows("x", torch.zeros(2, 0, 4), 2)[1] == 4
    assert _rows("b", torch.zeros(5, 2, 3, 4)[:, 1], 1)[1] == 24
    with pytest.raises(ValueError):
        _rows("x", wide[:, :4, :4], 2)                       # batches a different stride apart than rows
    with pytest.raises(ValueError):
        _rows("x", wide[:, :, ::2], 2)                       # elements apart
    with pytest.raises(ValueError):
        _rows("x", torch.zeros(1, 1, 4).expand(1, 5, 4), 2)  # one row for all
