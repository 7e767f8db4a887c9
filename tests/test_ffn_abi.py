"""CPU checks of the feed-forward entry points: arguments are refused, with
the stated code, before any HIP call; workspaces are sized."""
import os

import pytest

P, Q = 0x100000, 0x200000  # aligned fake device addresses: never dereferenced
INVALID, UNSUPPORTED, MISALIGNED, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def L():
    import quantized_linear_layer_scaled_amd as q
    if not os.path.exists(q.LIB_PATH):
        from quantized_linear_layer_scaled_amd import build
        build.build()
    return q.load_library()


def linear(L, A=P, B=P, bias=None, res=None, act=0, out=Q, od=0, M=16, N=64, K=128, ws=None, wsb=0):
    return L.gemm_bf16_epilogue(A, B, bias, res, act, out, od, M, N, K, ws, wsb, None)


def linear8(L, A=P, B=P, sa=P, sb=P, bias=None, res=None, act=0, out=Q, od=0, M=16, N=64, K=128, ws=None,
            wsb=0):
    return L.gemm_fp8_epilogue(A, B, sa, sb, bias, res, act, out, od, M, N, K, ws, wsb, None)


def linear_bwd(L, A=P, B=P, d=P, bias=None, act=4, dA=Q, dB=Q, db=None, M=16, N=64, K=128, ws=P, wsb=1 << 40):
    return L.gemm_bf16_epilogue_backward(A, B, d, bias, act, dA, dB, db, M, N, K, ws, wsb, None)


def gated(L, A=P, G=P, U=P, act=4, out=Q, od=0, M=16, N=64, K=128):
    return L.gated_bf16(A, G, U, act, out, od, M, N, K, None)


def gated8(L, A=P, G=P, U=P, sa=P, sg=P, su=P, act=4, out=Q, od=0, M=16, N=64, K=128):
    return L.gated_fp8(A, G, U, sa, sg, su, act, out, od, M, N, K, None)


def gated_bwd(L, A=P, G=P, U=P, d=P, act=4, dA=Q, dG=Q, dU=Q, M=16, N=64, K=128, ws=P, wsb=1 << 40):
    return L.gated_bf16_backward(A, G, U, d, act, dA, dG, dU, M, N, K, ws, wsb, None)


def norm(L, y=P, r=P, rd=0, w1=None, g=None, w2=P, al=1.0, be=1.0, eps=1e-6, ro=Q, no=Q, ns=None, M=16, K=128):
    return L.residual_norm(y, r, rd, w1, g, w2, al, be, eps, ro, no, ns, M, K, None)


def norm_bwd(L, y=P, r=P, rd=0, w1=None, g=None, w2=P, al=1.0, be=1.0, eps=1e-6, dn=P, do=P, dy=Q, dr=Q,
             dw1=None, dg=None, dw2=Q, M=16, K=128, ws=P, wsb=1 << 40):
    return L.residual_norm_backward(y, r, rd, w1, g, w2, al, be, eps, dn, do, dy, dr, dw1, dg, dw2, M, K, ws,
                                    wsb, None)


@pytest.mark.parametrize("f", [linear, linear8, linear_bwd, gated, gated8, gated_bwd])
def test_products_refuse_sizes(L, f):
    for bad in (dict(M=-1), dict(N=0), dict(N=-8), dict(K=0), dict(K=-16), dict(K=132), dict(act=-1),
                dict(act=6), dict(M=1 << 31), dict(N=1 << 31), dict(M=1 << 29, N=1 << 29)):
        assert f(L, **bad) == INVALID, bad
    assert f(L, K=1 << 24, M=1) == UNSUPPORTED


@pytest.mark.parametrize("f", [linear, linear8, gated, gated8])
def test_forward_products(L, f):
    assert f(L, M=0) == 0
    assert f(L, M=0, A=None, out=None) == 0
    for bad in (dict(A=None), dict(out=None), dict(od=2), dict(od=-1)):
        assert f(L, **bad) == INVALID, bad
    for bad in (dict(A=P + 8), dict(out=Q + 4)):
        assert f(L, **bad) == MISALIGNED, bad


def test_forward_details(L):
    assert linear8(L, K=136) == INVALID  # e4m3 rows are whole 16-byte chunks
    for f in (linear, linear8):
        assert f(L, B=None) == INVALID
        assert f(L, bias=P + 2) == MISALIGNED
        assert f(L, res=P + 2) == MISALIGNED
    assert linear8(L, sa=None) == INVALID and linear8(L, sb=P + 2) == MISALIGNED
    assert gated(L, U=None) == INVALID and gated(L, G=P + 8) == MISALIGNED
    assert gated8(L, su=None) == INVALID and gated8(L, sg=P + 1) == MISALIGNED


@pytest.mark.parametrize("fp8", [0, 1])
def test_split_k_workspace(L, fp8):
    f = linear8 if fp8 else linear
    M, N, K = 80, 64, 16384
    need = L.qll_epilogue_workspace_bytes(fp8, M, N, K)
    assert need > 0 and need % (M * N * 4) == 0
    assert f(L, M=M, N=N, K=K) == WORKSPACE
    assert f(L, M=M, N=N, K=K, ws=P, wsb=need - 1) == WORKSPACE
    assert f(L, M=M, N=N, K=K, ws=P + 8, wsb=need) == MISALIGNED
    assert L.qll_epilogue_workspace_bytes(fp8, 16, N, K) == 0
    assert L.qll_epilogue_workspace_bytes(fp8, 0, N, K) == 0
    assert L.qll_epilogue_workspace_bytes(fp8, M, N, 20) == -INVALID
    assert L.qll_epilogue_workspace_bytes(fp8, M, N, 1 << 24) == -UNSUPPORTED


def test_linear_backward_refusals(L):
    assert linear_bwd(L, N=60) == INVALID
    assert linear_bwd(L, dA=None, dB=None) == INVALID
    assert linear_bwd(L, M=0, dB=None) == 0
    for bad in (dict(A=None), dict(B=None), dict(d=None)):
        assert linear_bwd(L, **bad) == INVALID, bad
    for bad in (dict(A=P + 8), dict(d=P + 8), dict(dA=Q + 8), dict(dB=Q + 8), dict(db=Q + 2), dict(bias=P + 2)):
        assert linear_bwd(L, **bad) == MISALIGNED, bad
    need = L.qll_epilogue_backward_workspace_bytes(4, 0, 16, 64, 128)
    assert need >= 16 * 64 * 2
    assert linear_bwd(L, wsb=need - 1) == WORKSPACE and linear_bwd(L, ws=None) == WORKSPACE
    assert linear_bwd(L, ws=P + 4) == MISALIGNED
    assert L.qll_epilogue_backward_workspace_bytes(4, 1, 16, 64, 128) > need
    assert L.qll_epilogue_backward_workspace_bytes(0, 0, 16, 64, 128) == 0
    assert L.qll_epilogue_backward_workspace_bytes(0, 0, 16, 60, 128) == -INVALID


def test_gated_backward_refusals(L):
    assert gated_bwd(L, N=60) == INVALID
    assert gated_bwd(L, dG=None) == INVALID and gated_bwd(L, dU=None) == INVALID
    assert gated_bwd(L, dA=None, dG=None, dU=None) == INVALID
    assert gated_bwd(L, M=0, dG=None, dU=None) == 0
    for bad in (dict(A=None), dict(G=None), dict(U=None), dict(d=None)):
        assert gated_bwd(L, **bad) == INVALID, bad
    for bad in (dict(U=P + 8), dict(d=P + 8), dict(dA=Q + 8), dict(dG=Q + 8), dict(dU=Q + 2)):
        assert gated_bwd(L, **bad) == MISALIGNED, bad
    need = L.qll_gated_backward_workspace_bytes(16, 64, 128)
    assert need >= 16 * 128 * 2
    assert gated_bwd(L, wsb=need - 1) == WORKSPACE and gated_bwd(L, ws=None) == WORKSPACE
    assert gated_bwd(L, ws=P + 4) == MISALIGNED


def test_norm_refusals(L):
    assert norm(L, M=0) == 0
    for bad in (dict(M=-1), dict(K=0), dict(K=12), dict(rd=2), dict(eps=-1.0), dict(eps=float("nan")),
                dict(w2=None), dict(r=None), dict(no=None), dict(ro=None), dict(y=None),
                dict(y=None, ro=None, g=P), dict(y=None, ro=None, w1=P), dict(y=None, ro=None, al=0.5),
                dict(ns=P, K=24)):
        assert norm(L, **bad) == INVALID, bad
    assert norm(L, K=32776) == UNSUPPORTED
    for bad in (dict(y=P + 8), dict(r=P + 8), dict(w1=P + 2), dict(g=P + 2), dict(w2=P + 2), dict(ro=Q + 8),
                dict(no=Q + 8), dict(ns=Q + 2)):
        assert norm(L, **bad) == MISALIGNED, bad


def test_norm_backward_refusals(L):
    for bad in (dict(K=12), dict(w1=P), dict(g=P), dict(dw1=Q), dict(dg=Q), dict(dw2=None), dict(dn=None),
                dict(dr=None), dict(dy=None), dict(y=None)):
        assert norm_bwd(L, **bad) == INVALID, bad
    for bad in (dict(dn=P + 8), dict(do=P + 8), dict(dy=Q + 8), dict(dr=Q + 8), dict(dw2=Q + 2)):
        assert norm_bwd(L, **bad) == MISALIGNED, bad
    need = L.qll_residual_norm_backward_workspace_bytes(16, 128)
    assert need > 0
    assert norm_bwd(L, wsb=need - 1) == WORKSPACE and norm_bwd(L, ws=None) == WORKSPACE
    assert norm_bwd(L, ws=P + 4) == MISALIGNED
    assert L.qll_residual_norm_backward_workspace_bytes(16, 12) == -INVALID
    assert L.qll_residual_norm_backward_workspace_bytes(16, 32776) == -UNSUPPORTED
