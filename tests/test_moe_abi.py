"""CPU checks of the expert and sampling entry points: arguments are refused,
with the stated code, before any HIP call; workspaces are sized.  And the
64-bit references against independent forms of the same formulas."""
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


def route(L, x=P, dt=1, bias=None, score=0, groups=1, keep=1, best=2, k=4, renorm=1, scale=1.0, ids=Q, w=Q, off=None,
          rows=None, places=None, T=16, E=64, ws=None, wsb=0):
    return L.moe_route(x, dt, bias, score, groups, keep, best, k, renorm, scale, ids, w, off, rows, places, T, E, ws, wsb, None)


def route_bwd(L, x=P, dt=1, score=0, renorm=1, scale=1.0, ids=P, dw=P, dx=Q, T=16, E=64, k=4):
    return L.moe_route_backward(x, dt, score, renorm, scale, ids, dw, dx, T, E, k, None)


def sort(L, ids=P, off=Q, rows=Q, places=Q, T=16, E=64, k=4, ws=None, wsb=0):
    return L.moe_sort(ids, off, rows, places, T, E, k, ws, wsb, None)


def gated(L, A=P, G=P, U=P, sa=P, sg=P, su=P, off=P, rows=P, act=4, out=Q, od=0, T=16, R=64, N=64, K=128, E=8):
    return L.gated_fp8_grouped(A, G, U, sa, sg, su, off, rows, act, out, od, T, R, N, K, E, None)


def combine(L, y=P, places=P, w=P, res=None, out=Q, od=0, T=16, R=64, K=128, k=4):
    return L.moe_combine(y, places, w, res, out, od, T, R, K, k, None)


def combine_bwd(L, y=P, places=P, w=P, dout=P, od=0, dy=Q, dw=Q, T=16, R=64, K=128, k=4):
    return L.moe_combine_backward(y, places, w, dout, od, dy, dw, T, R, K, k, None)


def sample(L, x=P, dt=1, ld=1000, u=P, t=None, k=None, p=None, m=None, tok=Q, probs=None, B=4, V=1000, ws=None, wsb=0):
    return L.sample_tokens(x, dt, ld, u, t, k, p, m, tok, probs, B, V, ws, wsb, None)


@pytest.mark.parametrize("f", [route, route_bwd, sort])
def test_routing_refuses_sizes(L, f):
    for bad in (dict(T=-1), dict(E=0), dict(k=0), dict(k=-1), dict(T=1 << 40)):
        assert f(L, **bad) == INVALID, bad
    for bad in (dict(E=1025), dict(k=65, E=100), dict(T=1 << 25, k=4)):
        assert f(L, **bad) == UNSUPPORTED, bad


def test_route_refusals(L):
    for bad in (dict(dt=2), dict(dt=-1), dict(score=2), dict(score=-1), dict(best=0), dict(best=3), dict(groups=0),
                dict(groups=3), dict(groups=65), dict(groups=4, keep=0), dict(groups=4, keep=5), dict(k=65, E=64),
                dict(groups=32, keep=1, k=3), dict(x=None), dict(ids=None), dict(w=None), dict(off=Q),
                dict(off=Q, rows=Q), dict(rows=Q, places=Q)):
        assert route(L, **bad) == INVALID, bad
    assert route(L, groups=128, keep=128, E=128) == UNSUPPORTED
    for bad in (dict(x=P + 4), dict(bias=P + 2), dict(ids=Q + 2), dict(w=Q + 1), dict(off=Q + 2, rows=Q, places=Q),
                dict(off=Q, rows=Q + 1, places=Q), dict(off=Q, rows=Q, places=Q + 2)):
        assert route(L, **bad) == MISALIGNED, bad
    need = L.qll_moe_sort_workspace_bytes(5000, 64, 4)
    assert need > 0
    lists = dict(off=Q, rows=Q, places=Q, T=5000)
    assert route(L, **lists) == WORKSPACE and route(L, **lists, ws=P, wsb=need - 1) == WORKSPACE
    assert route(L, **lists, ws=P + 4, wsb=need) == MISALIGNED
    assert route(L, T=0) == 0 and route(L, T=0, x=None, ids=None, w=None) == 0


def test_route_backward_refusals(L):
    for bad in (dict(dt=2), dict(score=2), dict(x=None), dict(ids=None), dict(dw=None), dict(dx=None)):
        assert route_bwd(L, **bad) == INVALID, bad
    for bad in (dict(x=P + 8), dict(ids=P + 2), dict(dw=P + 2), dict(dx=Q + 4)):
        assert route_bwd(L, **bad) == MISALIGNED, bad
    assert route_bwd(L, T=0, x=None, ids=None, dw=None, dx=None) == 0


def test_sort_refusals(L):
    for bad in (dict(ids=None), dict(off=None), dict(rows=None), dict(places=None), dict(T=0, off=None)):
        assert sort(L, **bad) == INVALID, bad
    for bad in (dict(ids=P + 2), dict(off=Q + 2), dict(rows=Q + 1), dict(places=Q + 2)):
        assert sort(L, **bad) == MISALIGNED, bad
    assert sort(L, T=5000) == WORKSPACE
    need = L.qll_moe_sort_workspace_bytes
    assert need(128, 64, 8) == 0 and need(0, 64, 8) == 0
    assert need(1 << 20, 1024, 8) <= 512 * 1024 * 4
    assert need(16, 0, 4) == -INVALID and need(16, 2000, 4) == -UNSUPPORTED and need(-1, 8, 1) == -INVALID


def test_gated_refusals(L):
    for bad in (dict(T=-1), dict(R=-1), dict(N=0), dict(K=0), dict(K=24), dict(E=0), dict(E=65537), dict(act=-1), dict(act=6),
                dict(od=2), dict(rows=None), dict(G=None), dict(U=None), dict(sg=None), dict(su=None), dict(off=None),
                dict(out=None), dict(A=None), dict(sa=None), dict(N=1 << 30, K=1 << 12), dict(R=1 << 31)):
        assert gated(L, **bad) == INVALID, bad
    for bad in (dict(K=1 << 23), dict(T=1 << 20, K=2048), dict(R=1 << 29, N=2048, K=16)):
        assert gated(L, **bad) == UNSUPPORTED, bad
    for bad in (dict(A=P + 8), dict(G=P + 4), dict(U=P + 8), dict(out=Q + 8), dict(sa=P + 2), dict(sg=P + 2), dict(su=P + 1),
                dict(off=P + 2), dict(rows=P + 2)):
        assert gated(L, **bad) == MISALIGNED, bad
    assert gated(L, R=0, rows=P) == 0
    assert gated(L, R=0, T=0, rows=None, A=None, out=None, sa=None) == 0


def test_combine_refusals(L):
    for f in (combine, combine_bwd):
        for bad in (dict(T=-1), dict(R=-1), dict(K=0), dict(K=12), dict(k=0), dict(od=2), dict(places=None), dict(y=None),
                    dict(T=1 << 31)):
            assert f(L, **bad) == INVALID, bad
        for bad in (dict(k=65), dict(T=1 << 25, k=3)):
            assert f(L, **bad) == UNSUPPORTED, bad
        for bad in (dict(y=P + 8), dict(places=P + 2), dict(w=P + 2)):
            assert f(L, **bad) == MISALIGNED, bad
        assert f(L, T=0, y=None, places=None, w=None) == 0
    assert combine(L, out=None) == INVALID
    assert combine(L, out=Q + 8) == MISALIGNED and combine(L, res=P + 8) == MISALIGNED
    for bad in (dict(dout=None), dict(dy=None, dw=None), dict(w=None)):
        assert combine_bwd(L, **bad) == INVALID, bad
    for bad in (dict(dout=P + 8), dict(dy=Q + 8), dict(dw=Q + 2)):
        assert combine_bwd(L, **bad) == MISALIGNED, bad


def test_sample_refusals(L):
    for bad in (dict(B=-1), dict(V=0), dict(dt=2), dict(ld=999), dict(x=None), dict(u=None), dict(tok=None),
                dict(B=1 << 22)):
        assert sample(L, **bad) == INVALID, bad
    assert sample(L, V=(1 << 20) + 1, ld=1 << 21) == UNSUPPORTED
    for bad in (dict(x=P + 2), dict(dt=0, x=P + 1), dict(u=P + 2), dict(t=P + 1), dict(k=P + 2), dict(p=P + 2), dict(m=P + 2),
                dict(tok=Q + 2), dict(probs=Q + 2)):
        assert sample(L, **bad) == MISALIGNED, bad
    need = L.qll_sample_workspace_bytes(1, 151936)
    assert need > 0 and L.qll_sample_workspace_bytes(256, 151936) == 0 == L.qll_sample_workspace_bytes(0, 9)
    big = dict(B=1, V=151936, ld=151936)
    assert sample(L, **big) == WORKSPACE and sample(L, **big, ws=P, wsb=need - 1) == WORKSPACE
    assert sample(L, **big, ws=P + 8, wsb=need) == MISALIGNED
    assert sample(L, B=0, x=None, u=None, tok=None) == 0
    assert L.qll_sample_workspace_bytes(-1, 10) == -INVALID
    assert L.qll_sample_workspace_bytes(1, 1 << 21) == -UNSUPPORTED


# --------------------------------------------------------------------------
# the references
# --------------------------------------------------------------------------

torch = pytest.importorskip("torch")


@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_reference_gradients(score, renorm):
    """route_backward against autograd, in 64 bits."""
    import moe_reference as ref
    g = torch.Generator().manual_seed(1)
    x = torch.randn(6, 11, generator=g, dtype=torch.float64, requires_grad=True)
    ids = x.detach().topk(4, dim=1).indices
    dw = torch.randn(6, 4, generator=g, dtype=torch.float64)
    p = torch.softmax(x, 1) if score == "softmax" else torch.sigmoid(x)
    w = p.gather(1, ids)
    w = w / w.sum(1, keepdim=True) if renorm else w
    (w * dw).sum().mul(1.5).backward()
    dx, _ = ref.route_backward(x.detach(), ids, dw, score, renorm, 1.5)
    assert (dx - x.grad).abs().max() < 1e-14


def test_reference_route_and_sort():
    import moe_reference as ref
    g = torch.Generator().manual_seed(2)
    x = torch.randn(20, 24, generator=g)
    ids, w, _ = ref.route(x, 5)
    top = x.topk(5, dim=1)
    assert torch.equal(ids.long(), top.indices)
    assert (w - torch.softmax(top.values.double(), 1)).abs().max() < 1e-14
    offsets, rows, places = ref.sort(ids, 24)
    order = torch.argsort(ids.reshape(-1).long(), stable=True)
    assert torch.equal(rows.long(), order // 5)
    assert torch.equal(offsets[1:], torch.bincount(ids.reshape(-1), minlength=24).cumsum(0).int())
    assert torch.equal(places.reshape(-1)[order].long(), torch.arange(100))


def test_reference_sampling():
    """Shares of the tokens by integrating over u, against masked softmaxes."""
    import moe_reference as ref
    x = torch.tensor([0.3, -1.0, 2.0, 0.0, 1.1, -0.4, 0.9, 1.7], dtype=torch.float64)
    order = torch.sort(x, descending=True).indices
    for kw, keep in ((dict(), 8), (dict(top_k=3), 3), (dict(temperature=0.5), 8), (dict(min_p=0.35), 3)):  # e^-0.9 and above
        z = x / kw.get("temperature", 1.0)
        z = torch.where(torch.isin(torch.arange(8), order[:keep]), z, torch.full_like(z, -torch.inf))
        p = torch.softmax(z, 0)
        count = torch.zeros(8)
        for i in range(2000):
            token, share = ref.sample_row(x, (i + 0.5) / 2000, **kw)
            count[token] += 1
            assert abs(share - float(p[token])) < 1e-12
        assert ((count - 2000 * p).abs() <= 1).all()
    # the smallest front that reaches p: 2.0, 1.7, 1.1 have 0.34, 0.59, 0.73
    for top_p, keep in ((0.3, 1), (0.36, 2), (0.6, 3), (0.0, 1), (1.0, 8)):
        seen = {ref.sample_row(x, (i + 0.5) / 500, top_p=top_p)[0] for i in range(500)}
        assert seen == set(order[:keep].tolist())
