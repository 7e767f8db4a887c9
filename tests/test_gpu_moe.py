"""GPU parity of the expert operators against their definitions in 64 bits
(tests/moe_reference.py, which derives the bounds): routing with ties, groups
and rows that are not finite, the sort by expert, the gathered gated products,
the combination and the backward passes, guard values behind the outputs,
other streams, HIP graphs, and a whole mixture-of-experts layer."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import ffn_reference as ffn  # noqa: E402
import moe_reference as ref  # noqa: E402
from test_gpu_ffn import BF, D, F32, check, gen, guarded, qll, quant, rnd  # noqa: E402,F401

I32 = torch.int32
NAN, INF = float("nan"), float("inf")


def same(got, want, what):
    got, want = got.cpu(), want.cpu()
    assert got.shape == want.shape and got.dtype == want.dtype, what
    bad = (got != want).reshape(-1)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} differ, first at {int(bad.nonzero()[0])}"


# --------------------------------------------------------------------------
# routing
# --------------------------------------------------------------------------

# tokens, experts, choices: one token, odd batches, every width of a lane's
# share of the experts, one expert, all of them chosen, one workgroup and many
ROUTES = [(1, 64, 8), (1, 1, 1), (3, 7, 7), (17, 9, 2), (64, 64, 8), (128, 128, 8), (129, 65, 8), (131, 256, 8),
          (40, 200, 6), (33, 500, 10), (70, 512, 16), (5, 1024, 64), (21, 1000, 3), (700, 64, 8), (1025, 16, 4)]


@pytest.mark.parametrize("T,E,k", ROUTES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_route(qll, dtype, score, T, E, k):
    g = gen(T + 31 * E + k)
    x = rnd(g, T, E, std=2.0, dtype=BF if dtype == "bf16" else F32)
    bias = rnd(g, E, std=0.1, dtype=F32)
    groups = next(n for n in (8, 5, 4, 3, 2, 1) if E % n == 0)
    least = -(-k * groups // E)
    for kw in (dict(), dict(renormalize=False, scale=2.5), dict(bias=bias), dict(bias=bias, renormalize=False),
               dict(groups=groups, topk_groups=least), dict(groups=groups, topk_groups=least, bias=bias),
               dict(groups=groups, topk_groups=min(groups, least + 1), group_best=1, bias=bias, scale=0.5)):
        ids, w, offsets, rows, places = qll.moe_route(x, k, score=score, plan=True, **kw)
        rid, rw, bound = ref.route(x, k, score=score, **kw)
        same(ids, rid, (kw, "ids"))
        assert ((w.cpu().to(D) - rw).abs() <= bound + 1e-37).all(), (kw, "weights")
        for got, want, name in zip((offsets, rows, places), ref.sort(rid, E), ("offsets", "rows", "places")):
            same(got, want, (kw, name))
        ids2, w2 = qll.moe_route(x, k, score=score, **kw)
        assert torch.equal(ids, ids2) and torch.equal(w, w2)


def test_route_ties_and_order(qll):
    """Equal logits go to the lower expert, -0 and 0 are equal, and equal
    scores with a bias too."""
    x = torch.zeros(6, 96, device="cuda")
    x[1, 1::2] = -0.0
    x[2, 50] = x[2, 70] = 1.0
    x[3] = torch.arange(96, device="cuda") % 3
    x[4] = 100.0  # (sigmoid and its sum with the bias: all equal)
    bias = torch.zeros(96, device="cuda")
    bias[7] = bias[90] = 0.25
    for score in ("softmax", "sigmoid"):
        for kw in (dict(), dict(bias=bias), dict(bias=bias, groups=12, topk_groups=2), dict(groups=12, topk_groups=3)):
            ids, _ = qll.moe_route(x, 10, score=score, **kw)
            same(ids, ref.route(x, 10, score=score, **kw)[0], (score, kw))


def test_route_close_values(qll):
    """Values that a 32-bit score cannot tell apart: sums with a bias one part
    in 2^30 from each other."""
    E = 64
    x = torch.full((2, E), 3.0, device="cuda")
    bias = torch.full((E,), 1e-3, device="cuda")
    bits = bias.view(I32)
    bits[40] += 1  # the next fp32 value: 1e-10 more, on scores of 0.95
    bits[13] -= 1
    ids, _ = qll.moe_route(x, 3, score="sigmoid", bias=bias)
    same(ids, torch.tensor([[40, 0, 1]] * 2, dtype=I32), "ids")
    ids, _ = qll.moe_route(x, E, score="sigmoid", bias=bias)
    assert ids[0, -1] == 13


def test_route_rows_that_are_not_finite(qll):
    """Masked experts come last, a NaN like them; ids stay in range and
    distinct; a row without a softmax has NaN weights, an empty one zeros."""
    g = gen(5)
    T, E, k = 6, 40, 6
    x = rnd(g, T, E, dtype=F32)
    clean = x.clone()
    x[0, 3:] = -INF
    x[1] = -INF
    x[2, 11] = NAN
    x[3, 12] = INF
    x[4] = NAN
    bias = rnd(g, E, std=0.1, dtype=F32)
    for score in ("softmax", "sigmoid"):
        for kw in (dict(), dict(renormalize=False), dict(bias=bias), dict(groups=8, topk_groups=3)):
            ids, w = qll.moe_route(x, k, score=score, **kw)
            for row in ids.tolist():
                assert len(set(row)) == k and all(0 <= e < E for e in row)
            if score == "softmax":
                assert torch.isnan(w[2:5]).all()
                assert (w[1] == 0).all()
            if not kw:
                same(ids, ref.route(x, k, score=score)[0], score)
                assert set(ids[0, :3].tolist()) == {0, 1, 2} and (w[0, 3:] == 0).all()
            i2, w2 = qll.moe_route(clean, k, score=score, **kw)
            assert torch.equal(ids[5], i2[5]) and torch.equal(w[5], w2[5])


@pytest.mark.parametrize("T,E,k", [(1, 64, 8), (5, 7, 7), (33, 130, 6), (50, 300, 10), (9, 1000, 64), (300, 64, 8)])
@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_backward(qll, score, renorm, T, E, k):
    g = gen(T + E)
    for dtype in (F32, BF):
        x = rnd(g, T, E, std=2.0, dtype=dtype)
        ids = x.float().topk(k, dim=1).indices.int()
        dw = rnd(g, T, k, dtype=F32)
        dx = qll.moe_route_backward(x, ids, dw, score=score, renormalize=renorm, scale=1.5)
        check(dx, ref.route_backward(x, ids, dw, score, renorm, 1.5), (dtype, "dlogits"))
        if k > 2:  # an expert named twice, and one that is none
            ids[:, 1] = ids[:, 0]
            ids[:, 2] = torch.where(torch.arange(T, device="cuda") % 2 == 0, -1, E).int()
            dx = qll.moe_route_backward(x, ids, dw, score=score, renormalize=renorm)
            check(dx, ref.route_backward(x, ids, dw, score, renorm), (dtype, "repeated"))


# --------------------------------------------------------------------------
# the sort
# --------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 64, 8), (128, 64, 8), (129, 64, 8), (1000, 3, 1), (2000, 300, 6),
                                   (4097, 1024, 2), (40, 5, 64), (17000, 64, 2)])
@pytest.mark.parametrize("kind", ["even", "one", "others"])
def test_sort(qll, kind, T, E, k):
    g = gen(T + E + k)
    if kind == "one":  # every choice the same expert
        ids = torch.full((T, k), E - 1, dtype=I32, device="cuda")
    else:  # repeated experts, and with `others` ids that are none
        lo, hi = (0, E) if kind == "even" else (-2, E + 2)
        ids = torch.randint(lo, hi, (T, k), generator=g, device="cuda", dtype=I32)
    whole = torch.full((T * k + 8,), 77, dtype=I32, device="cuda")
    got = qll.moe_sort(ids, E, rows=whole[:T * k])
    for a, b, name in zip(got, ref.sort(ids.cpu(), E), ("offsets", "rows", "places")):
        same(a, b, name)
    assert (whole[T * k:] == 77).all()


def test_no_tokens(qll):
    x = torch.empty(0, 16, device="cuda")
    ids, w, offsets, rows, places = qll.moe_route(x, 4, plan=True, offsets=torch.full((17,), 5, dtype=I32, device="cuda"))
    assert ids.shape == (0, 4) and w.shape == (0, 4) and rows.shape == (0,) and places.shape == (0, 4)
    assert (offsets == 0).all()
    offsets, rows, places = qll.moe_sort(ids, 16)
    assert (offsets == 0).all() and rows.numel() == 0
    assert qll.moe_route_backward(x, ids, w).shape == (0, 16)
    y = torch.empty(0, 32, dtype=BF, device="cuda")
    assert qll.moe_combine(y, places, w).shape == (0, 32)
    dy, dw = qll.moe_combine_backward(y, places, w, torch.empty(0, 32, dtype=BF, device="cuda"))
    assert dy.shape == (0, 32) and dw.shape == (0, 4)


# --------------------------------------------------------------------------
# the experts' products
# --------------------------------------------------------------------------

def experts(g, E, N, K):
    wg, wu = rnd(g, E, N, K, std=0.05), rnd(g, E, N, K, std=0.05)
    qg, sg = quant(wg.view(E * N, K))
    qu, su = quant(wu.view(E * N, K))
    return qg.view(E, N, K), qu.view(E, N, K), sg.view(E, N), su.view(E, N)


def gated_rows(x, sx, wg, wu, sg, su, bounds, rows, act, out):
    """(reference, bound) expert by expert; rows of no expert are NaN."""
    R, N = len(rows), wg.shape[1]
    y = torch.full((R, N), NAN, dtype=D, device="cuda")
    e = torch.zeros(R, N, dtype=D, device="cuda")
    for i, (a, b) in enumerate(zip(bounds, bounds[1:])):
        if b > a:
            t = rows[a:b].long()
            y[a:b], e[a:b] = ffn.gated(x[t].to(D), wg[i].to(D), wu[i].to(D), sx[t].to(D), sg[i].to(D), su[i].to(D), act, out)
    return y, e


# counts of rows per expert: one row, none, ragged tiles, one expert for all;
# the mean decides the kernel (few rows, 64- and 128-row tiles)
LOADS = [[1], [0, 0, 1], [1] * 8 + [0] * 56, [15, 16, 17, 0, 1], [3, 40, 0, 2, 1], [0, 65, 1, 64, 0, 63, 9, 14],
         [17, 100, 3, 33], [130, 0, 127, 129, 1], [300, 5, 260, 400], [700]]


@pytest.mark.parametrize("counts", LOADS, ids=lambda c: "-".join(map(str, c[:5])))
@pytest.mark.parametrize("N,K", [(64, 128), (1, 16), (9, 48), (129, 272), (200, 1040), (520, 2064)])
def test_gated_grouped(qll, counts, N, K):
    g = gen(sum(counts) + N + K)
    E, R = len(counts), sum(counts)
    T = max(1, R // 3)
    x, sx = quant(rnd(g, T, K))
    w = experts(g, E, N, K)
    offsets = torch.tensor([0] + counts, dtype=I32, device="cuda").cumsum(0).int()
    rows = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=I32)
    bounds = offsets.tolist()
    act = ("silu", "gelu", "gelu_tanh")[R % 3]
    for out in ("bf16", "fp32"):
        whole, o = guarded(R, N, BF if out == "bf16" else F32)
        qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], offsets, rows=rows, act=act, out_dtype=out, out=o)
        check(o, gated_rows(x, sx, w[0], w[1], w[2], w[3], bounds, rows, act, out), (counts, out), whole)
    # the same tokens, sorted by hand
    o2 = qll.gated_fp8_grouped(x[rows.long()], *w[:2], sx[rows.long()], *w[2:], offsets, act=act, out_dtype="fp32")
    assert torch.equal(o, o2)


@pytest.mark.parametrize("per", [2, 40, 150])
def test_gated_grouped_rows_of_nobody(qll, per):
    """Rows behind the last expert's are left as they were; a token that is
    none reads as zeros; offsets out of range and falling reach no other row."""
    E, N, K, T = 5, 72, 160, 64
    g = gen(per)
    x, sx = quant(rnd(g, T, K))
    w = experts(g, E, N, K)
    R = E * per + 7
    rows = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=I32)
    offsets = (torch.arange(E + 1, device="cuda") * per).int()
    bad = rows.clone()
    bad[1::3] = torch.tensor([-1, T, 1 << 30], dtype=I32, device="cuda").repeat(R)[:len(bad[1::3])]
    o = torch.full((R, N), 7.0, dtype=F32, device="cuda")
    qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], offsets, rows=bad, out_dtype="fp32", out=o)
    assert (o[E * per:] == 7.0).all()
    assert (o[1:E * per:3] == 0).all()
    good = torch.ones(E * per, dtype=torch.bool)
    good[1::3] = False
    y, e = gated_rows(x, sx, *w, offsets.tolist(), rows, "silu", "fp32")
    assert ((o[:E * per].to(D) - y[:E * per]).abs()[good] <= e[:E * per][good] + 1e-30).all()
    # [3, -4, 2 per, per, R + 9, 5]: read as running maxima in [0, R]
    odd = torch.tensor([3, -4, 2 * per, per, R + 9, 5], dtype=I32, device="cuda")
    seen = torch.tensor([3, 3, 2 * per, 2 * per, R, R] if 2 * per > 3 else [3, 3, 4, 4, R, R])
    o = torch.full((R, N), 7.0, dtype=F32, device="cuda")
    qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], odd, rows=rows, out_dtype="fp32", out=o)
    assert (o[:3] == 7.0).all()
    y, e = gated_rows(x, sx, *w, seen.tolist(), rows, "silu", "fp32")
    check(o[3:], (y[3:], e[3:]), "clamped")


def test_gated_grouped_bad_token_stays_its_own(qll):
    """A NaN scale reaches its token's rows and no others."""
    E, N, K, T = 4, 40, 64, 9
    g = gen(77)
    x, sx = quant(rnd(g, T, K))
    w = experts(g, E, N, K)
    ids = torch.randint(0, E, (T, 2), generator=g, device="cuda", dtype=I32)
    offsets, rows, _ = qll.moe_sort(ids, E)
    clean = qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], offsets, rows=rows)
    sx[4] = NAN
    o = qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], offsets, rows=rows)
    hit = rows == 4
    assert torch.isnan(o[hit]).all() and torch.equal(o[~hit], clean[~hit])


# --------------------------------------------------------------------------
# combination
# --------------------------------------------------------------------------

@pytest.mark.parametrize("T,k,K", [(1, 8, 2048), (1, 1, 8), (7, 3, 40), (65, 8, 264), (33, 64, 128), (300, 6, 4104)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_combine(qll, dtype, T, k, K):
    g = gen(T + k + K)
    R = T * k + 3
    y, w = rnd(g, R, K), rnd(g, T, k, dtype=F32)
    places = torch.randperm(R, generator=g, device="cuda")[:T * k].view(T, k).int()
    res, dout = rnd(g, T, K, dtype=dtype), rnd(g, T, K, dtype=dtype)
    name = "bf16" if dtype == BF else "fp32"
    for at in (places, torch.where(torch.rand(T, k, generator=g, device="cuda") < 0.3, R, places).int()):
        at = at.clone()
        at[0, 0] = -1
        for kw in (dict(weights=w, residual=res), dict(weights=w), dict(residual=res), dict()):
            whole, o = guarded(T, K, dtype)
            qll.moe_combine(y, at, out_dtype=name, out=o, **kw)
            check(o, ref.combine(y, at, dtype=dtype, **kw), (sorted(kw), "out"), whole)
        own = res.clone()  # in place
        qll.moe_combine(y, at, w, residual=own, out=own, out_dtype=name)
        assert torch.equal(own, qll.moe_combine(y, at, w, residual=res))
        dy = torch.full((R, K), 7.0, dtype=BF, device="cuda")
        _, dw = qll.moe_combine_backward(y, at, w, dout, dy=dy)
        rdy, edy, rdw, edw = ref.combine_backward(y, at, w, dout)
        named = torch.zeros(R, dtype=torch.bool, device="cuda")
        named[at[(at >= 0) & (at < R)].long()] = True
        check(dy[named], (rdy[named], edy[named]), "dy")
        assert (dy[~named] == 7.0).all()
        check(dw, (rdw, edw), "dweights")
        only, none = qll.moe_combine_backward(y, at, None, dout, dy=torch.full_like(dy, 7.0))
        assert none is None
        check(only[named], (ref.combine_backward(y, at, None, dout)[0][named], edy[named].new_zeros(()) + 2.0 ** -8 * dout.abs().max()), "ones")
        none, dw2 = qll.moe_combine_backward(y, at, w, dout, need_y=False)
        assert none is None and torch.equal(dw, dw2)


def test_combine_keeps_bad_rows_out(qll):
    """A row that no place names may hold anything."""
    y = torch.full((6, 16), NAN, dtype=BF, device="cuda")
    y[2], y[4] = 1.0, 2.0
    places = torch.tensor([[2, -1], [4, 6]], dtype=I32, device="cuda")
    w = torch.tensor([[0.5, NAN], [0.25, INF]], device="cuda")
    o = qll.moe_combine(y, places, w)
    assert (o[0] == 0.5).all() and (o[1] == 0.5).all()


# --------------------------------------------------------------------------
# gradients against differences
# --------------------------------------------------------------------------

@pytest.mark.parametrize("renorm", [True, False])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_gradients_against_differences(qll, score, renorm):
    """d/dx of sum(out * c) for out = moe_combine(y, places, moe_route(x)):
    the backward passes against central differences of the 64-bit formulas."""
    g = gen(3)
    T, E, k, K = 5, 12, 4, 24
    x = rnd(g, T, E, dtype=F32)
    y, c = rnd(g, T * k, K), rnd(g, T, K, dtype=F32)
    ids, w, _, _, places = qll.moe_route(x, k, score=score, renormalize=renorm, plan=True)
    _, dw = qll.moe_combine_backward(y, places, w, c, need_y=False)
    dx = qll.moe_route_backward(x, ids, dw, score=score, renormalize=renorm).cpu().to(D)
    ys, cs, at = y.cpu().to(D)[places.cpu().long()], c.cpu().to(D), ids.cpu().long()

    def loss(x):
        p = ref.scores(x, score).gather(1, at)
        p = p / p.sum(1, keepdim=True) if renorm else p
        return ((p[:, :, None] * ys).sum(1) * cs).sum()

    x64, h = x.cpu().to(D), 1e-5
    for t in range(T):
        for e in range(E):
            d = torch.zeros_like(x64)
            d[t, e] = h
            want = float((loss(x64 + d) - loss(x64 - d)) / (2 * h))
            # differences: h^2 of a third derivative (at most sum |y c| here, some 40); the kernels: 2^-18 of dw
            assert abs(float(dx[t, e]) - want) <= 1e-8 + 2.0 ** -18 * float(dw[t].abs().max())


# --------------------------------------------------------------------------
# a layer, streams, graphs
# --------------------------------------------------------------------------

def layer(qll, x, logits, res, w, down, k, score="softmax", plan=None, outs=None):
    q, sx = qll.quantize_per_token_fp8(x)
    ids, weights, offsets, rows, places = qll.moe_route(logits, k, score=score, plan=True)
    a = qll.gated_fp8_grouped(q, *w[:2], sx, *w[2:], offsets, rows=rows)
    qa, sa = qll.quantize_per_token_fp8(a)
    y = qll.gemm_fp8_grouped(qa, down[0], sa, down[1], offsets)
    return qll.moe_combine(y, places, weights, residual=res), ids, weights, (q, sx, a, y)


def make_layer(qll, g, T, E, N, K):
    w = experts(g, E, N, K)
    qd, sd = quant(rnd(g, E * K, N, std=0.05))
    return rnd(g, T, K), rnd(g, T, E, std=2.0, dtype=F32), rnd(g, T, K), w, (qd.view(E, K, N), sd.view(E, K))


@pytest.mark.parametrize("T", [1, 19, 300])
def test_layer(qll, T):
    """The whole layer against the dense formula: every token's experts one by
    one in 64 bits, from the codes the products take."""
    E, N, K, k = 16, 208, 144, 4
    x, logits, res, w, down = make_layer(qll, gen(T), T, E, N, K)
    out, ids, weights, (q, sx, a, y) = layer(qll, x, logits, res, w, down, k)
    q64, d64 = q.to(D) * sx.to(D).view(-1, 1), down[0].to(D) * down[1].to(D)[:, :, None]
    wg, wu = w[0].to(D) * w[2].to(D)[:, :, None], w[1].to(D) * w[3].to(D)[:, :, None]
    want = res.to(D).clone()
    mag = want.abs()
    for t in range(T):
        for j in range(k):
            e = int(ids[t, j])
            zg, zu = wg[e] @ q64[t], wu[e] @ q64[t]
            h = zg * torch.sigmoid(zg) * zu
            # the quantizer's step is at most 2^-4 of a value or 2^-9 of the
            # row's largest over 448, the products and roundings well below
            want[t] += float(weights[t, j]) * (d64[e] @ h)
            mag[t] += float(weights[t, j]) * (d64[e].abs() @ (h.abs() + h.abs().max() / 64))
    assert ((out.to(D) - want).abs() <= (2.0 ** -4 + 2.0 ** -6) * mag).all()


def test_layer_on_another_stream_and_in_a_graph(qll):
    T, E, N, K, k = 150, 8, 144, 160, 3  # (more than one workgroup sorts)
    x, logits, res, w, down = make_layer(qll, gen(8), T * 4, E, N, K)
    want, wid, ww, _ = layer(qll, x, logits, res, w, down, k)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = layer(qll, x, logits, res, w, down, k)[0]
    s.synchronize()
    assert torch.equal(got, want)
    ids, weights, offsets, rows, places = qll.moe_route(logits, k, plan=True, stream=s)
    s.synchronize()
    assert torch.equal(ids, wid) and torch.equal(weights, ww)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        layer(qll, x, logits, res, w, down, k)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        out, gid, gw, inner = layer(qll, x, logits, res, w, down, k)
        dlogits = qll.moe_route_backward(logits, gid, gw)
    for rep in range(3):
        out.fill_(7.0)
        for t in inner[2:]:
            t.fill_(3.0)
        gid.fill_(-5)
        dlogits.fill_(9.0)
        if rep == 1:  # other inputs in the same tensors
            logits.copy_(logits.flip(0))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        eager, eid, ew, _ = layer(qll, x, logits, res, w, down, k)
        assert torch.equal(out, eager) and torch.equal(gid, eid) and torch.equal(gw, ew), rep
        assert torch.equal(dlogits, qll.moe_route_backward(logits, eid, ew)), rep


def test_results_repeat(qll):
    """Bit for bit the same, call after call."""
    x, logits, res, w, down = make_layer(qll, gen(11), 900, 32, 80, 96)
    first = layer(qll, x, logits, res, w, down, 8)
    for _ in range(3):
        again = layer(qll, x, logits, res, w, down, 8)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1]) and torch.equal(first[2], again[2])


def test_binding_refusals(qll):
    x = torch.randn(4, 16, device="cuda")
    ids, w, offsets, rows, places = qll.moe_route(x, 2, plan=True)
    y = torch.zeros(8, 16, dtype=BF, device="cuda")
    for call in (lambda: qll.moe_route(x.half(), 2), lambda: qll.moe_route(x, 0), lambda: qll.moe_route(x, 2, score="max"),
                 lambda: qll.moe_route(x.t(), 2), lambda: qll.moe_route(x, 2, offsets=offsets),
                 lambda: qll.moe_route(x, 2, bias=x[0].double()), lambda: qll.moe_route(x.cpu(), 2),
                 lambda: qll.moe_route_backward(x, ids.long(), w), lambda: qll.moe_route_backward(x, ids, w[:3]),
                 lambda: qll.moe_sort(ids.long(), 16), lambda: qll.moe_sort(ids, 0), lambda: qll.moe_sort(ids[0], 16),
                 lambda: qll.moe_combine(y.float(), places, w), lambda: qll.moe_combine(y, places, w[:3]),
                 lambda: qll.moe_combine(y, places, w, residual=torch.zeros(4, 16, dtype=BF, device="cuda"), out_dtype="fp32"),
                 lambda: qll.moe_combine_backward(y, places, None, y[:4], need_y=False),
                 lambda: qll.moe_combine_backward(y, places, w, y)):
        with pytest.raises((ValueError, TypeError)):
            call()
    for call in (lambda: qll.moe_route(x, 17), lambda: qll.moe_route(x, 2, groups=3),
                 lambda: qll.moe_route(x, 9, groups=4, topk_groups=2), lambda: qll.moe_route(x, 2, group_best=3),
                 lambda: qll.moe_combine(y[:, :12].contiguous(), places, w)):
        with pytest.raises(qll.QllError):
            call()
    q, s = quant(y + 1)
    wq = q.view(2, 4, 16)
    sw = s.view(2, 4)
    off = torch.tensor([0, 3, 8], dtype=I32, device="cuda")
    qll.gated_fp8_grouped(q, wq, wq, s, sw, sw, off)
    for call in (lambda: qll.gated_fp8_grouped(q, q, q, s, sw, sw, off), lambda: qll.gated_fp8_grouped(q, wq, wq, s, s, s, off),
                 lambda: qll.gated_fp8_grouped(q, wq, wq, s, sw, sw, off[:2]),
                 lambda: qll.gated_fp8_grouped(q, wq, wq[:1], s, sw, sw, off),
                 lambda: qll.gated_fp8_grouped(q, wq, wq, s, sw, sw, off, rows=ids),
                 lambda: qll.gated_fp8_grouped(q, wq, wq, s, sw, sw, off, act="swish")):
        with pytest.raises((ValueError, TypeError)):
            call()
