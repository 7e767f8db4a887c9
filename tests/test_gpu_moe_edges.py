"""GPU tests of the expert operators and the sampler where few calls go: many
tokens, scores that 32 bits cannot tell apart, every kernel of the gated
products, sizes past 32-bit offsets, and calls on two streams at once."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import moe_reference as ref  # noqa: E402
from test_gpu_ffn import BF, D, F32, check, gen, guarded, qll, quant, rnd  # noqa: E402,F401
from test_gpu_moe import I32, INF, experts, gated_rows, same  # noqa: E402
from test_gpu_sample import expand, run  # noqa: E402


# --------------------------------------------------------------------------
# many tokens: chunks of 16, 32 and more of them
# --------------------------------------------------------------------------

@pytest.mark.parametrize("T,E,k", [(4097, 64, 8), (9001, 100, 6), (20000, 64, 2), (70001, 16, 4)])
def test_many_tokens(qll, T, E, k):
    g = gen(T)
    x = rnd(g, T, E, dtype=F32)
    ids, w, offsets, rows, places = qll.moe_route(x, k, plan=True)
    order = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :k]
    same(ids, order.int(), "ids")
    p = torch.softmax(x.to(D).gather(1, order), 1)
    # (2 D + 40) u of a weight, D < 12 for normal logits
    assert ((w.to(D) - p).abs() <= 64 * 2.0 ** -24 * p).all()
    for lists in ((offsets, rows, places), qll.moe_sort(ids, E)):
        flat = ids.reshape(-1).long()
        by = torch.argsort(flat, stable=True)
        same(lists[1], (by // k).int(), "rows")
        same(lists[2].reshape(-1)[by], torch.arange(T * k, dtype=I32, device="cuda"), "places")
        same(lists[0][1:], torch.bincount(flat, minlength=E).cumsum(0).int(), "offsets")
        assert lists[0][0] == 0


# --------------------------------------------------------------------------
# close calls
# --------------------------------------------------------------------------

@pytest.mark.parametrize("E,groups,keep", [(64, 1, 1), (64, 8, 3), (96, 4, 2), (256, 8, 4), (250, 5, 2), (512, 16, 5), (1000, 8, 3)])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_close_scores(qll, score, E, groups, keep):
    """Logits a few last bits apart and biases of few values: whole rows of
    sums that agree to 1e-7 and less, exact ties among them."""
    T, k = 40, 7
    g = gen(E + groups)
    steps = torch.randint(0, 6, (T, E), generator=g, device="cuda")
    x = 1.0 + steps * 2.0 ** -23
    x[::4] = 1.0 + steps[::4] * 2.0 ** -16  # (further apart: some in 32 bits)
    x[1::4] += rnd(g, len(x[1::4]), E, dtype=F32) * 1e-6
    bias = torch.randint(0, 3, (E,), generator=g, device="cuda") * 1e-8
    for b in (bias, bias * 0, bias * 1e6, None):
        for best in (1, 2):
            kw = dict(score=score, bias=None if b is None else b.float(), groups=groups, topk_groups=keep, group_best=best)
            ids, _ = qll.moe_route(x, k, **kw)
            same(ids, ref.route(x, k, **kw)[0], (best, b is None))


@pytest.mark.parametrize("k", [1, 8, 61, 62, 63, 64])
def test_close_scores_of_many_choices(qll, k):
    g = gen(k)
    x = 0.5 + torch.randint(0, 4, (20, 70), generator=g, device="cuda") * 2.0 ** -24
    bias = torch.full((70,), 0.125, device="cuda")
    for score in ("sigmoid", "softmax"):
        ids, w = qll.moe_route(x, k, score=score, bias=bias)
        rid, rw, bound = ref.route(x, k, score=score, bias=bias)
        same(ids, rid, score)
        assert ((w.cpu().to(D) - rw).abs() <= bound).all()


def test_masked_experts_with_a_bias(qll):
    """-infinity logits among the picks, with a bias that would prefer them."""
    g = gen(4)
    x = rnd(g, 30, 128, dtype=F32)
    x[:, 5:] = torch.where(torch.rand(30, 123, generator=g, device="cuda") < 0.98, -float("inf"), x[:, 5:])
    bias = rnd(g, 128, std=0.3, dtype=F32)
    for score in ("sigmoid", "softmax"):
        for kw in (dict(), dict(groups=8, topk_groups=2), dict(groups=16, topk_groups=3, renormalize=False)):
            ids, w = qll.moe_route(x, 9, score=score, bias=bias, **kw)
            rid, rw, bound = ref.route(x, 9, score=score, bias=bias, **kw)
            same(ids, rid, (score, kw))
            assert ((w.cpu().to(D) - rw).abs() <= bound + 1e-37).all()


# experts of a token and groups: groups of a lane, of several lanes, of none's
# multiple, of more experts than a lane holds
BIASED = [(32, 32, 8, 5), (64, 8, 3, 6), (96, 4, 2, 9), (250, 5, 2, 7), (256, 8, 4, 8), (1000, 8, 3, 8)]


@pytest.mark.parametrize("E,groups,keep,k", BIASED)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_infinite_biases(qll, score, E, groups, keep, k):
    """Experts that are always and never chosen, together in a group: +infinity
    and -infinity add up to no number, which counts as -infinity."""
    T, size = 50, E // groups
    g = gen(E)
    x = rnd(g, T, E, dtype=F32)
    bias = rnd(g, E, std=0.1, dtype=F32)
    rand = torch.rand(E, generator=g, device="cuda")
    bias[rand < 0.2] = -INF
    mixed = bias.clone()
    for at in (0, groups // 2, groups - 1):  # one of +infinity, the rest out
        mixed[at * size:(at + 1) * size] = -INF
        mixed[at * size + size // 2] = INF
    mixed[size:2 * size] = INF
    out = torch.full_like(bias, -INF)  # one group left
    out[-size:] = bias[-size:]
    for b in (bias, mixed, out, -mixed):
        for best in (1, 2):
            kw = dict(score=score, bias=b, groups=groups, topk_groups=keep, group_best=best)
            ids, w = qll.moe_route(x, k, **kw)
            rid, rw, bound = ref.route(x, k, **kw)
            same(ids, rid, (score, best))
            assert ((w.cpu().to(D) - rw).abs() <= bound + 1e-37).all()


@pytest.mark.parametrize("E,groups,keep,k", BIASED)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_close_groups_beside_experts_out_of_service(qll, score, E, groups, keep, k):
    """Groups whose values 32 bits cannot tell apart, with biases of -infinity,
    of the lowest value and of large sizes among them."""
    T = 40
    g = gen(E + k)
    steps = torch.randint(0, 6, (T, E), generator=g, device="cuda")
    x = 1.0 + steps * 2.0 ** -23
    x[::4] = 1.0 + steps[::4] * 2.0 ** -16
    bias = torch.randint(0, 3, (E,), generator=g, device="cuda") * 1e-8
    gone = torch.rand(E, generator=g, device="cuda") < 0.3
    for level in (-INF, torch.finfo(F32).min, -1e9, INF):
        for best in (1, 2):
            kw = dict(score=score, bias=torch.where(gone, level, bias).float(), groups=groups, topk_groups=keep, group_best=best)
            ids, _ = qll.moe_route(x, k, **kw)
            same(ids, ref.route(x, k, **kw)[0], (level, best))


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_groups_masked_in_two_ways(qll, score, dtype):
    """A group of -infinity and one of the type's lowest value both have scores
    of 0 in 64 bits: the first of them is open."""
    x = rnd(gen(8), 12, 32, dtype=dtype)
    x[:, :8] = -INF
    x[:, 16:24] = torch.finfo(dtype).min
    for best in (1, 2):
        for flip in (x, x.flip(1)):
            flip = flip.contiguous()
            kw = dict(score=score, groups=4, topk_groups=3, group_best=best)
            same(qll.moe_route(flip, 20, **kw)[0], ref.route(flip, 20, **kw)[0], (score, best))


def test_far_chosen_experts(qll):
    """Renormalised weights of experts far below the largest logit, which lies
    in a group that is not open."""
    x = torch.full((3, 32), -300.0, device="cuda")
    x[:, 8:16] = torch.tensor([0.0, 1.0, 2.0, -1.0, 0.5, 0.0, 0.0, 0.0], device="cuda") - 120
    x[:, 20] = 0.0
    bias = torch.zeros(32, device="cuda")
    bias[8:16] = 1.0
    ids, w = qll.moe_route(x, 3, bias=bias, groups=4, topk_groups=1)
    rid, rw, bound = ref.route(x, 3, bias=bias, groups=4, topk_groups=1)
    same(ids, rid, "ids")
    want = torch.softmax(x.cpu().to(D).gather(1, rid.long()), 1)
    assert ((w.cpu().to(D) - want).abs() <= 64 * 2.0 ** -24).all()


# --------------------------------------------------------------------------
# every kernel of the gated products, more than 64 experts
# --------------------------------------------------------------------------

def spread(E, R, g):
    """R rows over E experts, uneven, some without any."""
    p = torch.rand(E, generator=g, device="cuda") ** 3
    p[::7] = 0
    p[0] = 0.1
    return torch.bincount(torch.multinomial(p, R, True, generator=g), minlength=E).tolist()


# tiles of 64x32, 64x64, 128x128 and 256x128 outputs
KERNELS = [(130, 300, 40, 144), (70, 40, 264, 272), (24, 100, 520, 160), (8, 80, 4104, 144), (130, 900, 1032, 80),
           (6, 700, 2056, 400), (70, 4000, 520, 272), (4, 2100, 4104, 144), (70, 14100, 264, 80), (3, 1500, 6001, 336)]


@pytest.mark.parametrize("E,R,N,K", KERNELS)
def test_gated_kernels(qll, E, R, N, K):
    g = gen(E + R + N + K)
    counts = spread(E, R, g)
    T = R // 2 + 1
    x, sx = quant(rnd(g, T, K))
    w = experts(g, E, N, K)
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    rows = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=I32)
    for out in ("bf16", "fp32"):
        whole, o = guarded(R, N, BF if out == "bf16" else F32)
        qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], offsets, rows=rows, out_dtype=out, out=o)
        check(o, gated_rows(x, sx, *w, offsets.tolist(), rows, "silu", out), (E, R, N, K, out), whole)
    o2 = qll.gated_fp8_grouped(x[rows.long()], *w[:2], sx[rows.long()], *w[2:], offsets, out_dtype="fp32")
    assert torch.equal(o, o2)


# more than 64 experts in the kernel for few rows and tiles (one row an expert or
# none, more rows than a block of 16); more than 1024, which the 256x128 tile's
# list of experts does not hold, in that one and in tiles of 64x64 and 128x128
MANY = [(70, 40, 40, 144), (130, 70, 9, 272), (65, 60, 64, 48), (1100, 90, 24, 160), (2000, 40, 40, 80),
        (1100, 900, 72, 80), (1100, 60000, 264, 48), (1100, 220000, 40, 16)]


@pytest.mark.parametrize("E,R,N,K", MANY)
def test_gated_kernels_of_many_experts(qll, E, R, N, K):
    g = gen(E + R + N + K)
    counts = spread(E, R, g)
    if R < 100:  # (an expert with several tiles of rows, behind the first 64)
        counts = [0] * E
        counts[E - 3], counts[E - 1], counts[66 if E > 69 else 1] = R // 2, R // 4, R - R // 2 - R // 4
    T = 50
    x, sx = quant(rnd(g, T, K))
    w = experts(g, E, N, K)
    offsets = torch.tensor([0] + counts, device="cuda").cumsum(0).int()
    rows = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=I32)
    whole, o = guarded(R, N, F32)
    qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], offsets, rows=rows, out_dtype="fp32", out=o)
    check(o, gated_rows(x, sx, *w, offsets.tolist(), rows, "silu", "fp32"), (E, R, N, K), whole)
    o2 = qll.gated_fp8_grouped(x[rows.long()], *w[:2], sx[rows.long()], *w[2:], offsets, out_dtype="fp32")
    assert torch.equal(o, o2)


@pytest.mark.parametrize("E,R,N", [(70, 14100, 264), (6, 700, 2056), (8, 80, 4104)])
def test_gated_kernels_rows_of_nobody(qll, E, R, N):
    """The large tiles leave the rows that no expert owns, and tokens that are
    none read as zeros."""
    K = 80
    g = gen(E + R)
    T = 100
    x, sx = quant(rnd(g, T, K))
    w = experts(g, E, N, K)
    counts = spread(E, R - 9, g)
    offsets = torch.tensor([4] + counts, device="cuda").cumsum(0).int()
    rows = torch.randint(0, T, (R,), generator=g, device="cuda", dtype=I32)
    rows[::5] = torch.tensor([-1, T, 1 << 30, -(1 << 31), T + 1], dtype=I32, device="cuda").repeat(R)[:len(rows[::5])]
    o = torch.full((R, N), 7.0, dtype=F32, device="cuda")
    qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], offsets, rows=rows, out_dtype="fp32", out=o)
    assert (o[:4] == 7.0).all() and (o[offsets[-1]:] == 7.0).all()
    mine = torch.zeros(R, dtype=torch.bool, device="cuda")
    mine[4:offsets[-1]] = True
    none = torch.zeros_like(mine)
    none[::5] = True
    assert (o[mine & none] == 0).all()
    y, e = gated_rows(x, sx, *w, offsets.tolist(), rows.clamp(0, T - 1), "silu", "fp32")
    sel = mine & ~none
    assert ((o[sel].to(D) - y[sel]).abs() <= e[sel] + 1e-30).all()


# --------------------------------------------------------------------------
# past 32-bit offsets
# --------------------------------------------------------------------------

@pytest.mark.parametrize("counts", [(2, 1), (90, 60), (400, 300)])
def test_gated_weights_past_32_bits(qll, counts):
    """Experts whose weights start past 4 GiB."""
    E, N, K = 36, 8192, 16384  # 128 MiB an expert
    g = gen(1)
    w = [torch.zeros(E, N, K, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    s = [torch.ones(E, N, device="cuda") for _ in range(2)]
    for e in (E - 2, E - 1):
        for a, b in zip(w, s):
            a[e], b[e] = quant(rnd(g, N, K, std=0.05))
    x, sx = quant(rnd(g, 20, K))
    offsets = torch.zeros(E + 1, dtype=I32, device="cuda")
    offsets[E - 1:] = torch.tensor([counts[0], sum(counts)], dtype=I32, device="cuda")
    rows = torch.randint(0, 20, (sum(counts),), generator=g, device="cuda", dtype=I32)
    o = qll.gated_fp8_grouped(x, *w, sx, *s, offsets, rows=rows)
    cols = torch.randint(0, N, (64,), generator=g, device="cuda")
    y, e = gated_rows(x, sx, w[0][-2:, cols], w[1][-2:, cols], s[0][-2:, cols], s[1][-2:, cols], [0, counts[0], sum(counts)],
                      rows, "silu", "bf16")
    check(o[:, cols], (y, e), counts)


# (the test above has few rows an expert on average: one kernel, tiles of 64x64.)
# Tiles of 128x128, from 48 rows an expert on, and 256x128, from 192 on
@pytest.mark.parametrize("counts", [(900, 861), (3500, 3471)])
def test_gated_weights_past_32_bits_in_large_tiles(qll, counts):
    E, N, K = 36, 8192, 16384  # 128 MiB an expert: the last two start past 4 GiB
    g = gen(3)
    w = [torch.zeros(E, N, K, dtype=torch.float8_e4m3fn, device="cuda") for _ in range(2)]
    s = [torch.ones(E, N, device="cuda") for _ in range(2)]
    for e in (E - 2, E - 1):
        for a, b in zip(w, s):
            a[e], b[e] = quant(rnd(g, N, K, std=0.05))
    x, sx = quant(rnd(g, 20, K))
    offsets = torch.zeros(E + 1, dtype=I32, device="cuda")
    offsets[E - 1:] = torch.tensor([counts[0], sum(counts)], dtype=I32, device="cuda")
    rows = torch.randint(0, 20, (sum(counts),), generator=g, device="cuda", dtype=I32)
    o = qll.gated_fp8_grouped(x, *w, sx, *s, offsets, rows=rows)
    cols = torch.randint(0, N, (64,), generator=g, device="cuda")
    y, e = gated_rows(x, sx, w[0][-2:, cols], w[1][-2:, cols], s[0][-2:, cols], s[1][-2:, cols], [0, counts[0], sum(counts)],
                      rows, "silu", "bf16")
    check(o[:, cols], (y, e), counts)
    # rows of one token and one expert are equal, in every column
    for a, b in ((0, counts[0]), (counts[0], sum(counts))):
        first = torch.stack([(rows[a:b] == t).int().argmax() + a for t in range(20)])
        assert torch.equal(o[a:b], o[first[rows[a:b].long()]])


def test_combine_past_32_bits(qll):
    R, K, T, k = 300000, 8192, 5, 4
    y = torch.zeros(R, K, dtype=BF, device="cuda")
    g = gen(2)
    places = torch.randint(R - 50, R, (T, k), generator=g, device="cuda").int()
    places[0, 0] = 3
    places[1:, 0] = torch.arange(R - 60, R - 56, device="cuda").int()
    at = places.unique().long()
    y[at] = rnd(g, len(at), K)
    w, dout = rnd(g, T, k, dtype=F32), rnd(g, T, K)
    small = torch.searchsorted(at, places.long()).int()
    assert torch.equal(qll.moe_combine(y, places, w), qll.moe_combine(y[at], small, w))
    _, dw = qll.moe_combine_backward(y, places, w, dout, need_y=False)
    assert torch.equal(dw, qll.moe_combine_backward(y[at], small, w, dout, need_y=False)[1])


def test_sample_past_32_bits(qll):
    B, V = 15000, 151936  # 2.3 G values
    x = torch.zeros(B, V, dtype=BF, device="cuda")
    g = gen(3)
    x[-3:] = rnd(g, 3, V, std=3.0)
    u = torch.rand(B, generator=g, device="cuda")
    t = qll.sample_tokens(x, u)
    assert torch.equal(t[-3:], qll.sample_tokens(x[-3:].clone(), u[-3:]))
    # (a constant row: the token up to which more than u lies; V is exact in 64 bits)
    assert torch.equal(t[:9].long(), torch.floor(u[:9].to(D) * V).long())


# tokens and choices whose waves fill 2^32 threads, or all but a few, and one
# more than a launch takes
@pytest.mark.parametrize("T,k", [(1 << 26, 1), ((1 << 26) - 3, 1), ((1 << 26) // 3, 3), ((1 << 25) + 1, 1)])
def test_most_choices(qll, T, k):
    E, K = 4, 8
    g = gen(k)
    x = torch.randint(-8, 8, (T, E), generator=g, device="cuda", dtype=torch.int8).to(BF)
    ids, w = qll.moe_route(x, k, score="sigmoid", renormalize=False)
    key = x.to(torch.int8) * 4 + (3 - torch.arange(E, dtype=torch.int8, device="cuda"))  # in order, ties too
    order = torch.empty_like(ids)
    for j in range(k):
        best = key.amax(1, keepdim=True)
        order[:, j:j + 1] = 3 - (best & 3)
        key = torch.where(key == best, -128, key)
    assert torch.equal(ids, order)
    # (logits of 16 values: a weight and a slope each, off by a few u; u = 2^-24)
    v = torch.arange(-8, 8, device="cuda", dtype=D)
    p = torch.sigmoid(v)
    at = x.gather(1, order.long()).long() + 8
    assert ((w - p[at].float()).abs() <= 40 * 2.0 ** -24 * w).all()
    dw = torch.randint(1, 3, (T, k), generator=g, device="cuda", dtype=torch.int8).float()
    dx = qll.moe_route_backward(x, ids, dw, score="sigmoid", renormalize=False)
    want = torch.zeros(T, E, device="cuda").scatter_(1, order.long(), dw * (p * torch.sigmoid(-v))[at].float())
    # (and the bf16 output's half step, 2^-8)
    assert ((dx.float() - want).abs() <= (2.0 ** -8 + 80 * 2.0 ** -24) * want).all()
    del x, key, dx, want, order, at
    planned = qll.moe_sort(ids, E)
    flat = ids.reshape(-1)
    assert torch.equal(planned[0][1:], torch.bincount(flat, minlength=E).cumsum(0).int())
    expert = torch.bucketize(planned[2].reshape(-1), planned[0][1:], right=True)
    assert torch.equal(expert.int(), flat)  # (each choice in its expert's rows)
    assert torch.equal(planned[1][planned[2].long()], torch.arange(T, device="cuda", dtype=I32)[:, None].expand(T, k))
    places = planned[2]
    y = torch.randint(-4, 5, (T * k, 1), generator=g, device="cuda", dtype=torch.int8).to(BF).repeat(1, K)
    dout = torch.randint(-4, 5, (T, 1), generator=g, device="cuda", dtype=torch.int8).to(BF).repeat(1, K)
    # (small whole numbers: every product and sum is exact)
    dy, got = qll.moe_combine_backward(y, places, dw, dout)
    assert torch.equal(got, K * dout[:, :1].float() * y[:, 0].float()[places.long()])
    assert torch.equal(dy[:, 0][places.long()], (dw * dout[:, :1]).to(BF))
    assert torch.equal(dy[:, 0], dy[:, K - 1])


# --------------------------------------------------------------------------
# two at once
# --------------------------------------------------------------------------

def test_two_streams_at_once(qll):
    """Calls that overlap on two streams keep to their own workspaces."""
    g = gen(6)
    x = [rnd(g, 3000, 64, dtype=F32) for _ in range(2)]
    logits = [rnd(g, 3, 60000, std=2.0, dtype=F32) for _ in range(2)]
    u = torch.rand(3, generator=g, device="cuda")
    want = [(qll.moe_route(a, 8, plan=True), qll.sample_tokens(b, u)) for a, b in zip(x, logits)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got.append((qll.moe_route(x[i], 8, plan=True), qll.sample_tokens(logits[i], u)))
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert all(torch.equal(p, q) for p, q in zip(a[0], b[0])) and torch.equal(a[1], b[1])


def test_two_graphs_share_a_workspace(qll):
    """Graphs captured with one workspace, replayed one after the other."""
    g = gen(7)
    x = [rnd(g, 2000, 48, dtype=F32) for _ in range(2)]
    logits = [rnd(g, 2, 50000, std=2.0) for _ in range(2)]
    u = torch.rand(2, generator=g, device="cuda")
    ws = torch.empty(max(qll.load_library().qll_moe_sort_workspace_bytes(2000, 48, 6),
                         qll.load_library().qll_sample_workspace_bytes(2, 50000)), dtype=torch.uint8, device="cuda")
    want = [(qll.moe_route(a, 6, plan=True), qll.sample_tokens(b, u)) for a, b in zip(x, logits)]
    s = torch.cuda.Stream()
    graphs, outs = [], []
    for i in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=s):
            outs.append((qll.moe_route(x[i], 6, plan=True, workspace=ws), qll.sample_tokens(logits[i], u, workspace=ws)))
        graphs.append(graph)
    for rep in range(4):
        ws.fill_(0xA5)
        for o in outs:
            for t in (*o[0], o[1]):
                t.fill_(0)
        torch.cuda.synchronize()
        for i in (rep % 2, 1 - rep % 2):
            graphs[i].replay()
        torch.cuda.synchronize()
        for a, b in zip(outs, want):
            assert all(torch.equal(p, q) for p, q in zip(a[0], b[0])) and torch.equal(a[1], b[1]), rep


# --------------------------------------------------------------------------
# sampling: rows whose sample misleads
# --------------------------------------------------------------------------

def test_sorted_and_clustered_rows(qll):
    """Largest values all at one end, in one place, or far above all others: the
    sample that sets the bins and the list sees none or only them."""
    V = 60000
    g = gen(9)
    x = torch.randn(10, V, generator=g, device="cuda") * 2
    x[0], x[1] = x[0].sort().values, x[1].sort(descending=True).values
    x[2, 30010:30400] += 30
    x[3, 59999] = 500.0
    x[4, 59000:] = 90.0
    x[5, 41] = 25.0
    x[6] = x[6].round()
    x[7, ::2] = -float("inf")
    x[8, :59990] = -float("inf")
    x[9, 20000:20003] = torch.tensor([60.0, 61.0, 62.0], device="cuda")
    opts = [dict(), dict(top_k=300), dict(top_p=0.9), dict(min_p=0.01), dict(top_k=3000, top_p=0.95), dict(temperature=0.0),
            dict(top_k=500, min_p=1e-3), dict(top_p=0.5, min_p=0.1)]
    for dtype in (F32, BF):
        for temp in (1.0, 0.3, 2.0):
            for o in opts:
                kw = expand([o], 10)
                kw["temperature"] = [t if t <= 0 else temp for t in kw["temperature"]]
                u = torch.rand(10, generator=g, device="cuda").tolist()
                run(qll, x.to(dtype), u, (dtype, temp, o), **kw)
                # one row at a time: split over workgroups
                run(qll, x[2:3].to(dtype), u[:1], (dtype, temp, o, "one"), **{k: v[:1] for k, v in kw.items()})


@pytest.mark.parametrize("B", [1, 2, 17, 128, 129, 300])
def test_rows_per_call(qll, B):
    """Rows over several workgroups, or one each."""
    V = 33000
    g = gen(B)
    x = torch.randn(B, V, generator=g, device="cuda") * 3
    u = torch.rand(B, generator=g, device="cuda").tolist()
    run(qll, x, u, B, **expand([dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.7), dict(min_p=0.02), dict(temperature=0.0)], B))


# --------------------------------------------------------------------------
# lists that start at any 4 bytes, outputs and workspaces of the caller
# --------------------------------------------------------------------------

def shifted(t, fill=0):
    """A copy of t, contiguous, that starts 4 bytes past a 16-byte border."""
    buf = torch.full((t.numel() + 9,), fill, dtype=t.dtype, device="cuda")
    at = next(i for i in range(1, 5) if buf[i:].data_ptr() % 16 == 4)
    out = buf[at:at + t.numel()].view(t.shape)
    out.copy_(t)
    return out


@pytest.mark.parametrize("T,k", [(5, 4), (300, 8)])
def test_lists_at_any_four_bytes(qll, T, k):
    E, N, K = 16, 144, 160
    g = gen(T)
    logits, w = rnd(g, T, E, dtype=F32), experts(g, E, N, K)
    want = qll.moe_route(logits, k, plan=True)
    outs = [shifted(t, 7) for t in want]
    for t in outs:
        t.fill_(-9)
    bias = rnd(g, E, dtype=F32)
    for b in (None, bias):
        want = qll.moe_route(logits, k, bias=b, plan=True)
        ws = torch.empty(max(16, qll.load_library().qll_moe_sort_workspace_bytes(T, E, k)), dtype=torch.uint8, device="cuda")
        got = qll.moe_route(logits, k, bias=None if b is None else shifted(b), plan=True, ids=outs[0], weights=outs[1],
                            offsets=outs[2], rows=outs[3], places=outs[4], workspace=ws)
        for a, o, t in zip(want, outs, got):
            assert t is o and torch.equal(a, o)
    ids, weights, offsets, rows, places = outs
    for a, o in zip(want[2:], qll.moe_sort(ids, E, offsets=shifted(offsets), rows=shifted(rows), places=shifted(places))):
        assert torch.equal(a, o)
    dw = rnd(g, T, k, dtype=F32)
    assert torch.equal(qll.moe_route_backward(logits, ids, shifted(dw)), qll.moe_route_backward(logits, want[0], dw))
    x, sx = quant(rnd(g, T, K))
    a = qll.gated_fp8_grouped(x, *w[:2], shifted(sx), *(shifted(s) for s in w[2:]), offsets, rows=rows)
    assert torch.equal(a, qll.gated_fp8_grouped(x, *w[:2], sx, *w[2:], want[2], rows=want[3]))
    y, dout = rnd(g, T * k, K), rnd(g, T, K)
    assert torch.equal(qll.moe_combine(y, places, weights), qll.moe_combine(y, want[4], want[1]))
    for p, q in zip(qll.moe_combine_backward(y, places, weights, dout, dweights=shifted(weights)),
                    qll.moe_combine_backward(y, want[4], want[1], dout)):
        assert torch.equal(p, q)
    u = torch.rand(T, generator=g, device="cuda")
    v = rnd(g, T, 501, dtype=F32)
    kw = dict(temperature=u + 0.5, top_k=(u * 50).int(), top_p=1 - u / 4, min_p=u / 50)
    want = qll.sample_tokens(v, u, probs=True, **kw)
    got = qll.sample_tokens(v, shifted(u), probs=shifted(u), tokens=shifted(want[0]), **{n: shifted(t) for n, t in kw.items()})
    assert all(torch.equal(p, q) for p, q in zip(want, got))


def test_choices_of_one_expert(qll):
    """Every token to the same few experts, and ids that name one twice."""
    T, E, k = 3000, 128, 4
    ids = torch.full((T, k), 77, dtype=I32, device="cuda")
    ids[:, 1] = 3
    offsets, rows, places = qll.moe_sort(ids, E)
    flat = ids.reshape(-1).long()
    by = torch.argsort(flat, stable=True)
    same(rows, (by // k).int(), "rows")
    same(places.reshape(-1)[by], torch.arange(T * k, dtype=I32, device="cuda"), "places")
    assert offsets[77] == T and offsets[78] == T * k and offsets[3] == 0 and offsets[E] == T * k
    # gradients of an expert that is named twice add up
    logits = rnd(gen(5), 64, E, dtype=F32)
    dw = rnd(gen(6), 64, k, dtype=F32)
    d = qll.moe_route_backward(logits, ids[:64].contiguous(), dw, renormalize=False)
    one = torch.tensor([[77, 3]], dtype=I32, device="cuda").repeat(64, 1)
    both = torch.stack([dw[:, 0] + dw[:, 2] + dw[:, 3], dw[:, 1]], 1)
    e = qll.moe_route_backward(logits, one, both, renormalize=False)
    # (sums of the same terms in another order: a few roundings of their sizes)
    assert ((d - e).abs() <= 16 * 2.0 ** -24 * dw.abs().sum(1, keepdim=True)).all()


@pytest.mark.parametrize("level", [-30.0, -38.0, -41.0, -60.0, -95.0, -150.0, -650.0])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_sigmoids_next_to_nothing(qll, dtype, level):
    """Renormalised sigmoids of logits far below zero are weights like any."""
    T, E, k = 50, 96, 6
    g = gen(int(-level))
    x = (level + rnd(g, T, E, std=3.0, dtype=F32)).to(dtype)
    ids, w = qll.moe_route(x, k, score="sigmoid")
    order = torch.sort(x.to(D), dim=1, descending=True, stable=True).indices[:, :k]
    same(ids, order.int(), "ids")
    chosen = x.to(D).gather(1, order)
    p = torch.sigmoid(chosen)
    want = p / p.sum(1, keepdim=True)
    # (the exponent's rounding, |x| 2^-24 where it is not relative to the largest)
    far = torch.where(chosen < -36, chosen[:, :1] - chosen, -chosen.clamp(max=0)) + 3
    far = far.clamp(min=0) + (-chosen).clamp(0, 42)
    bound = (2 * far.amax(1, keepdim=True) + 40) * 2.0 ** -24
    assert ((w.to(D) - want).abs() <= bound * want).all()
    dw = rnd(g, T, k, dtype=F32)
    dx = qll.moe_route_backward(x, ids, dw, score="sigmoid")
    mag = want * torch.sigmoid(-chosen)
    dot = (dw.to(D) * want).sum(1, keepdim=True)
    got = dx.to(D).gather(1, order)
    size = mag * (dw.to(D).abs() + (dw.to(D).abs() * want).sum(1, keepdim=True))
    step = torch.finfo(dtype).eps / 2
    assert ((got - mag * (dw.to(D) - dot)).abs() <= (2 * bound + step * 1.01) * size + 1e-37).all()
    assert (dx.scatter(1, order, 0) == 0).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_experts_at_the_lowest_value(qll, dtype):
    """A row of the type's lowest value: sigmoids and gradients are 0, softmax
    weights even; a row with two other experts takes these first."""
    x = torch.full((3, 40), torch.finfo(dtype).min, dtype=dtype, device="cuda")
    x[1, 33], x[1, 5] = 1.0, 0.0
    x[2] = -INF
    ids, w = qll.moe_route(x, 4, score="sigmoid")
    assert ids[0].tolist() == [0, 1, 2, 3] and ids[1].tolist() == [33, 5, 0, 1] and ids[2].tolist() == [0, 1, 2, 3]
    assert (w[0] == 0).all() and (w[2] == 0).all() and (w[1, 2:] == 0).all()
    p = torch.sigmoid(torch.tensor([1.0, 0.0], dtype=D, device="cuda"))
    assert ((w[1, :2].to(D) - p / p.sum()).abs() <= 50 * 2.0 ** -24).all()
    for renorm in (True, False):
        dx = qll.moe_route_backward(x, ids, torch.ones_like(w), score="sigmoid", renormalize=renorm)
        assert (dx[0] == 0).all() and (dx[2] == 0).all() and torch.isfinite(dx.float()).all()
    w = qll.moe_route(x, 4)[1]
    assert ((w[0] - 0.25).abs() <= 1e-6).all() and (w[2] == 0).all() and (w[1, 2:] == 0).all()
