"""GPU parity of sample_tokens against its definition in 64 bits
(moe_reference.sample_row): the same tokens, exactly, and shares within 2^-22
(a few fp32 roundings of a 64-bit quotient): every option alone and together,
ties, vocabularies from one token to 2^20, padded and unaligned rows, rows that
are not finite, temperatures from tiny to infinite."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import moe_reference as ref  # noqa: E402
from test_gpu_ffn import BF, F32, gen, qll  # noqa: E402,F401

NAN, INF = float("nan"), float("inf")
I32 = torch.int32


def run(qll, x, u, what="", **kw):
    """Calls with per-row lists, checks every row, returns the tokens."""
    t = {k: torch.tensor(v, dtype=I32 if k == "top_k" else F32, device="cuda") for k, v in kw.items()}
    ut = torch.tensor(u, dtype=F32, device="cuda")
    tokens, probs = qll.sample_tokens(x, ut, probs=True, **t)
    assert torch.equal(tokens, qll.sample_tokens(x, ut, **t))
    host = x.cpu()
    for b in range(x.shape[0]):
        opts = {k: v[b].item() for k, v in t.items()}
        token, share = ref.sample_row(host[b], ut[b].item(), **opts)
        got = (tokens[b].item(), probs[b].item())
        assert got[0] == token, (what, b, opts, u[b], got, (token, share))
        assert abs(got[1] - share) <= 2.0 ** -22 * share + 1e-30, (what, b, opts, got, share)
    return tokens


def rows(seed, B, V, dtype, std=2.0, likely=0, height=10.0):
    g = gen(seed)
    x = torch.randn(B, V, generator=g, device="cuda") * std
    if likely:
        at = torch.randint(0, V, (B, likely), generator=g, device="cuda")
        x.scatter_(1, at, height + torch.randn(B, likely, generator=g, device="cuda") * 2)
    u = torch.rand(B, generator=g, device="cuda").tolist()
    return x.to(dtype), u


OPTIONS = [dict(), dict(top_k=1), dict(top_k=2), dict(top_k=50), dict(top_k=5000), dict(top_p=0.9), dict(top_p=0.3),
           dict(top_p=0.0), dict(min_p=0.05), dict(min_p=1.0), dict(min_p=3.0), dict(top_k=40, top_p=0.8),
           dict(top_k=40, top_p=0.95, min_p=0.02), dict(top_p=0.97, min_p=1e-4), dict(top_k=3000, top_p=0.99),
           dict(top_k=20000, top_p=0.9999, min_p=1e-6), dict(min_p=1e-9), dict(top_p=0.999999), dict(temperature=0.0),
           dict(temperature=-1.0, top_k=5), dict(top_k=-3, top_p=2.0, min_p=-1.0)]


def expand(options, n):
    """Per-row lists of every option that any row sets."""
    off = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)
    options = [options[i % len(options)] for i in range(n)]
    return {k: [o.get(k, v) for o in options] for k, v in off.items()}


@pytest.mark.parametrize("V", [1, 2, 3, 7, 8, 63, 64, 1000, 4099, 32000, 50021, 151936])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_options(qll, dtype, V):
    B = len(OPTIONS)
    for likely, height in ((0, 0.0), (min(V, 20), 9.0), (min(V, 20), 14.0)):
        x, u = rows(V + likely, B, V, dtype, likely=likely, height=height)
        for temp in (None, 0.7, 1.3):
            kw = expand(OPTIONS, B)
            if temp:
                kw["temperature"] = [t if t <= 0 else temp for t in kw["temperature"]]
            run(qll, x, u, (V, likely, height, temp), **kw)


@pytest.mark.parametrize("name", ["temperature", "top_k", "top_p", "min_p", None])
def test_options_alone(qll, name):
    x, u = rows(5, 8, 3001, F32)
    values = dict(temperature=[0.5, 2.0] * 4, top_k=[3, 0] * 4, top_p=[0.5, 1.0] * 4, min_p=[0.1, 0.0] * 4)
    run(qll, x, u, name, **({name: values[name]} if name else {}))


@pytest.mark.parametrize("temp", [1e-42, 1e-30, 1e-6, 0.01, 0.1, 10.0, 1e4, 1e30, INF, NAN])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_temperatures(qll, dtype, temp):
    """A narrow scale has one token, a wide one makes all equal (more values in
    a bin than the list holds)."""
    opts = [dict(), dict(top_k=7), dict(top_p=0.5), dict(top_k=9000, top_p=0.7), dict(min_p=0.2), dict(top_p=0.9, min_p=0.5)]
    for V in (500, 20011):
        x, u = rows(V, len(opts), V, dtype)
        kw = expand(opts, len(opts))
        kw["temperature"] = [temp] * len(opts)
        run(qll, x, u, (V, temp), **kw)


@pytest.mark.parametrize("V", [5, 4096, 4097, 30000, 262144])
def test_equal_logits(qll, V):
    """Ties go to the lower index: a constant row, two values, half masked."""
    opts = [dict(), dict(top_k=3), dict(top_k=V // 2 + 1), dict(top_p=0.5), dict(top_p=0.25, top_k=V // 2), dict(min_p=0.5),
            dict(min_p=1.0, top_p=0.75)]
    B = len(opts)
    u = [(i + 0.5) / B for i in range(B)]
    for make in (lambda x: x, lambda x: x.__setitem__((slice(None), slice(1, None, 2)), 0.5),
                 lambda x: x.__setitem__((slice(None), slice(0, V // 2)), -INF),
                 lambda x: x.__setitem__((slice(None), slice(0, None, 3)), -3e38)):
        x = torch.zeros(B, V, device="cuda")
        make(x)
        run(qll, x, u, V, **expand(opts, B))
        run(qll, x, [0.0] * B, V, **expand(opts, B))
        run(qll, x, [1.0 - 2.0 ** -24] * B, V, **expand(opts, B))


def test_rounded_logits(qll):
    """Few distinct values, many ties at every border."""
    for V in (3000, 60000):
        x, u = rows(V, len(OPTIONS), V, F32)
        run(qll, (x * 2).round() / 2, u, V, **expand(OPTIONS, len(OPTIONS)))


def test_rows_that_are_not_finite(qll):
    V = 5000
    x, u = rows(3, 12, V, F32)
    x[0] = -INF
    x[1] = NAN
    x[2, ::2] = NAN
    x[3, 100] = NAN
    x[4, 77] = INF
    x[5, 10::10] = INF
    x[6, 1:] = -INF
    x[7, 5] = -3.4e38
    x[8] = -3.4e38
    x[9, 3:] = -3.4e38
    x[10] *= 1e30
    for opts in ([dict()], [dict(top_k=20)], [dict(top_p=0.6)], [dict(min_p=0.3)], [dict(temperature=0.0)],
                 [dict(top_k=100, top_p=0.5, min_p=0.01)], [dict(min_p=2.0)]):
        run(qll, x, u, opts, **expand(opts, 12))
        run(qll, x[:2], [0.5, NAN], opts, **expand(opts, 2))


@pytest.mark.parametrize("V", [8000, 20011])
def test_rows_with_the_largest_value(qll, V):
    """The type's largest value, once among rows that are masked in part, many
    times, or in every place: a number like any other."""
    opts = [dict(), dict(top_k=5), dict(top_k=V // 3), dict(top_p=0.5), dict(min_p=0.3), dict(top_p=0.9, min_p=0.5),
            dict(temperature=INF), dict(temperature=INF, top_k=V - 3), dict(temperature=INF, top_p=0.75), dict(temperature=0.0)]
    B = len(opts)
    u = [(i + 0.5) / B for i in range(B)]
    for dtype in (F32, BF):
        x, _ = rows(V, B, V, dtype)
        top = torch.finfo(dtype).max
        x[:, 1000] = top
        kinds = [x, x.clone(), x.clone(), torch.full_like(x, top), torch.full_like(x, top)]
        kinds[1][:, :V // 4] = -INF
        kinds[1][:, V - 1] = top
        kinds[2][:, ::2] = top
        kinds[4][:, 1::3] = -top
        for i, t in enumerate(kinds):
            run(qll, t, u, (V, i), **expand(opts, B))
            run(qll, t, [0.0] * B, (V, i), **expand(opts, B))
            run(qll, t, [1.0 - 2.0 ** -24] * B, (V, i), **expand(opts, B))


def run_small_weights(qll, x, u, what, **kw):
    """As run, for rows that have weights below e^-31.9, which may be taken as 0.
    Their sum `gone` moves a sum over all weights to anywhere in [z - gone, z],
    and a bin's weight is off by up to 2^-37 of itself (err).  The kept front then
    ends at the first token whose sum reaches p z or p (z - gone), and the token
    is one of those between the first sums past u times the least and the most
    that is kept."""
    t = {k: torch.tensor(v, dtype=I32 if k == "top_k" else F32, device="cuda") for k, v in kw.items()}
    ut = torch.tensor(u, dtype=F32, device="cuda")
    tokens, probs = qll.sample_tokens(x, ut, probs=True, **t)
    for b in range(x.shape[0]):
        k, p, m = (t[n][b].item() for n in ("top_k", "top_p", "min_p"))
        xs, order = torch.sort(x[b].cpu().double(), descending=True, stable=True)
        w = torch.exp((xs - xs[0]) / t["temperature"][b].item())
        n = k if 0 < k < len(w) else len(w)
        c = torch.cumsum(w, 0)
        gone, err = float(w[:n][w[:n] < math.exp(-31.9)].sum()), 2.0 ** -37 * float(c[n - 1])
        first = lambda v: min(int((c < v).sum()), n - 1)  # noqa: E731
        ends = [n - 1, n - 1] if p >= 1 else [first(p * (c[n - 1] - gone) - err), first(p * c[n - 1] + err)]
        if m > 0:
            ends = [min(e, int((w >= m).sum()) - 1) for e in ends]
        least, most = (float(c[ends[0]]) - gone - err) * ut[b].item(), (float(c[ends[1]]) + err) * ut[b].item()
        at = int((order == tokens[b].item()).nonzero())
        assert min(int((c <= least - err).sum()), ends[0]) <= at <= min(int((c <= most + err).sum()), ends[1]), (what, b, u[b], at)
        share = float(w[at] / c[ends[1]])
        assert abs(probs[b].item() - share) <= 2.0 ** -22 * share + 1e-30, (what, b, u[b], probs[b].item(), share)


@pytest.mark.parametrize("temp,above", [(0.75, 12.0234375), (1.5, 24.046875), (3.0, 48.09375), (0.375, 6.01171875)])
def test_maximum_at_the_border_of_the_first_bin(qll, temp, above):
    """A maximum outside the sample that lies 1026 / 64 temperatures above the
    sample's, in exact numbers; the rounded inverse temperature puts it a last
    bit inside of the first bin."""
    V = 20011
    check = run if (above + 8) / temp < 31.9 else run_small_weights
    for B in (1, 3, 140):
        g = gen(B)
        x = -torch.rand(B, V, generator=g, device="cuda") * 8
        x[:, ::100] = 0.0
        x[:, 4500] = above
        for o in (dict(), dict(top_k=50), dict(top_p=0.9), dict(min_p=1e-7), dict(top_p=0.99999995, top_k=9000)):
            kw = expand([dict(o, temperature=temp)], B)
            check(qll, x, torch.rand(B, generator=g, device="cuda").tolist(), (B, o), **kw)
            check(qll, x, [1.0 - 2.0 ** -24] * B, (B, o), **kw)


def test_random_numbers_at_the_ends(qll):
    """0, the last value below 1, and what is no random number at all."""
    x, _ = rows(9, 6, 2000, F32)
    for o in (dict(), dict(top_k=10), dict(top_p=0.7)):
        run(qll, x, [0.0, 1.0 - 2.0 ** -24, 2.0 ** -30, 0.5, -1.0, NAN], o, **expand([o], 6))
        t = qll.sample_tokens(x, torch.full((6,), 1.5, device="cuda"), top_k=torch.full((6,), 4, dtype=I32, device="cuda"))
        assert (t == x.topk(4, dim=1).indices[:, 3].int()).all()


@pytest.mark.parametrize("V,ld,start", [(999, 1024, 0), (1000, 1001, 1), (4097, 4100, 3), (5, 7, 1)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_padded_and_unaligned_rows(qll, dtype, V, ld, start):
    """What lies between the rows is never chosen."""
    B = 7
    g = gen(V)
    whole = torch.full((B * ld + start + 8,), 100.0, device="cuda", dtype=dtype)
    x = whole[start:start + B * ld].view(B, ld)[:, :V]
    x.copy_(torch.randn(B, V, generator=g, device="cuda"))
    u = torch.rand(B, generator=g, device="cuda").tolist()
    run(qll, x, u, (V, ld), **expand([dict(), dict(top_k=3), dict(top_p=0.9)], B))


def test_largest_vocabulary(qll):
    V = 1 << 20
    x, u = rows(1, 4, V, F32)
    run(qll, x, u, V, **expand([dict(), dict(top_p=0.9), dict(top_k=1000, top_p=0.5), dict(min_p=1e-5)], 4))
    run(qll, torch.zeros(4, V, device="cuda"), u, V, **expand([dict(), dict(top_p=0.9), dict(top_k=700001), dict(min_p=1e-5)], 4))


def test_many_rows(qll):
    x, u = rows(2, 700, 257, BF)
    run(qll, x, u, "rows", **expand(OPTIONS, 700))


def test_distribution(qll):
    """Evenly spread random numbers give every token its share: a row of 8
    tokens, u = (i + 0.5) / 4096, counts within one of 4096 p."""
    x = torch.tensor([[0.3, -1.0, 2.0, 0.0, 1.1, -0.4, 0.9, 1.7]], device="cuda").repeat(4096, 1)
    u = (torch.arange(4096, device="cuda") + 0.5) / 4096
    t = qll.sample_tokens(x, u)
    p = torch.softmax(x[0].double(), 0)
    assert ((torch.bincount(t.long(), minlength=8) - 4096 * p).abs() <= 1).all()


def test_streams_and_graphs(qll):
    x, u = rows(21, 5, 40000, F32, likely=10)
    kw = {k: torch.tensor(v, dtype=I32 if k == "top_k" else F32, device="cuda")
          for k, v in expand([dict(), dict(top_k=30), dict(top_p=0.9), dict(min_p=0.01)], 5).items()}
    ut = torch.tensor(u, device="cuda")
    want = qll.sample_tokens(x, ut, probs=True, **kw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = qll.sample_tokens(x, ut, probs=True, stream=s, **kw)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    tokens, probs = torch.empty(5, dtype=I32, device="cuda"), torch.empty(5, device="cuda")
    with torch.cuda.stream(s):
        qll.sample_tokens(x, ut, probs=probs, tokens=tokens, **kw)
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=s):
        qll.sample_tokens(x, ut, probs=probs, tokens=tokens, **kw)
    for rep in range(4):
        if rep == 2:
            x.copy_(x.flip(1))
        tokens.fill_(-9)
        probs.fill_(-9.0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = qll.sample_tokens(x, ut, probs=True, **kw)
        assert torch.equal(tokens, want[0]) and torch.equal(probs, want[1]), rep


def test_no_rows_and_refusals(qll):
    x, u = torch.zeros(3, 50, device="cuda"), torch.zeros(3, device="cuda")
    assert qll.sample_tokens(x[:0], u[:0]).shape == (0,)
    for call in (lambda: qll.sample_tokens(x.half(), u), lambda: qll.sample_tokens(x, u[:2]),
                 lambda: qll.sample_tokens(x.cpu(), u), lambda: qll.sample_tokens(x.t(), torch.zeros(50, device="cuda")),
                 lambda: qll.sample_tokens(x[0], u), lambda: qll.sample_tokens(x, u, top_k=u),
                 lambda: qll.sample_tokens(x, u, temperature=1.0), lambda: qll.sample_tokens(x[:1].expand(3, 50), u),
                 lambda: qll.sample_tokens(x, u, tokens=torch.zeros(3, dtype=torch.int64, device="cuda"))):
        with pytest.raises((ValueError, TypeError)):
            call()
    with pytest.raises(qll.QllError):
        qll.sample_tokens(torch.zeros(1, (1 << 20) + 1, device="cuda"), u[:1])
