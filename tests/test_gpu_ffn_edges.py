"""GPU tests of the feed-forward operators at their edges: empty batches, rows
that are not finite, activations far from zero, and the paths that only some
sizes take.  Formulas and bounds: tests/ffn_reference.py."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import ffn_reference as ref  # noqa: E402
from test_gpu_ffn import BF, D, F32, check, gen, guarded, qll, rnd  # noqa: E402,F401

NAN, INF = float("nan"), float("inf")


# --------------------------------------------------------------------------
# empty batches
# --------------------------------------------------------------------------

@pytest.mark.parametrize("act", ["none", "silu"])
def test_no_tokens_with_frozen_weights(qll, act):
    """No tokens and the input's gradient alone (an empty tensor's address is
    null): an empty gradient, as for the forward calls."""
    g = gen(1)
    x, d = torch.empty(0, 64, dtype=BF, device="cuda"), torch.empty(0, 24, dtype=BF, device="cuda")
    w, b = rnd(g, 24, 64), rnd(g, 24)
    dA, dB, db = qll.gemm_bf16_epilogue_backward(x, w, d, act=act, need_weight=False)
    assert dA.shape == (0, 64) and dB is None and db is None
    dA, dB, db = qll.gemm_bf16_epilogue_backward(x, w, d, bias=b, act=act, need_weight=False)
    assert dA.shape == (0, 64) and dB is None and (db == 0).all()
    got = qll.gated_bf16_backward(x, w, w, d, need_weight=False)
    assert got[0].shape == (0, 64) and got[1] is None and got[2] is None


# --------------------------------------------------------------------------
# rows that are not finite
# --------------------------------------------------------------------------

@pytest.mark.parametrize("M,K", [(3, 16), (5, 4096), (4, 6160), (1100, 2048), (3, 32768)])
@pytest.mark.parametrize("post", [False, True])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_bad_rows_of_the_e4m3_norm(qll, stream, post, M, K):
    """A row with a NaN or an infinity has a NaN scale (its normed values are
    NaN where the row's rms or the value is), never a clean zero row; NaN
    normed values have NaN codes; the other rows keep their bits."""
    g = gen(M + K)
    st = BF if stream == "bf16" else F32
    y, r = rnd(g, M, K), rnd(g, M, K, dtype=st)
    w, w1 = rnd(g, K, std=0.2) + 1, (rnd(g, K, std=0.2) + 1 if post else None)
    at = M // 2
    rest = [m for m in range(M) if m != at]
    _, q0, s0 = qll.residual_norm(y, r, w, w_post=w1, quantize=True)
    for block in (True, False):
        clean = (s0, q0) if block else qll.residual_norm(None, r, w, quantize=True)[:0:-1]
        for which in ("y", "r"):
            for bad in (NAN, INF, -INF):
                if which == "y" and not block:
                    continue
                y2, r2 = y.clone(), r.clone()
                (y2 if which == "y" else r2)[at, K - 1] = bad
                a = (y2 if block else None, r2, w)
                kw = dict(w_post=w1 if block else None)
                n = qll.residual_norm(*a, **kw)[1].float()
                _, q, s = qll.residual_norm(*a, quantize=True, **kw)
                what = (which, bad, block)
                assert torch.isnan(n[at]).any(), what
                assert torch.isnan(s[at]).all(), what
                assert torch.isnan(q[at].float()).all(), what
                assert torch.equal(s[rest], clean[0][rest]), what
                assert torch.equal(q.view(torch.uint8)[rest], clean[1].view(torch.uint8)[rest]), what


def test_infinite_normed_values_of_the_e4m3_norm(qll):
    """An infinite norm weight: an infinite scale, by the formula, under which
    infinite values have NaN codes and finite ones zero codes."""
    g = gen(3)
    r, w = rnd(g, 4, 64) + 3, rnd(g, 64, std=0.2) + 1
    w[7] = INF
    _, q, s = qll.residual_norm(None, r, w, quantize=True)
    q = q.float()
    assert torch.isinf(s).all() and torch.isnan(q[:, 7]).all()
    assert (torch.cat([q[:, :7], q[:, 8:]], 1) == 0).all()


@pytest.mark.parametrize("M", [5, 70, 300])
@pytest.mark.parametrize("act", ["gelu", "gelu_tanh", "silu", "sigmoid"])
def test_a_bad_token_has_bad_gradients(qll, act, M):
    """A NaN pre-activation has a NaN slope: the token's own gradient, and
    those of the weights and biases, which sum over the tokens, show it."""
    N, K = 200, 80
    g = gen(M)
    x, wg, wu, dout, b = rnd(g, M, K), rnd(g, N, K), rnd(g, N, K), rnd(g, M, N), rnd(g, N)
    x[M // 2] = NAN
    rest = [m for m in range(M) if m != M // 2]
    for bias in (b, None):
        dA, dB, db = qll.gemm_bf16_epilogue_backward(x, wg, dout, bias=bias, act=act)
        assert torch.isnan(dA[M // 2]).all() and torch.isfinite(dA[rest]).all()
        assert torch.isnan(dB).all() and (bias is None or torch.isnan(db).all())
    # the gate's pre-activation alone: through its weights
    clean = x.clone()
    clean[M // 2] = 1
    bad = wg.clone()
    bad[3] = NAN
    dA, dB, db = qll.gemm_bf16_epilogue_backward(clean, bad, dout, bias=b, act=act, need_input=False)
    assert torch.isnan(dB[3]).all() and torch.isnan(db[3])
    assert torch.isfinite(dB[:3]).all() and torch.isfinite(dB[4:]).all() and torch.isfinite(db[:3]).all()
    _, dBg, dBu = qll.gated_bf16_backward(clean, bad, wu, dout, act=act, need_input=False)
    for t in (dBg, dBu):
        assert torch.isnan(t[3]).all() and torch.isfinite(t[:3]).all() and torch.isfinite(t[4:]).all()


# --------------------------------------------------------------------------
# activations far from zero: bounds relative to the value itself
# --------------------------------------------------------------------------

def diagonal(z):
    """x [M][K], w [N][K] with x w^T = z in every row, exactly: one product of
    z[n] with 1, the rest zero."""
    N = z.numel()
    return torch.ones(70, N, dtype=BF, device="cuda"), torch.diag(z).to(BF).contiguous()


@pytest.mark.parametrize("M", [1, 70])
def test_gelu_is_accurate_relative_to_itself(qll, M):
    """gelu(z) = z Phi(z) in fp32, the product exact.  Phi(z) is e^(-z^2/2)
    times a function fitted to 2^-23; the exponent is off by z^2/2 times 2.5
    u (its square, its product, the constant), u = 2^-24; the exponential and
    the reciprocal by 2 u each, ten roundings of at most u follow: at most
    (1.25 z^2 + 16) u of the result.  The exponential keeps its bits down to
    2^-126, z = -13."""
    z = torch.cat([torch.linspace(-12, 12, 769), torch.linspace(-3, 3, 511)]).to(BF)
    z = torch.cat([z, z[:1280 - z.numel()]]).cuda()
    x, w = diagonal(z)
    got = qll.gemm_bf16_epilogue(x[:M], w, act="gelu", out_dtype="fp32").to(D)
    zd = z.to(D)
    want = zd * 0.5 * torch.special.erfc(-zd / math.sqrt(2))
    bound = (1.25 * zd * zd + 16) * 2.0 ** -24 * want.abs()
    for m in range(M):
        check(got[m], (want, bound), ("gelu", m))


def test_sigmoid_slope_is_accurate_relative_to_itself(qll):
    """dA[m][k] = sigma'(z_k) z_k: two roundings to bf16 (dz and dA; the weight is
    exact) and fp32 arithmetic, on both sides of zero."""
    z = torch.cat([torch.linspace(-24, 24, 97), torch.linspace(-3, 3, 31)]).to(BF).cuda()
    x, w = diagonal(z)
    zd = z.to(D)
    want = torch.sigmoid(zd) * torch.sigmoid(-zd) * zd
    dA, _, db = qll.gemm_bf16_epilogue_backward(x, w, torch.ones(70, z.numel(), dtype=BF, device="cuda"),
                                                bias=torch.zeros_like(z), act="sigmoid")
    for m in (0, 69):
        check(dA[m], (want, 2.02 * 2.0 ** -8 * want.abs()), m)
    want = 70 * torch.sigmoid(zd) * torch.sigmoid(-zd)
    # each term: the exponent's |z| u, a few roundings; 70 terms summed
    check(db, (want, (2 * zd.abs() + 16 + 70) * 2.0 ** -24 * want), "dbias")


# --------------------------------------------------------------------------
# paths that only some sizes take
# --------------------------------------------------------------------------

@pytest.mark.parametrize("M,K", [(300, 8208), (700, 8200), (300, 16384), (140, 32768)])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_norm_backward_of_many_long_rows(qll, stream, M, K):
    """Past 8192 columns, with more rows than strips of the vector gradients."""
    g = gen(M + K)
    st = BF if stream == "bf16" else F32
    y, r = rnd(g, M, K), rnd(g, M, K, std=2.0, dtype=st)
    dn, dr = rnd(g, M, K, std=0.1), rnd(g, M, K, std=0.1, dtype=st)
    w2, w1, gt = (rnd(g, K, std=0.2) + 1 for _ in range(3))
    d = lambda t: None if t is None else t.to(D)
    for post, gate, block, up, al in ((w1, gt, y, dr, 0.75), (None, gt, y, None, 1.0), (None, None, None, dr, 1.0)):
        want = ref.norm_backward(d(block), d(r), d(w2), d(dn), d(up), d(post), d(gate), al, 0.5)
        got = qll.residual_norm_backward(block, r, w2, dn, up, w_post=post, gate=gate, alpha=al, beta=0.5)
        for name, t in zip(("dy", "dr", "dw_pre", "dw_post", "dgate"), got):
            assert (t is None) == (name not in want), name
            if t is not None:
                v, e = want[name]
                check(t, (v, e + ref.rounding(v, "bf16" if t.dtype == BF else "fp32")), (name, M, K))


@pytest.mark.parametrize("M,N,K", [(130, 1160, 264), (64, 1160, 64), (65, 2056, 136), (200, 1544, 72)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_split_input_gradient_across_both_weights(qll, act, M, N, K):
    """Split-K pieces of the gated input's gradient that cross from the gate's
    weight to the up projection's, and pieces that start inside the second:
    pieces of ceil(stages / splits) stages, N / 64 stages per weight."""
    tiles, seam = -(-M // 64) * -(-K // 64), -(-N // 64)
    splits = min(256 // tiles, 2 * seam // 12, 32)
    per = -(-2 * seam // splits)
    starts = [s * per for s in range(splits)]
    assert splits > 1 and seam not in starts and any(s > seam for s in starts)
    g = gen(M + N)
    x, wg, wu, dout = rnd(g, M, K), rnd(g, N, K, std=0.05), rnd(g, N, K, std=0.05), rnd(g, M, N, std=0.1)
    want = ref.gated_backward(x.to(D), wg.to(D), wu.to(D), dout.to(D), act)
    whole, dA = guarded(M, K, BF)
    got = qll.gated_bf16_backward(x, wg, wu, dout, act=act, dA=dA)
    for t, r, w, name in zip(got, want, (whole, None, None), ("dA", "dBg", "dBu")):
        check(t, r, (name, M, N, K), w)


# sizes of the 256x256 tile (forward), and of both gradients in one launch
@pytest.mark.parametrize("M,N,K", [(4100, 4360, 80), (4097, 4105, 208)])
def test_bad_rows_on_the_large_tile(qll, M, N, K):
    g = gen(M)
    x, wg, wu = rnd(g, M, K), rnd(g, N, K), rnd(g, N, K)
    for m in (0, 300, M - 1):
        bad = x.clone()
        bad[m] = NAN
        rest = torch.arange(M, device="cuda") != m
        for f in (lambda a: qll.gemm_bf16_epilogue(a, wg, act="silu"), lambda a: qll.gated_bf16(a, wg, wu)):
            a, b = f(x), f(bad)
            assert torch.equal(a[rest], b[rest]) and torch.isnan(b[m]).all()
    for n in (0, 300, N - 1):
        bad = wg.clone()
        bad[n] = NAN
        rest = torch.arange(N, device="cuda") != n
        for f in (lambda w: qll.gemm_bf16_epilogue(x, w, act="silu"), lambda w: qll.gated_bf16(x, w, wu),
                  lambda w: qll.gated_bf16(x, wu, w)):
            a, b = f(wg), f(bad)
            assert torch.equal(a[:, rest], b[:, rest]) and torch.isnan(b[:, n]).all()


# 64x64 tiles, 128x128 tiles, the 256x256 tile in one product, one launch for both
@pytest.mark.parametrize("M,N,K", [(70, 88, 72), (300, 520, 264), (1600, 1608, 1032), (4100, 4360, 72),
                                   (2000, 2304, 4360), (4100, 2056, 2056)])
def test_bad_columns_stay_in_their_gradients(qll, M, N, K):
    """dA = dz B and dB = dz^T A: a NaN in column k of an operand that is read
    along its rows changes column k of the gradient and no other, also where
    a tile reaches past the last column into the next line."""
    g = gen(M)
    x, w, dout = rnd(g, M, K), rnd(g, N, K), rnd(g, M, N)
    dA, dB, _ = qll.gemm_bf16_epilogue_backward(x, w, dout)
    for k in (0, K // 2, K - 1):
        rest = torch.arange(K, device="cuda") != k
        w2, x2 = w.clone(), x.clone()
        w2[N // 2, k] = NAN
        x2[M // 3, k] = NAN
        a, b, _ = qll.gemm_bf16_epilogue_backward(x2, w2, dout)
        assert torch.equal(a[:, rest], dA[:, rest]) and torch.isnan(a[:, k]).all()
        assert torch.equal(b[:, rest], dB[:, rest]) and torch.isnan(b[:, k]).all()
    # (the same launch: either gradient alone may run on another tile)
    for n in (0, N // 2, N - 1):
        d2 = dout.clone()
        d2[M // 2, n] = INF
        rows, cols = torch.arange(M, device="cuda") != M // 2, torch.arange(N, device="cuda") != n
        a, b, _ = qll.gemm_bf16_epilogue_backward(x, w, d2)
        assert torch.equal(a[rows], dA[rows]) and not torch.isfinite(a[M // 2]).any()
        assert torch.equal(b[cols], dB[cols]) and not torch.isfinite(b[n]).any()
