"""GPU parity of the feed-forward operators against their formulas in 64 bits
(tests/ffn_reference.py, which derives the bounds): sizes at which tiles, K
stages and Split-K end raggedly, every activation, one token to several
tiles, output types, rows that hold infinities and NaN, guard rows behind the
outputs, HIP graphs, other streams, and a whole feed-forward block."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
import ffn_reference as ref  # noqa: E402

BF, F32, D = torch.bfloat16, torch.float32, torch.float64
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]


@pytest.fixture(scope="module")
def qll():
    import quantized_linear_layer_scaled_amd as q
    q.load_library()
    q.init()
    return q


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def rnd(g, *shape, std=1.0, dtype=BF):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def quant(t):
    s = t.float().abs().amax(1, keepdim=True) / 448
    return (t.float() / s).clamp(-448, 448).to(torch.float8_e4m3fn), s[:, 0].contiguous()


def guarded(M, N, dtype):
    """[M][N] output with three rows of a fixed pattern behind it."""
    whole = torch.full((M + 3, N), 7.0, dtype=dtype, device="cuda")
    return whole, whole[:M]


def check(y, want, what, whole=None):
    r, bound = want
    d = (y.to(D) - r).abs()
    bad = ~(d <= bound + 1e-30)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, worst {float((d / (bound + 1e-30)).max()):.3g} x the bound"
    if whole is not None:
        assert (whole[y.shape[0]:] == 7.0).all(), f"{what}: rows behind the output were written"


# M: one token, decode blocks, the first tile sizes, ragged tiles; N: one
# column, less than a vector, odd, ragged tiles; K: one chunk, ragged stages
SIZES = [(1, 64, 128), (1, 1, 16), (3, 9, 48), (16, 129, 272), (17, 40, 1040),
         # two blocks of tokens: the few-row kernel and, past its rules, the tile
         (24, 4104, 272), (32, 4099, 144), (31, 2056, 13392), (32, 8200, 80), (33, 257, 528),
         (64, 520, 1056), (65, 64, 128), (65, 7, 32), (100, 333, 1040), (129, 130, 64), (200, 1000, 4112),
         (257, 264, 656), (300, 2056, 400), (1025, 1041, 144),
         # the 256x256 tile: one, two and several stages, ragged
         (4100, 4360, 80), (4097, 4105, 208), (4200, 4104, 1040)]


@pytest.mark.parametrize("M,N,K", SIZES)
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_linear(qll, kind, M, N, K):
    g = gen(M * 7 + N + K)
    x, w = rnd(g, M, K), rnd(g, N, K, std=0.05)
    b, res = rnd(g, N, std=0.5), rnd(g, M, N)
    for out, act, bias, residual in (("bf16", "none", None, res), ("fp32", ACTS[(M + N) % 6], b, None),
                                     ("bf16", ACTS[(M + K // 16) % 6], b, res), ("fp32", "none", None, None)):
        whole, o = guarded(M, N, BF if out == "bf16" else F32)
        kw = dict(bias=bias, residual=residual, act=act, out_dtype=out, out=o)
        rk = dict(bias=None if bias is None else bias.to(D), res=None if residual is None else residual.to(D),
                  act=act, out=out)
        if kind == "bf16":
            qll.gemm_bf16_epilogue(x, w, **kw)
            want = ref.linear(x.to(D), w.to(D), **rk)
        else:
            (xq, sx), (wq, sw) = quant(x), quant(w)
            qll.gemm_fp8_epilogue(xq, wq, sx, sw, **kw)
            want = ref.linear(xq.to(D), wq.to(D), sx.to(D), sw.to(D), **rk)
        check(o, want, (kind, M, N, K, out, act), whole)


@pytest.mark.parametrize("M,N,K", SIZES + [(2100, 1300, 208)])
@pytest.mark.parametrize("kind", ["bf16", "fp8"])
def test_gated(qll, kind, M, N, K):
    g = gen(M + N * 3 + K)
    x, wg, wu = rnd(g, M, K), rnd(g, N, K, std=0.05), rnd(g, N, K, std=0.05)
    for out, act in (("bf16", "silu"), ("fp32", ACTS[(M + N) % 6])):
        whole, o = guarded(M, N, BF if out == "bf16" else F32)
        if kind == "bf16":
            qll.gated_bf16(x, wg, wu, act=act, out_dtype=out, out=o)
            want = ref.gated(x.to(D), wg.to(D), wu.to(D), act=act, out=out)
        else:
            (xq, sx), (gq, sg), (uq, su) = quant(x), quant(wg), quant(wu)
            qll.gated_fp8(xq, gq, uq, sx, sg, su, act=act, out_dtype=out, out=o)
            want = ref.gated(xq.to(D), gq.to(D), uq.to(D), sx.to(D), sg.to(D), su.to(D), act, out)
        check(o, want, (kind, M, N, K, out, act), whole)


GRAD_SIZES = [(1, 64, 128), (1, 8, 8), (5, 24, 40), (64, 72, 136), (65, 136, 72), (130, 264, 520),
              (257, 520, 264), (300, 1032, 512), (1025, 264, 136), (2100, 1304, 264), (4096, 64, 64),
              # the 256x256 tile in one of the products each
              (4100, 72, 4360), (72, 4104, 4360), (4100, 4360, 72), (4100, 4360, 200)]
# both gradients in one launch
PAIR_SIZES = [(4100, 4104, 2056), (4100, 2056, 2056), (2000, 2304, 4360)]


@pytest.mark.parametrize("M,N,K", GRAD_SIZES + PAIR_SIZES)
@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
def test_linear_backward(qll, act, M, N, K):
    g = gen(M + N + K)
    x, w, b, dout = rnd(g, M, K), rnd(g, N, K, std=0.05), rnd(g, N, std=0.5), rnd(g, M, N, std=0.1)
    want = ref.linear_backward(x.to(D), w.to(D), dout.to(D), b.to(D), act)
    wA, dA = guarded(M, K, BF)
    wB, dB = guarded(N, K, BF)
    got = qll.gemm_bf16_epilogue_backward(x, w, dout, bias=b, act=act, dA=dA, dB=dB)
    for t, r, whole, name in zip(got, want, (wA, wB, None), ("dA", "dB", "dbias")):
        check(t, r, (name, act, M, N, K), whole)
    only = qll.gemm_bf16_epilogue_backward(x, w, dout, bias=b, act=act, need_input=False)
    assert only[0] is None and torch.equal(only[1], dB) and torch.equal(only[2], got[2])
    only = qll.gemm_bf16_epilogue_backward(x, w, dout, act="none", need_weight=False)
    check(only[0], ref.linear_backward(x.to(D), w.to(D), dout.to(D))[0], "dA alone")


@pytest.mark.parametrize("act", ACTS)
def test_backward_of_every_activation(qll, act):
    M, N, K = 70, 88, 64
    g = gen(5)
    x, w, wu = rnd(g, M, K), rnd(g, N, K, std=0.3), rnd(g, N, K, std=0.3)
    b, dout = rnd(g, N, std=0.5), rnd(g, M, N)
    got = qll.gemm_bf16_epilogue_backward(x, w, dout, bias=b, act=act)
    for t, r in zip(got, ref.linear_backward(x.to(D), w.to(D), dout.to(D), b.to(D), act)):
        check(t, r, act)
    got = qll.gated_bf16_backward(x, w, wu, dout, act=act)
    for t, r in zip(got, ref.gated_backward(x.to(D), w.to(D), wu.to(D), dout.to(D), act)):
        check(t, r, act)


@pytest.mark.parametrize("M,N,K", GRAD_SIZES + PAIR_SIZES)
@pytest.mark.parametrize("act", ["silu", "gelu_tanh"])
def test_gated_backward(qll, act, M, N, K):
    g = gen(M + N + K)
    x, wg, wu, dout = rnd(g, M, K), rnd(g, N, K, std=0.05), rnd(g, N, K, std=0.05), rnd(g, M, N, std=0.1)
    want = ref.gated_backward(x.to(D), wg.to(D), wu.to(D), dout.to(D), act)
    outs = [guarded(*s, BF) for s in ((M, K), (N, K), (N, K))]
    got = qll.gated_bf16_backward(x, wg, wu, dout, act=act, dA=outs[0][1], dBg=outs[1][1], dBu=outs[2][1])
    for t, r, (whole, _), name in zip(got, want, outs, ("dA", "dBg", "dBu")):
        check(t, r, (name, act, M, N, K), whole)


def test_no_tokens(qll):
    x, w = torch.empty(0, 64, dtype=BF, device="cuda"), rnd(gen(1), 24, 64)
    d = torch.empty(0, 24, dtype=BF, device="cuda")
    assert qll.gemm_bf16_epilogue(x, w).shape == (0, 24)
    assert qll.gated_bf16(x, w, w).shape == (0, 24)
    for act in ("none", "silu"):
        dA, dB, db = qll.gemm_bf16_epilogue_backward(x, w, d, bias=rnd(gen(2), 24), act=act)
        assert dA.shape == (0, 64) and (dB == 0).all() and (db == 0).all()
    dA, dg, du = qll.gated_bf16_backward(x, w, w, d)
    assert dA.shape == (0, 64) and (dg == 0).all() and (du == 0).all()
    v = rnd(gen(3), 64)
    h, n = qll.residual_norm(x, x, v)
    assert h.shape == n.shape == (0, 64)
    got = qll.residual_norm_backward(x, x, v, x, w_post=v, gate=v)
    assert all((t == 0).all() for t in got[2:])


# A token that holds NaN or infinities changes its own rows and no others,
# also where rows share a K stage with the end of the row before.
@pytest.mark.parametrize("M", [5, 70, 300])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_bad_token_stays_in_its_row(qll, M, bad):
    N, K = 200, 80
    g = gen(M)
    x, wg, wu, dout = rnd(g, M, K), rnd(g, N, K), rnd(g, N, K), rnd(g, M, N)
    rest = [m for m in range(M) if m != M // 2]
    clean = x.clone()
    x[M // 2] = bad
    xq, sx = quant(clean)
    wq, sw = quant(wg)
    xb = xq.clone()
    xb.view(torch.uint8)[M // 2] = 0x7F
    for f in (lambda a: qll.gemm_bf16_epilogue(a, wg, act="silu"), lambda a: qll.gated_bf16(a, wg, wu),
              lambda a: qll.gated_bf16_backward(a, wg, wu, dout, need_weight=False)[0],
              lambda a: qll.gemm_bf16_epilogue_backward(a, wg, dout, act="gelu", need_weight=False)[0]):
        assert torch.equal(f(x)[rest], f(clean)[rest])
    assert torch.isnan(qll.gemm_bf16_epilogue(x, wg)[M // 2]).any()
    f = lambda a: qll.gemm_fp8_epilogue(a, wq, sx, sw)
    assert torch.equal(f(xb)[rest], f(xq)[rest]) and torch.isnan(f(xb)[M // 2]).all()
    d = dout.clone()
    d[M // 2] = bad
    f = lambda t: qll.gemm_bf16_epilogue_backward(clean, wg, t, need_weight=False)[0]
    assert torch.equal(f(d)[rest], f(dout)[rest])


# A weight row that holds NaN changes its own output column and no others.
@pytest.mark.parametrize("M", [5, 70, 300])
def test_a_bad_weight_row_stays_in_its_column(qll, M):
    N, K = 203, 72
    g = gen(M)
    x, wg = rnd(g, M, K), rnd(g, N, K)
    bad = wg.clone()
    bad[N - 1] = float("nan")
    a, b = qll.gemm_bf16_epilogue(x, wg), qll.gemm_bf16_epilogue(x, bad)
    assert torch.equal(a[:, :N - 1], b[:, :N - 1]) and torch.isnan(b[:, N - 1]).all()
    a, b = qll.gated_bf16(x, wg, wg), qll.gated_bf16(x, wg, bad)
    assert torch.equal(a[:, :N - 1], b[:, :N - 1]) and torch.isnan(b[:, N - 1]).all()


@pytest.mark.parametrize("M", [4, 300])
def test_large_preactivations(qll, M):
    """Activations and slopes at their ends: no NaN from overflow inside."""
    K, N = 16, 48
    g = gen(9)
    x = rnd(g, M, K, std=300.0)
    w = rnd(g, N, K, std=300.0)
    for act in ACTS:
        want = ref.linear(x.to(D), w.to(D), act=act)
        check(qll.gemm_bf16_epilogue(x, w, act=act), want, act)
        if M > 64:
            d = rnd(g, M, N)
            got = qll.gemm_bf16_epilogue_backward(x, w, d, act=act)
            for t, r in zip(got, ref.linear_backward(x.to(D), w.to(D), d.to(D), None, act)):
                if t is not None:
                    check(t, r, act)


def test_residual_in_place(qll):
    g = gen(4)
    for M, N, K in ((3, 130, 256), (150, 264, 4096), (400, 520, 128)):
        x, w, res = rnd(g, M, K), rnd(g, N, K, std=0.05), rnd(g, M, N)
        want = qll.gemm_bf16_epilogue(x, w, residual=res)
        got = qll.gemm_bf16_epilogue(x, w, residual=res, out=res)
        assert got is res and torch.equal(got, want)


def test_offsets_past_32_bits(qll):
    """An output of more than 2^31 elements, and gradients whose operand spans
    more than 2^31 bytes along the contraction; checked on rows at both ends."""
    g = gen(8)
    M, N, K = 66000, 33000, 16
    x, w = rnd(g, M, K), rnd(g, N, K)
    out = qll.gemm_bf16_epilogue(x, w, act="silu")
    rows = torch.tensor([0, 1, 65063, 65075, 65999], device="cuda")
    check(out[rows], ref.linear(x[rows].to(D), w.to(D), act="silu"), "out")
    del out
    M, N, K = 66000, 17000, 2568
    x, w, d = rnd(g, M, K), rnd(g, N, K, std=0.05), rnd(g, M, N, std=0.1)
    dA, dB, _ = qll.gemm_bf16_epilogue_backward(x, w, d)
    cols = torch.tensor([0, 8191, 16383, 16999], device="cuda")
    want = d[:, cols].to(D).t() @ x.to(D)
    mag = d[:, cols].to(D).abs().t() @ x.to(D).abs()
    check(dB[cols], (want, ref.gamma(M) * mag + ref.rounding(want, "bf16")), "dB")
    rows = torch.tensor([0, 33000, 63161, 63170, 65999], device="cuda")
    want, mag = d[rows].to(D) @ w.to(D), d[rows].to(D).abs() @ w.to(D).abs()
    check(dA[rows], (want, ref.gamma(N) * mag + ref.rounding(want, "bf16")), "dA")


NORM_SIZES = [(1, 16), (1, 4096), (3, 512), (2, 528), (7, 2048), (5, 2064), (3, 4112), (130, 8192),
              (4, 8208), (2, 16384), (3, 32768), (1030, 1040), (1030, 4096), (1025, 6160)]


def test_more_columns_than_one_launch_of_few_row_workgroups(qll):
    """One token and so many columns that 512 threads for each 8 of them would
    be 2^32 threads."""
    g = gen(81)
    N, K = (1 << 26) + 72, 16
    codes = [torch.randint(0, 120, (N, K), generator=g, device="cuda", dtype=torch.uint8)
             .view(torch.float8_e4m3fn) for _ in range(2)]
    x = torch.randint(0, 120, (1, K), generator=g, device="cuda",
                      dtype=torch.uint8).view(torch.float8_e4m3fn)
    sa = torch.full((1,), 1e-3, device="cuda")
    sb = torch.rand(N, generator=g, device="cuda") * 1e-3
    cols = torch.cat([torch.arange(64, device="cuda"), torch.arange(N - 200, N, device="cuda"),
                      torch.randint(0, N, (2000,), generator=g, device="cuda")])
    w = [c.view(torch.uint8)[cols].view(torch.float8_e4m3fn).to(D) for c in codes]
    y = qll.gemm_fp8_epilogue(x, codes[0], sa, sb)
    check(y[:, cols], ref.linear(x.to(D), w[0], sa.to(D), sb[cols].to(D)), "linear")
    y = qll.gated_fp8(x, codes[0], codes[1], sa, sb, sb)
    check(y[:, cols], ref.gated(x.to(D), w[0], w[1], sa.to(D), sb[cols].to(D),
                                sb[cols].to(D)), "gated")


@pytest.mark.parametrize("K,backward", [(4104, False), (8200, True)])
def test_more_long_rows_than_workgroups(qll, K, backward):
    """More rows than a launch of one workgroup per row may hold: each row's
    results are those of a call on few rows, bit for bit."""
    g = gen(82)
    M, P = (1 << 21) + 1100, 1031
    base, w = rnd(g, P, K), rnd(g, K)
    x = torch.empty((M, K), dtype=BF, device="cuda")
    for i in range(0, M, P):
        x[i:i + P] = base[:min(P, M - i)]
    if backward:
        want = qll.residual_norm_backward(None, base, w, base)[1]
        got = qll.residual_norm_backward(None, x, w, x)[1]
    else:
        want, got = qll.residual_norm(None, base, w)[1], qll.residual_norm(None, x, w)[1]
    bad = torch.zeros((), dtype=torch.bool, device="cuda")
    for i in range(0, M, P):
        bad |= (got[i:i + P] != want[:min(P, M - i)]).any()
    assert not bool(bad)
    del x, got
    torch.cuda.empty_cache()


@pytest.mark.parametrize("M,K", NORM_SIZES)
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_residual_norm(qll, stream, M, K):
    g = gen(M + K)
    st = BF if stream == "bf16" else F32
    y, r = rnd(g, M, K), rnd(g, M, K, std=2.0, dtype=st)
    w2, w1, gt = (rnd(g, K, std=0.2) + 1 for _ in range(3))
    if M > 2:
        y[1] = 0  # a row whose norm is eps alone
        r[2] = 0
        y[2] = 0  # an empty row: zero codes, scale 0
    d = lambda t: None if t is None else t.to(D)
    for post, gate, block, al in ((w1, gt, y, 0.75), (None, gt, y, 1.0), (w1, None, y, 1.0),
                                  (None, None, y, 0.5), (None, None, None, 1.0)):
        want = ref.norm_forward(d(block), d(r), d(w2), d(post), d(gate), al, 0.5)
        wh, ho = guarded(M, K, st)
        wn, no = guarded(M, K, BF)
        kw = dict(w_post=post, gate=gate, alpha=al, beta=0.5)
        h, n = qll.residual_norm(block, r, w2, r_out=None if block is None else ho, n_out=no, **kw)
        if block is None:
            assert h is r
        else:
            check(h, (want["h"], want["eh"] + ref.rounding(want["h"], stream)), ("h", M, K), wh)
        check(n, (want["n"], want["en"] + ref.rounding(want["n"], "bf16")), ("n", M, K), wn)
        h2, q, s = qll.residual_norm(block, r, w2, quantize=True, **kw)
        assert block is None or torch.equal(h2, h)
        amax = want["n"].abs().amax(1, keepdim=True)
        top = want["en"].amax(1, keepdim=True)
        check(s, (amax / 448, top / 448 + 2.0 ** -22 * amax / 448), ("scale", M, K))
        # a code is off by half a step of its value (2^-4, or 2^-10 below the
        # normal range), of the fp32 n over the scale that was stored
        v = want["n"] / s.to(D).clamp_min(1e-300)
        ev = want["en"] / s.to(D).clamp_min(1e-300) + 2.0 ** -22 * v.abs()
        v = torch.where(s == 0, torch.zeros_like(v), v)
        ev = torch.where(s == 0, torch.zeros_like(v), ev)
        check(q, (v, ev + torch.maximum(v.abs() * 2.0 ** -4, torch.full_like(v, 2.0 ** -10))), ("codes", M, K))


@pytest.mark.parametrize("M,K", [(1, 16), (1, 4096), (3, 512), (2, 528), (7, 1024), (5, 2064), (3, 4112),
                                 (600, 1032), (1100, 512), (530, 4096), (4, 8208), (3, 16384), (2, 32768)])
@pytest.mark.parametrize("stream", ["bf16", "fp32"])
def test_residual_norm_backward(qll, stream, M, K):
    g = gen(M + K)
    st = BF if stream == "bf16" else F32
    y, r = rnd(g, M, K), rnd(g, M, K, std=2.0, dtype=st)
    dn, dr = rnd(g, M, K, std=0.1), rnd(g, M, K, std=0.1, dtype=st)
    w2, w1, gt = (rnd(g, K, std=0.2) + 1 for _ in range(3))
    d = lambda t: None if t is None else t.to(D)
    for post, gate, block, up, al in ((w1, gt, y, dr, 0.75), (None, gt, y, None, 1.0), (w1, None, y, dr, 1.0),
                                      (None, None, y, dr, 0.5), (None, None, None, dr, 1.0)):
        want = ref.norm_backward(d(block), d(r), d(w2), d(dn), d(up), d(post), d(gate), al, 0.5)
        wr, ro = guarded(M, K, st)
        got = qll.residual_norm_backward(block, r, w2, dn, up, w_post=post, gate=gate, alpha=al, beta=0.5, dr=ro)
        for name, t in zip(("dy", "dr", "dw_pre", "dw_post", "dgate"), got):
            assert (t is None) == (name not in want), name
            if t is not None:
                v, e = want[name]
                kind = "bf16" if t.dtype == BF else "fp32"
                check(t, (v, e + ref.rounding(v, kind)), (name, M, K), wr if name == "dr" else None)


def test_norm_in_place_and_bad_rows(qll):
    g = gen(6)
    for M, K in ((5, 4096), (1100, 2048)):
        y, r, w = rnd(g, M, K), rnd(g, M, K), rnd(g, K)
        h, n = qll.residual_norm(y, r, w, w_post=w)
        r2 = r.clone()
        h2, n2 = qll.residual_norm(y, r2, w, w_post=w, r_out=r2)
        assert h2 is r2 and torch.equal(h, h2) and torch.equal(n, n2)
        y[3] = float("nan")
        h3, n3 = qll.residual_norm(y, r, w, w_post=w)
        rest = [m for m in range(M) if m != 3]
        assert torch.equal(h[rest], h3[rest]) and torch.equal(n[rest], n3[rest]) and torch.isnan(n3[3]).all()


# --------------------------------------------------------------------------
# together, as a model runs them
# --------------------------------------------------------------------------

def block_forward(qll, s):
    """A feed-forward block behind an attention block's output y: the norms,
    the gated projections, the down projection onto the stream."""
    h, n = qll.residual_norm(s["y"], s["r"], s["w2"], w_post=s["w1"], gate=s["gt"], beta=0.5)
    a = qll.gated_bf16(n, s["wg"], s["wu"])
    return h, n, a, qll.gemm_bf16_epilogue(a, s["wd"], bias=s["b"], residual=h)


def block_backward(qll, s, h, n, a, dout):
    da, dwd, db = qll.gemm_bf16_epilogue_backward(a, s["wd"], dout, bias=s["b"])
    dn, dwg, dwu = qll.gated_bf16_backward(n, s["wg"], s["wu"], da)
    dy, dr, dw2, dw1, dgt = qll.residual_norm_backward(s["y"], s["r"], s["w2"], dn, dout, w_post=s["w1"],
                                                       gate=s["gt"], beta=0.5)
    return dict(y=dy, r=dr, w2=dw2, w1=dw1, gt=dgt, wg=dwg, wu=dwu, wd=dwd, b=db)


def block_state(M, H, F, seed):
    g = gen(seed)
    s = dict(y=rnd(g, M, H), r=rnd(g, M, H), wg=rnd(g, F, H, std=0.05), wu=rnd(g, F, H, std=0.05),
             wd=rnd(g, H, F, std=0.05), b=rnd(g, H, std=0.1))
    for k in ("w1", "w2", "gt"):
        s[k] = rnd(g, H, std=0.2) + 1
    return s


def block_autograd(s, dout):
    """The same block in 64 bits, its gradients by torch's autograd."""
    p = {k: v.to(D).requires_grad_() for k, v in s.items()}
    rms = lambda t: t / torch.sqrt((t * t).mean(1, keepdim=True) + 1e-6)
    h = p["r"] + 0.5 * p["gt"] * rms(p["y"]) * p["w1"]
    n = rms(h) * p["w2"]
    a = torch.nn.functional.silu(n @ p["wg"].t()) * (n @ p["wu"].t())
    out = a @ p["wd"].t() + p["b"] + h
    out.backward(dout.to(D))
    return out.detach(), {k: v.grad for k, v in p.items()}


@pytest.mark.parametrize("M,H,F", [(1, 256, 520), (40, 256, 520), (333, 512, 1000)])
def test_feed_forward_block(qll, M, H, F):
    """A chain of bf16 tensors: each of the at most six roundings on a path
    adds at most 2^-8 of the tensor it rounds; as errors of many terms of one
    size they come to less than 6 * 2^-8 of the result's norm."""
    s = block_state(M, H, F, M)
    dout = rnd(gen(M + 1), M, H)
    h, n, a, out = block_forward(qll, s)
    grads = block_backward(qll, s, h, n, a, dout)
    want, wg = block_autograd(s, dout)
    off = lambda t, r: float((t.to(D) - r).norm() / r.norm())
    assert off(out, want) <= 6 * 2.0 ** -8
    for k, r in wg.items():
        assert off(grads[k], r) <= 6 * 2.0 ** -8, k


def test_fp8_block(qll):
    """The serving form: norms with codes out, FP8 projections, the quantizer
    between them; held to the same operators' formulas stage by stage."""
    for M in (1, 20, 200):
        g = gen(M)
        H, F = 256, 528
        s = block_state(M, H, F, M)
        (gq, sg), (uq, su), (dq, sd) = quant(s["wg"]), quant(s["wu"]), quant(s["wd"])
        h, q, sc = qll.residual_norm(s["y"], s["r"], s["w2"], w_post=s["w1"], gate=s["gt"], quantize=True)
        a = qll.gated_fp8(q, gq, uq, sc, sg, su)
        aq, sa = qll.quantize_per_token_fp8(a)
        out = qll.gemm_fp8_epilogue(aq, dq, sa, sd, residual=h)
        scd, sad = sc[:, 0].to(D), sa[:, 0].to(D)
        check(a, ref.gated(q.to(D), gq.to(D), uq.to(D), scd, sg.to(D), su.to(D)), M)
        check(out, ref.linear(aq.to(D), dq.to(D), sad, sd.to(D), res=h.to(D)), M)


def test_train_step_in_a_graph(qll):
    """Forward and backward captured; replays after other work on the same
    memory, with eager runs of the same leaves between, give the eager bits."""
    s = block_state(150, 256, 520, 3)
    dout = rnd(gen(4), 150, 256)

    def step():
        h, n, a, out = block_forward(qll, s)
        return [out] + list(block_backward(qll, s, h, n, a, dout).values())

    want = [t.clone() for t in step()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step()
    for _ in range(3):
        for t in outs:
            t.fill_(3.0)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(step(), want))


def test_serving_calls_in_a_graph(qll):
    """FP8 serving calls of several kernels, Split-K among them, captured with
    outputs and workspace of the caller's; replays after both were overwritten
    give the eager bits."""
    H, F = 256, 16384
    s = block_state(80, H, H, 7)
    g = gen(8)
    (gq, sg), (uq, su) = quant(rnd(g, F, H, std=0.05)), quant(rnd(g, F, H, std=0.05))
    dq, sd = quant(rnd(g, H, F, std=0.05))
    L = qll.load_library()
    for M in (1, 16, 80):
        y, r = s["y"][:M].contiguous(), s["r"][:M].contiguous()
        n = torch.empty(M, H, dtype=torch.float8_e4m3fn, device="cuda")
        sc, h = torch.empty(M, 1, device="cuda"), torch.empty_like(r)
        a, out = torch.empty(M, F, dtype=BF, device="cuda"), torch.empty(M, H, dtype=F32, device="cuda")
        aq, sa = torch.empty(M, F, dtype=torch.float8_e4m3fn, device="cuda"), torch.empty(M, 1, device="cuda")
        need = L.qll_epilogue_workspace_bytes(1, M, H, F)
        assert (need > 0) == (M == 80)
        ws = torch.empty(max(need, 16), dtype=torch.uint8, device="cuda")

        def step():
            qll.residual_norm(y, r, s["w2"], w_post=s["w1"], quantize=True, r_out=h, n_out=n, scales=sc)
            qll.gated_fp8(n, gq, uq, sc, sg, su, out=a)
            qll.quantize_per_token_fp8(a, q=aq, scales=sa)
            qll.gemm_fp8_epilogue(aq, dq, sa, sd, residual=h, act="gelu", out_dtype="fp32", out=out, workspace=ws)

        step()
        want = [t.clone() for t in (h, a, out)]
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        for _ in range(3):
            for t in (h, a, out):
                t.fill_(3.0)
            ws.fill_(0x5A)
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(t, w) for t, w in zip((h, a, out), want))


def test_repeatable_and_on_other_streams(qll):
    s = block_state(700, 512, 1032, 5)
    dout = rnd(gen(6), 700, 512)

    def step(**kw):
        da, dwd, db = qll.gemm_bf16_epilogue_backward(s["a"], s["wd"], dout, bias=s["b"], act="gelu", **kw)
        return [da, dwd, db, *qll.gated_bf16_backward(s["y"], s["wg"], s["wu"], da, **kw),
                *qll.residual_norm_backward(s["y"], s["r"], s["w2"], dout, w_post=s["w1"], gate=s["gt"], **kw)]

    s["a"] = qll.gated_bf16(s["y"], s["wg"], s["wu"])
    want = step()
    torch.cuda.synchronize()
    st = [torch.cuda.Stream() for _ in range(2)]
    got = [step(stream=x) for x in st for _ in range(2)]
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(g, want))


def test_refusals(qll):
    g = gen(1)
    x, w, b = rnd(g, 4, 64), rnd(g, 24, 64), rnd(g, 24)
    with pytest.raises(ValueError):
        qll.gemm_bf16_epilogue(x, w, act="tanh")
    with pytest.raises(ValueError):
        qll.gemm_bf16_epilogue(x.t().contiguous().t(), w)
    with pytest.raises(ValueError):
        qll.gemm_bf16_epilogue(x, rnd(g, 24, 32))
    with pytest.raises(ValueError):
        qll.gemm_bf16_epilogue(x, w, bias=b.float())
    with pytest.raises(ValueError):
        qll.gemm_bf16_epilogue(x, w, residual=rnd(g, 4, 23))
    with pytest.raises(ValueError):
        qll.gemm_bf16_epilogue(x, w, out_dtype="int32")
    with pytest.raises(ValueError):
        qll.gemm_bf16_epilogue(x.cpu(), w)
    with pytest.raises(qll.QllError):
        qll.gemm_bf16_epilogue(x[:, :60].contiguous(), w[:, :60].contiguous())
    with pytest.raises(qll.QllError):
        qll.gemm_bf16_epilogue_backward(x, rnd(g, 23, 64), rnd(g, 4, 23))
    with pytest.raises(ValueError):
        qll.gemm_bf16_epilogue_backward(x, w, rnd(g, 4, 24), need_input=False, need_weight=False)
    with pytest.raises(qll.QllError) as e:
        qll.gated_bf16_backward(x, w, w, rnd(g, 4, 24), workspace=torch.empty(16, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 4
    with pytest.raises(ValueError):
        qll.gated_bf16(x, w, rnd(g, 16, 64))
    for bad in (lambda: qll.gemm_bf16_epilogue(None, w), lambda: qll.gemm_bf16_epilogue(x, None),
                lambda: qll.gated_bf16(x, w, None), lambda: qll.gated_bf16_backward(x, w, w, None),
                lambda: qll.gemm_fp8_epilogue(*quant(x)[:1], *quant(w)[:1], None, quant(w)[1]),
                lambda: qll.residual_norm(x, None, b), lambda: qll.residual_norm(x, x, None),
                lambda: qll.residual_norm_backward(x, x, rnd(g, 64), None)):
        with pytest.raises(TypeError):
            bad()
    with pytest.raises(ValueError):
        qll.residual_norm(None, x, rnd(g, 64), gate=rnd(g, 64))
    with pytest.raises(ValueError):
        qll.residual_norm(x, x.half(), rnd(g, 64))
    with pytest.raises(qll.QllError):
        qll.residual_norm(rnd(g, 2, 40), rnd(g, 2, 40), rnd(g, 40), quantize=True)
