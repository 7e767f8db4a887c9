"""CPU checks of the 64-bit formulas behind the feed-forward tests: every
gradient against central differences of its forward formula, the activations
against torch's own."""
import pytest

torch = pytest.importorskip("torch")
import ffn_reference as ref  # noqa: E402

D = torch.float64
ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"]


def rnd(*shape, seed=0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g, dtype=D)


def differences(f, x, step=1e-5):
    out = torch.zeros_like(x)
    flat, o = x.view(-1), out.view(-1)
    for i in range(flat.numel()):
        keep = flat[i].item()
        flat[i] = keep + step
        up = f().item()
        flat[i] = keep - step
        o[i] = (up - f().item()) / (2 * step)
        flat[i] = keep
    return out


@pytest.mark.parametrize("act", ACTS)
def test_activation_and_slope(act):
    z = torch.linspace(-6.03, 6.01, 401, dtype=D)
    v, s = ref.value_slope(z, act)
    want = {"none": lambda t: t, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
            "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh"),
            "silu": torch.nn.functional.silu, "sigmoid": torch.sigmoid}[act](z)
    assert torch.allclose(v, want, rtol=1e-12, atol=1e-12)
    h = 1e-5
    d = (ref.value_slope(z + h, act)[0] - ref.value_slope(z - h, act)[0]) / (2 * h)
    assert torch.allclose(s, d, atol=1e-8)
    assert s.abs().max() <= ref.MAX_SLOPE
    if act != "relu":
        curve = (ref.value_slope(z + h, act)[1] - ref.value_slope(z - h, act)[1]) / (2 * h)
        assert curve.abs().max() <= ref.MAX_CURVE


# The gradients of the products: the reference rounds dz to bf16 as the kernels
# do, so the differences hold it to that rounding (2^-8 of each term).
@pytest.mark.parametrize("act", ACTS)
def test_linear_gradients_against_differences(act):
    x, w, b, dout = rnd(5, 8, seed=1), rnd(6, 8, seed=2), rnd(6, seed=3), rnd(5, 6, seed=4)
    got = ref.linear_backward(x, w, dout, b, act)
    f = lambda: (ref.value_slope(x @ w.t() + b, act)[0] * dout).sum()
    _, s = ref.value_slope(x @ w.t() + b, act)
    dz = (dout * s).abs()
    for (g, _), t, mag in zip(got, (x, w, b), (dz @ w.abs(), dz.t() @ x.abs(), dz.sum(0))):
        assert ((g - differences(f, t)).abs() <= 2.0 ** -8 * mag + 1e-7).all()


@pytest.mark.parametrize("act", ACTS)
def test_gated_gradients_against_differences(act):
    x, wg, wu, dout = rnd(5, 8, seed=1), rnd(6, 8, seed=2), rnd(6, 8, seed=3), rnd(5, 6, seed=4)
    got = ref.gated_backward(x, wg, wu, dout, act)
    f = lambda: (ref.value_slope(x @ wg.t(), act)[0] * (x @ wu.t()) * dout).sum()
    v, s = ref.value_slope(x @ wg.t(), act)
    dg, du = (dout * s * (x @ wu.t())).abs(), (dout * v).abs()
    mags = (dg @ wg.abs() + du @ wu.abs(), dg.t() @ x.abs(), du.t() @ x.abs())
    for (g, _), t, mag in zip(got, (x, wg, wu), mags):
        assert ((g - differences(f, t)).abs() <= 2.0 ** -8 * mag + 1e-7).all()


@pytest.mark.parametrize("post,gate,block", [(True, True, True), (True, False, True),
                                             (False, True, True), (False, False, True),
                                             (False, False, False)])
def test_norm_gradients_against_differences(post, gate, block):
    M, K = 4, 8
    y = rnd(M, K, seed=1) if block else None
    r, w2 = rnd(M, K, seed=2), 1 + 0.2 * rnd(K, seed=3)
    w1 = 1 + 0.2 * rnd(K, seed=4) if post else None
    g = 0.5 + 0.2 * rnd(K, seed=5) if gate else None
    dn, dr = rnd(M, K, seed=6), rnd(M, K, seed=7)
    al, be = (0.9, 0.5) if block else (1.0, 1.0)

    def f():
        o = ref.norm_forward(y, r, w2, w1, g, al, be, 1e-3)
        return (o["n"] * dn).sum() + (o["h"] * dr).sum()

    got = ref.norm_backward(y, r, w2, dn, dr, w1, g, al, be, 1e-3)
    for name, t in (("dy", y), ("dr", r), ("dw_pre", w2), ("dw_post", w1), ("dgate", g)):
        assert (t is None) == (name not in got)
        if t is not None:
            assert torch.allclose(got[name][0], differences(f, t), atol=1e-8), name
