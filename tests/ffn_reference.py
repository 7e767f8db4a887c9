"""The feed-forward operators in 64 bits, straight from their formulas, and
the error bounds of the GPU tests.

Bounds, per output element (u = 2^-24, the fp32 rounding):
  * a stored bf16 value is off by at most 2^-8 of itself, an fp32 one by 2^-24;
  * a matrix-core sum over K is off by at most G(K) = ((K + 4) 2^-23 + t) of
    the sum of its terms' magnitudes, t = 2^-12 for e4m3 (its steps add their
    products coarsely) and 0 for bf16;
  * an activation's own arithmetic is off by at most 2^-20 (1 + |z|): the
    exponential's argument carries |z| u, which moves e^-z by |z| u of itself
    and z s(z) by at most |z|^2 s (1 - s) u < u, and a handful of roundings
    of at most 2^-23 follow; the erf is within a few u.  Every activation
    here has a slope of at most 1.13 and a second slope of at most 1.2.
  * a value that is rounded to bf16 on its way (the pre-activation gradients)
    is rounded here too; where the kernel's fp32 value may fall on the other
    side of a rounding border its bf16 value may differ by the gap, which is
    carried through the product (`rounded`).
"""
import math

import torch

D = torch.float64
MAX_SLOPE, MAX_CURVE = 1.13, 1.2


def value_slope(z, act):
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).to(z.dtype)
    if act in ("silu", "sigmoid"):
        q = torch.sigmoid(z)
        return (q, q * (1 - q)) if act == "sigmoid" else (z * q, q + z * q * (1 - q))
    if act == "gelu":
        cdf = 0.5 * (1 + torch.erf(z / math.sqrt(2)))
        return z * cdf, cdf + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    assert act == "gelu_tanh"
    c = math.sqrt(2 / math.pi)
    t = torch.tanh(c * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * c * (1 + 3 * 0.044715 * z * z)


def gamma(K, fp8=False):
    return (K + 4) * 2.0 ** -23 + (2.0 ** -12 if fp8 else 0.0)


def product(x, w, sx=None, sw=None):
    """(x w^T, the bound of a matrix-core sum's error), scaled per row and
    column; x and w in 64 bits."""
    z, mag = x @ w.t(), x.abs() @ w.abs().t()
    if sx is not None:
        s = sx.view(-1, 1) * sw.view(1, -1)
        z, mag = z * s, mag * s.abs()
    return z, gamma(x.shape[1], sx is not None) * mag + 2.0 ** -22 * z.abs()


def rounding(ref, dtype):
    return ref.abs() * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -23)


def act_error(z, ez):
    return MAX_SLOPE * ez + 2.0 ** -20 * (1 + z.abs())


def linear(x, w, sx=None, sw=None, bias=None, res=None, act="none", out="bf16"):
    """(reference, bound)"""
    z, e = product(x, w, sx, sw)
    if bias is not None:
        z = z + bias
        e = e + 2.0 ** -23 * z.abs()
    y, _ = value_slope(z, act)
    if act != "none":
        e = act_error(z, e)
    if res is not None:
        y = y + res
        e = e + 2.0 ** -23 * y.abs()
    return y, e + rounding(y, out)


def gated(x, wg, wu, sx=None, sg=None, su=None, act="silu", out="bf16"):
    g, eg = product(x, wg, sx, sg)
    u, eu = product(x, wu, sx, su)
    f, _ = value_slope(g, act)
    ef = act_error(g, eg)
    y = f * u
    return y, f.abs() * eu + u.abs() * ef + ef * eu + 2.0 ** -23 * y.abs() + rounding(y, out)


def rounded(v, e):
    """(v as bf16, how far the bf16 value of anything within e of v may be)"""
    b = v.to(torch.float32).to(torch.bfloat16).to(D)
    lo = (v - e).to(torch.float32).to(torch.bfloat16).to(D)
    hi = (v + e).to(torch.float32).to(torch.bfloat16).to(D)
    return b, torch.maximum((hi - b).abs(), (b - lo).abs())


def gradient_products(dzs, x, ws):
    """dA and the dB of each (dz, its bound) with its weight, all bf16."""
    out = []
    dA = eA = 0
    for (dz, e), w in zip(dzs, ws):
        b, slack = rounded(dz, e)
        dA = dA + b @ w
        eA = eA + slack @ w.abs() + gamma(2 * w.shape[0]) * (b.abs() @ w.abs())
        dB = b.t() @ x
        eB = slack.t() @ x.abs() + gamma(x.shape[0]) * (b.abs().t() @ x.abs())
        out.append((dB, eB + rounding(dB, "bf16")))
    return [(dA, eA + rounding(dA, "bf16"))] + out


def linear_backward(x, w, dout, bias=None, act="none"):
    """[(dA, bound), (dB, bound), (dbias, bound)]"""
    if act == "none":
        dz, e = dout, torch.zeros_like(dout)
    else:
        z, ez = product(x, w)
        if bias is not None:
            z = z + bias
            ez = ez + 2.0 ** -23 * z.abs()
        _, s = value_slope(z, act)
        # relu's slope jumps at 0: where z may be on either side, both are right
        es = MAX_CURVE * ez + 2.0 ** -20 * (1 + z.abs())
        if act == "relu":
            es = (z.abs() <= ez).to(D)
        dz = dout * s
        e = dout.abs() * es + 2.0 ** -23 * dz.abs()
    M = x.shape[0]
    db = (dz.sum(0), e.sum(0) + (M + 16) * 2.0 ** -24 * dz.abs().sum(0))
    return gradient_products([(dz, e)], x, [w]) + [db]


def gated_backward(x, wg, wu, dout, act="silu"):
    """[(dA, bound), (dBg, bound), (dBu, bound)]"""
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    f, s = value_slope(g, act)
    ef = act_error(g, eg)
    es = (g.abs() <= eg).to(D) if act == "relu" else MAX_CURVE * eg + 2.0 ** -20 * (1 + g.abs())
    dg, du = dout * u * s, dout * f
    return gradient_products(
        [(dg, dout.abs() * (u.abs() * es + s.abs() * eu + es * eu) + 2.0 ** -22 * dg.abs()),
         (du, dout.abs() * ef + 2.0 ** -23 * du.abs())], x, [wg, wu])


# --------------------------------------------------------------------------
# residual norms
#
# A sum of K squares or products is added in fp32 by threads over at most 64
# terms each, then in a tree: off by at most (64 + 16) u < 2^-17 of the terms'
# magnitudes.  An inverse rms is then within 2^-17 of itself, and h within
# 2^-16 of (|alpha r| + |beta gate p|).
# --------------------------------------------------------------------------

def norm_forward(y, r, w_pre, w_post=None, gate=None, alpha=1.0, beta=1.0, eps=1e-6):
    """dict of h, n and their fp32 bounds eh, en (no output rounding)."""
    mag = r.abs() * abs(alpha)
    if y is None:
        h, p, iy = r, None, None
        eh = torch.zeros_like(h)
    else:
        iy = 1 / torch.sqrt((y * y).mean(1, keepdim=True) + eps) if w_post is not None else None
        p = y * iy * w_post if w_post is not None else y
        t = p * gate if gate is not None else p
        h = alpha * r + beta * t
        mag = mag + abs(beta) * t.abs()
        eh = 2.0 ** -16 * mag
    ih = 1 / torch.sqrt((h * h).mean(1, keepdim=True) + eps)
    n = h * ih * w_pre
    # ih moves with h: by at most ih^3 mean(|h| eh) / 1
    eih = 2.0 ** -17 * ih + ih ** 3 * (h.abs() * eh).mean(1, keepdim=True)
    en = (eh * ih + h.abs() * eih) * w_pre.abs() + 2.0 ** -22 * n.abs()
    return dict(h=h, n=n, eh=eh, en=en, p=p, iy=iy, ih=ih)


def norm_backward(y, r, w_pre, dn, dr_out, w_post=None, gate=None, alpha=1.0, beta=1.0, eps=1e-6):
    """dict name -> (reference, fp32 bound without the output rounding).

    Every factor is within 2^-15 of itself (h within 2^-16 of its terms, whose
    magnitude is at most `amp` times |h|'s scale; the tests keep h's terms
    from cancelling by comparing against their magnitudes), so each gradient
    is within 2^-13 of the sum of the magnitudes of its terms."""
    f = norm_forward(y, r, w_pre, w_post, gate, alpha, beta, eps)
    h, ih, iy, p = f["h"], f["ih"], f["iy"], f["p"]
    hm = abs(alpha) * r.abs()
    if y is not None:
        hm = hm + abs(beta) * (p * gate if gate is not None else p).abs()
    T = 2.0 ** -13
    u = dn * w_pre
    muh = (u * h).mean(1, keepdim=True)
    d = ih * (u - h * ih * ih * muh)
    dm = ih * (u.abs() + hm * ih * ih * (u.abs() * hm).mean(1, keepdim=True))
    if dr_out is not None:
        d, dm = d + dr_out, dm + dr_out.abs()
    rows = (r.shape[0] + 64) * 2.0 ** -24
    out = {"dr": (alpha * d, T * abs(alpha) * dm),
           "dw_pre": ((dn * h * ih).sum(0), (T + rows) * (dn.abs() * hm * ih).sum(0))}
    if y is None:
        return out
    dt, tm = beta * d, abs(beta) * dm
    if gate is not None:
        out["dgate"] = ((dt * p).sum(0), (T + rows) * (tm * p.abs()).sum(0))
        dt, tm = dt * gate, tm * gate.abs()
    if w_post is not None:
        out["dw_post"] = ((dt * y * iy).sum(0), (T + rows) * (tm * y.abs() * iy).sum(0))
        v, vm = dt * w_post, tm * w_post.abs()
        dt = iy * (v - y * iy * iy * (v * y).mean(1, keepdim=True))
        tm = iy * (vm + y.abs() * iy * iy * (vm * y.abs()).mean(1, keepdim=True))
    out["dy"] = (dt, T * tm)
    return out
