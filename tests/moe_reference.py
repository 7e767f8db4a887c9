"""The expert operators and the sampler in 64 bits, straight from their
definitions, and the error bounds of the GPU tests.

Bounds (u = 2^-24, the fp32 rounding):
  * an exponential's argument x - m is rounded once (|x - m| u of the value),
    the exponential, the reciprocal and each sum or product that follows add a
    few u; a softmax's sum has at most 16 + 6 additions one after the other
    (experts of a lane, then lanes), a renormalising one 6: a weight is off by
    at most (2 D + 40) u of itself, D the largest |x - m| of the row (a
    sigmoid's argument is exact, so D is 0 there);
  * a gradient p (dp - <dp, p>) is off by that much of p (|dp| + <|dp|, p>),
    twice (both factors carry it), and by its own rounding;
  * a combined row is a sum of topk products and the residual, each addition
    off by u of the magnitudes so far: (topk + 2) u of their sum;
  * a dot product over K: a lane adds K / 64 products one after the other (and
    the products are rounded), 6 additions join the lanes: (K / 64 + 16) u of
    the sum of magnitudes.
A stored value is rounded once more: 2^-8 of itself in bf16, u in fp32.
"""
import math

import torch

D = torch.float64
U = 2.0 ** -24


def half_step(dtype):
    return 2.0 ** -8 if dtype == torch.bfloat16 else U


# --------------------------------------------------------------------------
# routing
# --------------------------------------------------------------------------

def scores(x, score):
    if score == "sigmoid":
        return torch.sigmoid(x)
    m = x.amax(1, keepdim=True)
    e = torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(x), torch.exp(x - m))
    return e / e.sum(1, keepdim=True).clamp_min(1e-300)


def route(logits, topk, score="softmax", bias=None, groups=1, topk_groups=None, group_best=2,
          renormalize=True, scale=1.0):
    """(ids, weights, bound): expert by expert, in Python."""
    x = logits.to(D).cpu()
    T, E = x.shape
    p = scores(x, score)
    c = p + bias.to(D).cpu() if bias is not None else p
    value = c if bias is not None else x
    size = E // groups
    ids = torch.zeros(T, topk, dtype=torch.int32)

    def rank(v):
        return -math.inf if math.isnan(v) else v

    for t in range(T):
        allowed = range(E)
        if topk_groups is not None and topk_groups < groups:
            of = []
            for g in range(groups):
                best = sorted((rank(v) for v in c[t, g * size:(g + 1) * size].tolist()), reverse=True)
                of.append(sum(best[:group_best]))
            kept = sorted(range(groups), key=lambda g: (-rank(of[g]), g))[:topk_groups]
            allowed = [e for e in range(E) if e // size in kept]
        row = value[t].tolist()
        ids[t] = torch.tensor(sorted(allowed, key=lambda e: (-rank(row[e]), e))[:topk])
    w = p.gather(1, ids.long())
    far = torch.zeros(T, 1, dtype=D)
    if score == "softmax":
        far = (x.amax(1, keepdim=True) - x.gather(1, ids.long())).amax(1, keepdim=True).clamp(0, 100)
        bad = (~(x < math.inf)).any(1, keepdim=True)
        w = torch.where(bad, torch.full_like(w, math.nan), w)
    if renormalize:
        s = w.sum(1, keepdim=True)
        w = torch.where(s == 0, torch.zeros_like(w), w / s)
    w = w * scale
    return ids, w, (2 * far + 40) * U * w.abs()


def route_backward(logits, ids, dw, score="softmax", renormalize=True, scale=1.0):
    """(dlogits, bound)"""
    x, g = logits.to(D), scale * dw.to(D)
    at = ids.long()
    live = (at >= 0) & (at < x.shape[1])
    at, g = at.clamp(0, x.shape[1] - 1), torch.where(live, g, torch.zeros_like(g))
    zero = torch.zeros_like(x)
    xc = x.gather(1, at)
    if score == "softmax":
        if renormalize:
            xc = torch.where(live, xc, torch.full_like(xc, -math.inf))
            r = scores(xc, "softmax")
            far = torch.where(live, xc.amax(1, keepdim=True) - xc, torch.zeros_like(xc)).amax(1, keepdim=True)
            d = r * (g - (g * r).sum(1, keepdim=True))
            mag = r * (g.abs() + (g.abs() * r).sum(1, keepdim=True))
            dx, mag = zero.scatter_add(1, at, torch.where(live, d, torch.zeros_like(d))), zero.scatter_add(1, at, mag)
        else:
            p = scores(x, "softmax")
            far = (x.amax(1, keepdim=True) - x).amax(1, keepdim=True).clamp(max=100)
            dp, adp = zero.scatter_add(1, at, g), zero.scatter_add(1, at, g.abs())
            dx = p * (dp - (dp * p).sum(1, keepdim=True))
            mag = p * (adp + (adp * p).sum(1, keepdim=True))
        bound = 2 * (2 * far + 40) * U * mag
    else:
        s = torch.where(live, torch.sigmoid(xc), torch.zeros_like(xc))
        slope = torch.sigmoid(xc) * torch.sigmoid(-xc)
        mag = g.abs()
        if renormalize:
            z = s.sum(1, keepdim=True).clamp_min(1e-300)
            mag = (g.abs() + (g.abs() * s / z).sum(1, keepdim=True)) / z
            g = (g - (g * s / z).sum(1, keepdim=True)) / z
        g, mag = torch.where(live, g * slope, torch.zeros_like(g)), torch.where(live, mag * slope, torch.zeros_like(g))
        dx, bound = zero.scatter_add(1, at, g), 80 * U * zero.scatter_add(1, at, mag)
    return dx, bound + half_step(logits.dtype) * dx.abs()


def sort(ids, E):
    """(offsets, rows, places), choice by choice."""
    T, k = ids.shape
    flat = ids.reshape(-1).tolist()
    of = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if 0 <= e < E:
            of[e].append(i)
    offsets, rows, places = [0], [], [-1] * len(flat)
    for entries in of:
        for i in entries:
            places[i] = len(rows)
            rows.append(i // k)
        offsets.append(len(rows))
    rows += [-1] * (len(flat) - len(rows))
    i32 = torch.int32
    return torch.tensor(offsets, dtype=i32), torch.tensor(rows, dtype=i32), torch.tensor(places, dtype=i32).view(T, k)


# --------------------------------------------------------------------------
# combination
# --------------------------------------------------------------------------

def combine(y, places, weights=None, residual=None, dtype=torch.bfloat16):
    """(out, bound)"""
    R = y.shape[0]
    y, at = y.to(D), places.long()
    live = ((at >= 0) & (at < R))[:, :, None]
    w = torch.ones(places.shape, dtype=D, device=y.device) if weights is None else weights.to(D)
    if R == 0:
        terms = torch.zeros(*places.shape, y.shape[1], dtype=D, device=y.device)
    else:
        terms = torch.where(live, w[:, :, None] * y[at.clamp(0, R - 1)], torch.zeros((), dtype=D, device=y.device))
    out, mag = terms.sum(1), terms.abs().sum(1)
    if residual is not None:
        out, mag = out + residual.to(D), mag + residual.to(D).abs()
    return out, (places.shape[1] + 2) * U * mag + half_step(dtype) * out.abs()


def combine_backward(y, places, weights, dout):
    """(dy, bound, dweights, bound); dy is 0 where no place is."""
    R, K = y.shape
    y, g = y.to(D), dout.to(D)
    w = torch.ones(places.shape, dtype=D, device=y.device) if weights is None else weights.to(D)
    dy = torch.zeros(R, K, dtype=D, device=y.device)
    dw, mag = torch.zeros_like(w), torch.zeros_like(w)
    for j in range(places.shape[1]):
        at = places[:, j].long()
        live = (at >= 0) & (at < R)
        dy[at[live]] = w[live, j, None] * g[live]
        terms = g[live] * y[at[live]]
        dw[live, j], mag[live, j] = terms.sum(1), terms.abs().sum(1)
    return dy, (2.0 ** -8 + U) * dy.abs(), dw, (K / 64 + 16) * U * mag


# --------------------------------------------------------------------------
# sampling
# --------------------------------------------------------------------------

def sample_row(x, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, its share of the kept weight) of one row of logits."""
    x = x.to(D)
    x = torch.where(torch.isnan(x), torch.full_like(x, -math.inf), x)
    m = float(x.max())
    if m == -math.inf:
        return -1, 0.0
    xs, order = torch.sort(x, descending=True, stable=True)
    if not temperature > 0:
        return int(order[0]), 1.0
    if m == math.inf:
        w = (xs == math.inf).to(D)
    else:
        w = torch.where(xs == m, torch.ones_like(xs), torch.exp((xs - m) / temperature))
        w = torch.where(xs == -math.inf, torch.zeros_like(xs), w)  # (-inf / inf is no number)
    n = len(x)
    if 0 < top_k < n:
        n = top_k
    if top_p < 1:
        c = torch.cumsum(w[:n], 0)
        before = torch.cat([c.new_zeros(1), c[:-1]])
        n = max(1, int((before < top_p * c[-1]).sum()))
    if min_p > 0:
        n = max(1, int((w[:n] >= min_p).sum()))
    c = torch.cumsum(w[:n], 0)
    i = min(int((c <= (u if u > 0 else 0.0) * c[-1]).sum()), int((w[:n] > 0).sum()) - 1)
    return int(order[i]), float(w[i] / c[-1])
