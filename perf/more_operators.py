"""Operators around the grouped products and the vocabulary projection, in
their plain form and as the library's calls.

A mixture-of-experts layer routes each token to a few experts, runs the
experts' products over the rows sorted by expert and joins their outputs; at
the end of a decoding step a token is drawn from the vocabulary's logits:

  route      moe_route: scores, the choice of experts, their weights, and the
             rows sorted by expert; route_bwd is its backward pass
  experts    gated_fp8_grouped: act(x Wg[e]^T) * (x Wu[e]^T) of every routed
             row with its expert's weights, the tokens gathered on the way
  combine    moe_combine: the weighted sum of each token's expert outputs on
             top of the residual stream; combine_bwd is its backward pass
  sample     sample_tokens: temperature, top-k, top-p and min-p, then one token
             per row from a given random number

A case names the operator, its sizes (T tokens, E experts, k of them per
token, N and K channels; B rows of V logits) and its options.
"""
import math

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # one token's router on its way to the experts
        dict(name="route_token", op="route", T=1, E=64, k=8, score="softmax", bias=False, groups=1, keep=1, renorm=True, dtype="bf16"),
        # a prompt of odd length over many experts in groups, balanced by a bias
        dict(name="route_prompt", op="route", T=8191, E=256, k=8, score="sigmoid", bias=True, groups=8, keep=4, renorm=True, dtype="fp32"),
        # a training micro-batch's router, backward
        dict(name="route_backward", op="route_bwd", T=8192, E=64, k=8, score="softmax", renorm=False, dtype="fp32"),
        # one token's experts
        dict(name="experts_token", op="experts", T=1, E=64, k=8, N=1536, K=2048, act="silu"),
        # a batch of decoding sequences: most experts have a few rows
        dict(name="experts_batch", op="experts", T=67, E=64, k=8, N=1536, K=2048, act="silu"),
        # a prompt: hundreds of rows per expert, ragged
        dict(name="experts_prompt", op="experts", T=2048, E=64, k=8, N=1536, K=2048, act="silu"),
        # one token's expert outputs, back onto the residual stream
        dict(name="combine_token", op="combine", T=1, k=8, K=2048, residual=True),
        # a prompt of odd length over an odd width
        dict(name="combine_prompt", op="combine", T=4093, k=8, K=4104, residual=True),
        # a training micro-batch, backward
        dict(name="combine_backward", op="combine_bwd", T=4096, k=8, K=2048),
        # one sequence decoding over a large vocabulary
        dict(name="sample_token", op="sample", B=1, V=151936, ld=151936, mode="mixed", dtype="bf16"),
        # a serving batch, every sequence with options of its own
        dict(name="sample_batch", op="sample", B=256, V=151936, ld=151936, mode="mixed", dtype="fp32"),
        # an odd vocabulary in padded rows, nucleus sampling
        dict(name="sample_odd", op="sample", B=48, V=50021, ld=50048, mode="nucleus", dtype="fp32"),
    ]


def draw(rng):
    def size(lo, hi, unit=1):
        return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / unit)) * unit)

    op = rng.choice(["route", "route", "route_bwd", "experts", "experts", "combine", "combine_bwd", "sample", "sample"])
    if op in ("route", "route_bwd"):
        E = size(8, 512, 8)
        case = dict(op=op, T=size(1, 8191), E=E, k=rng.randint(1, min(16, E)), score=rng.choice(["softmax", "sigmoid"]),
                    renorm=rng.random() < 0.5, dtype=rng.choice(["bf16", "fp32"]))
        if op == "route":
            groups = rng.choice([1, 1, 4, 8])
            keep = rng.randint(max(1, -(-case["k"] * groups // E)), groups)
            case.update(bias=rng.random() < 0.5, groups=groups, keep=keep)
        return case
    if op == "experts":
        E = size(4, 64)
        return dict(op=op, T=size(1, 1024), E=E, k=rng.randint(1, min(8, E)), N=size(64, 1536), K=size(64, 2048, 16),
                    act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]))
    if op in ("combine", "combine_bwd"):
        case = dict(op=op, T=size(1, 4093), k=rng.randint(1, 8), K=size(64, 4104, 8))
        if op == "combine":
            case["residual"] = rng.random() < 0.5
        return case
    V = size(1000, 151936)
    return dict(op=op, B=size(1, 256), V=V, ld=V if rng.random() < 0.5 else (V + 63) // 64 * 64,
                mode=rng.choice(["mixed", "mixed", "nucleus", "temperature"]), dtype=rng.choice(["bf16", "fp32"]))


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV) * std


def _uniform(g, *shape):
    return torch.rand(*shape, generator=g, device=DEV)


def _type(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _e4m3(x):
    """Codes and one fp32 scale per row, as the FP8 path keeps them."""
    s = x.abs().amax(dim=-1, keepdim=True) / 448.0
    return (x / s.clamp_min(1e-30)).clamp(-448.0, 448.0).to(torch.float8_e4m3fn), s[..., 0].contiguous()


def _router_logits(g, T, E):
    """A token's own preferences on top of a load that is skewed over experts."""
    return _normal(g, T, E, std=1.5) + _normal(g, E, std=0.7)


def _sorted_rows(ids, E):
    """(offsets, rows, places) of rows sorted by expert, stable."""
    flat = ids.reshape(-1).long()
    order = torch.argsort(flat, stable=True)
    places = torch.empty_like(order)
    places[order] = torch.arange(order.numel(), device=ids.device)
    offsets = torch.zeros(E + 1, dtype=torch.long, device=ids.device)
    offsets[1:] = torch.cumsum((flat[:, None] == torch.arange(E, device=ids.device)).sum(0), 0)
    return offsets.int(), (order // ids.shape[1]).int(), places.view(ids.shape).int()


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s, bf = dict(case), torch.bfloat16
    if case["op"] == "sample":
        B, V, ld = case["B"], case["V"], case["ld"]
        x = _normal(g, B, ld, std=2.0)
        # a couple of dozen likely tokens a row, from hardly to far above the
        # rest: an open question's distribution to a nearly certain one
        likely = torch.randint(0, V // 24, (B, 24), generator=g, device=DEV) + V // 24 * torch.arange(24, device=DEV)
        x.scatter_(1, likely, 6.0 + 8.0 * _uniform(g, B, 1) + _normal(g, B, 24, std=2.5))
        s["logits"] = x.to(_type(case))[:, :V]
        s["u"] = _uniform(g, B)
        pick, a = _uniform(g, 4, B), _uniform(g, 4, B)
        if case["mode"] == "temperature":
            s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 0.6 + 0.7 * a[0], None, None, None
        elif case["mode"] == "nucleus":
            s["temperature"], s["top_k"], s["top_p"], s["min_p"] = 0.6 + 0.7 * a[0], None, 0.8 + 0.18 * a[2], None
        else:  # every row its own; zeros and ones switch an option off
            s["temperature"] = torch.where(pick[0] < 0.1, 0.0, 0.6 + 0.7 * a[0])
            s["top_k"] = torch.where(pick[1] < 0.5, 0.0, 1 + 200 * a[1] ** 2).int()
            s["top_p"] = torch.where(pick[2] < 0.3, 1.0, 0.8 + 0.18 * a[2])
            s["min_p"] = torch.where(pick[3] < 0.7, 0.0, 0.02 + 0.1 * a[3])
        return s
    T, k = case["T"], case["k"]
    if case["op"] in ("route", "route_bwd"):
        E = case["E"]
        s["logits"] = _router_logits(g, T, E).to(_type(case))
        s["b"] = _normal(g, E, std=0.05) if case.get("bias") else None
        if case["op"] == "route_bwd":
            s["ids"] = s["logits"].float().topk(k, dim=1).indices.int()
            s["dw"] = _normal(g, T, k)
        return s
    K = case["K"]
    if case["op"] == "experts":
        E, N = case["E"], case["N"]
        ids = _router_logits(g, T, E).topk(k, dim=1).indices
        s["offsets"], s["rows"], _ = _sorted_rows(ids, E)
        s["bounds"] = s["offsets"].tolist()  # the plain form walks over the experts
        x = _normal(g, T, K)
        x[:, torch.randperm(K, generator=g, device=DEV)[:max(1, K // 100)]] *= 20.0
        s["x"], s["sx"] = _e4m3(x)
        s["wg"], s["sg"] = _e4m3(_normal(g, E, N, K, std=0.02))
        s["wu"], s["su"] = _e4m3(_normal(g, E, N, K, std=0.02))
        return s
    E = 64 if k <= 8 else 128
    ids = _router_logits(g, T, E).topk(k, dim=1).indices
    s["places"] = _sorted_rows(ids, E)[2]
    s["y"] = _normal(g, T * k, K).to(bf)
    w = _uniform(g, T, k) + 0.05
    s["w"] = w / w.sum(1, keepdim=True)
    if case.get("residual"):
        s["res"] = _normal(g, T, K).to(bf)
    if case["op"] == "combine_bwd":
        s["dout"] = _normal(g, T, K, std=0.1).to(bf)
    return s


# --------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------

def _scores(x, score):
    if score == "sigmoid":
        return 1 / (1 + torch.exp(-x))
    e = torch.exp(x - x.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _plain_route(s):
    T, E, k, groups, keep = s["T"], s["E"], s["k"], s["groups"], s["keep"]
    x = s["logits"].double()  # (a choice is right or wrong)
    p = _scores(x, s["score"])
    by = p + s["b"].double() if s["bias"] else p
    order = torch.sort(by if s["bias"] else x, dim=1, descending=True, stable=True).indices
    if keep < groups:
        best = torch.sort(by.view(T, groups, E // groups), dim=2, descending=True).values[:, :, :2].sum(2)
        kept = torch.sort(best, dim=1, descending=True, stable=True).indices[:, :keep]
        out = ~(torch.div(order, E // groups, rounding_mode="floor")[:, :, None] == kept[:, None, :]).any(2)
        order = order.gather(1, torch.sort(out.int(), dim=1, stable=True).indices)
    ids = order[:, :k]
    w = p.gather(1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    offsets, rows, places = _sorted_rows(ids, E)
    return {"ids": ids.int(), "weights": w.float(), "offsets": offsets, "rows": rows, "places": places}


def _plain_route_bwd(s):
    x, ids, dw = s["logits"].float(), s["ids"].long(), s["dw"]
    p = _scores(x, s["score"])
    w = p.gather(1, ids)
    if s["renorm"]:
        total = w.sum(1, keepdim=True)
        dw = (dw - (dw * w).sum(1, keepdim=True) / total) / total
    dp = torch.zeros_like(p).scatter_add_(1, ids, dw)
    if s["score"] == "sigmoid":
        dx = dp * p * (1 - p)
    else:
        dx = p * (dp - (dp * p).sum(1, keepdim=True))
    return dx.to(s["logits"].dtype)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * (1 + torch.erf(z * math.sqrt(0.5)))
    c = math.sqrt(2 / math.pi)
    return 0.5 * z * (1 + torch.tanh(c * (z + 0.044715 * z * z * z)))


def _plain_experts(s):
    rows = s["rows"].long()
    x = s["x"].float() * s["sx"][:, None]
    out = torch.empty(rows.numel(), s["N"], dtype=torch.bfloat16, device=x.device)
    for e in range(s["E"]):
        a, b = s["bounds"][e], s["bounds"][e + 1]
        if a == b:
            continue
        xe = x[rows[a:b]]
        zg = (xe @ s["wg"][e].float().t()) * s["sg"][e]
        zu = (xe @ s["wu"][e].float().t()) * s["su"][e]
        out[a:b] = (_act(zg, s["act"]) * zu).to(torch.bfloat16)
    return out


def _plain_combine(s):
    out = (s["y"].float()[s["places"].long()] * s["w"][:, :, None]).sum(1)
    if s["residual"]:
        out = out + s["res"].float()
    return out.to(torch.bfloat16)


def _plain_combine_bwd(s):
    at, dout = s["places"].long(), s["dout"].float()
    dy = torch.empty_like(s["y"])
    dy[at] = (dout[:, None, :] * s["w"][:, :, None]).to(dy.dtype)
    return {"dy": dy, "dweights": (s["y"].float()[at] * dout[:, None, :]).sum(2)}


def _plain_sample(s):
    x = s["logits"].double()  # (long sums, and borders between tokens)
    B, V = x.shape
    t = s["temperature"].double()[:, None]
    xs, index = torch.sort(x, dim=1, descending=True, stable=True)
    greedy = t <= 0
    w = torch.exp((xs - xs[:, :1]) / torch.where(greedy, 1.0, t))
    rank = torch.arange(V, device=x.device)[None]
    first = rank == 0
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        w = w * ((k <= 0) | (rank < k))
    if s["top_p"] is not None:
        c = torch.cumsum(w, 1)
        p = s["top_p"].double()[:, None]
        w = w * (first | (p >= 1) | (c - w < p * c[:, -1:]))
    if s["min_p"] is not None:
        w = w * (first | (w >= s["min_p"].double()[:, None]))
    w = torch.where(greedy, first.double(), w)
    c = torch.cumsum(w, 1)
    at = (c <= s["u"].double()[:, None] * c[:, -1:]).sum(1, keepdim=True)
    at = torch.minimum(at, (w > 0).sum(1, keepdim=True) - 1)
    return {"tokens": index.gather(1, at)[:, 0].int(), "probs": (w.gather(1, at) / c[:, -1:])[:, 0].float()}


PLAIN = dict(route=_plain_route, route_bwd=_plain_route_bwd, experts=_plain_experts, combine=_plain_combine,
             combine_bwd=_plain_combine_bwd, sample=_plain_sample)


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------

def _own(s):
    import quantized_linear_layer_scaled_amd as qll
    op = s["op"]
    if op == "route":
        r = qll.moe_route(s["logits"], s["k"], score=s["score"], bias=s["b"], groups=s["groups"], topk_groups=s["keep"],
                          renormalize=s["renorm"], plan=True)
        return dict(zip(("ids", "weights", "offsets", "rows", "places"), r))
    if op == "route_bwd":
        return qll.moe_route_backward(s["logits"], s["ids"], s["dw"], score=s["score"], renormalize=s["renorm"])
    if op == "experts":
        return qll.gated_fp8_grouped(s["x"], s["wg"], s["wu"], s["sx"], s["sg"], s["su"], s["offsets"], rows=s["rows"],
                                     act=s["act"])
    if op == "combine":
        return qll.moe_combine(s["y"], s["places"], s["w"], residual=s.get("res"))
    if op == "combine_bwd":
        return dict(zip(("dy", "dweights"), qll.moe_combine_backward(s["y"], s["places"], s["w"], s["dout"])))
    r = qll.sample_tokens(s["logits"], s["u"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                          min_p=s["min_p"], probs=True)
    return dict(zip(("tokens", "probs"), r))


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


def work(case):
    op = case["op"]
    e = 2 if case.get("dtype") == "bf16" else 4
    if op == "sample":
        return {"bytes": case["B"] * (case["V"] * e + 28), "flops": 4 * case["B"] * case["V"]}
    T, k = case["T"], case["k"]
    if op == "route":
        E = case["E"]
        return {"bytes": T * E * e + 16 * T * k + 4 * E * (2 if case["bias"] else 1), "flops": T * E * (6 + k)}
    if op == "route_bwd":
        return {"bytes": 2 * T * case["E"] * e + 8 * T * k, "flops": 8 * T * case["E"]}
    K = case["K"]
    if op == "experts":
        E, N = case["E"], case["N"]
        met = E * (1 - (1 - k / E) ** T)  # experts that an even load reaches
        return {"bytes": int(met * (2 * N * K + 8 * N)) + T * (K + 4) + 2 * T * k * N + 4 * (E + T * k), "flops": 4 * T * k * N * K}
    if op == "combine":
        return {"bytes": 2 * T * K * (k + 1 + case["residual"]) + 8 * T * k, "flops": 2 * T * k * K}
    return {"bytes": 2 * T * K * (2 * k + 1) + 12 * T * k, "flops": 3 * T * k * K}


# --------------------------------------------------------------------------
# the definitions in 64 bits
# --------------------------------------------------------------------------

def _largest(v):
    """Index of each row's largest value, the lowest of equals."""
    at = torch.arange(v.shape[1], device=v.device).expand_as(v)
    return torch.where(v == v.max(1, keepdim=True).values, at, v.shape[1]).min(1, keepdim=True).values


def _pick(v, n):
    """The n largest of each row, one at a time."""
    v, out = v.clone(), []
    for _ in range(n):
        out.append(_largest(v))
        v.scatter_(1, out[-1], -math.inf)
    return torch.cat(out, 1)


def _exact_route(s, T):
    x = s["logits"].to(torch.float64)
    p = torch.sigmoid(x) if s["score"] == "sigmoid" else torch.softmax(x, 1)
    value = p if s["b"] is None else p + s["b"].to(torch.float64)
    size = s["E"] // s["groups"]
    if s["keep"] < s["groups"]:
        of = torch.stack([value[:, i * size:(i + 1) * size].topk(min(2, size), dim=1).values.sum(1)
                          for i in range(s["groups"])], 1)
        allowed = torch.zeros(T, s["groups"], dtype=torch.bool, device=DEV).scatter_(1, _pick(of, s["keep"]), True)
        allowed = allowed.repeat_interleave(size, 1)
    else:
        allowed = torch.ones_like(x, dtype=torch.bool)
    ids = _pick(torch.where(allowed, x if s["b"] is None else value, -math.inf), s["k"])
    w = torch.gather(p, 1, ids)
    if s["renorm"]:
        w = w / w.sum(1, keepdim=True)
    # places: the entries of lower experts, and the earlier ones of the same
    flat = ids.reshape(-1)
    count = torch.bincount(flat, minlength=s["E"])
    ends = torch.cumsum(count, 0)
    rows = torch.cat([torch.nonzero(flat == e)[:, 0] for e in range(s["E"])])
    places = torch.empty_like(flat).scatter_(0, rows, torch.arange(flat.numel(), device=DEV))
    return {"ids": ids, "weights": w, "offsets": torch.cat([ends.new_zeros(1), ends]), "rows": rows // s["k"],
            "places": places.view(T, s["k"])}


def _exact_sample(s):
    tokens, probs = [], []
    for b in range(s["B"]):
        x, t = s["logits"][b].to(torch.float64), float(s["temperature"][b])
        by_value = torch.sort(-x, stable=True).indices
        if t <= 0:
            tokens.append(by_value[0])
            probs.append(torch.ones((), dtype=torch.float64, device=DEV))
            continue
        w = torch.exp(x[by_value] / t - x.max() / t)
        n = s["V"]
        if s["top_k"] is not None and int(s["top_k"][b]) > 0:
            n = min(n, int(s["top_k"][b]))
        if s["top_p"] is not None and float(s["top_p"][b]) < 1:
            c = torch.cumsum(w[:n], 0)
            n = min(n, 1 + int(torch.searchsorted(c, float(s["top_p"][b]) * c[-1])))
        if s["min_p"] is not None:
            n = max(1, min(n, int((w[:n] >= float(s["min_p"][b])).sum())))
        c = torch.cumsum(w[:n], 0)
        at = min(n - 1, int(torch.searchsorted(c, float(s["u"][b]) * c[-1], right=True)))
        tokens.append(by_value[at])
        probs.append(w[at] / c[-1])
    return {"tokens": torch.stack(tokens), "probs": torch.stack(probs)}


def exact(case, seed):
    s = prepare(case, seed)
    d, op = torch.float64, case["op"]
    if op == "sample":
        return _exact_sample(s)
    if op == "route":
        return _exact_route(s, case["T"])
    if op == "route_bwd":
        x, ids, g = s["logits"].to(d), s["ids"].long(), s["dw"].to(d)
        if case["score"] == "sigmoid":
            q = torch.sigmoid(x)
            slope, v = (q * torch.sigmoid(-x)).gather(1, ids), q.gather(1, ids)
            if case["renorm"]:
                r = v / v.sum(1, keepdim=True)
                g = (g - (g * r).sum(1, keepdim=True)) / v.sum(1, keepdim=True)
            return torch.zeros_like(x).scatter_(1, ids, g * slope)
        if case["renorm"]:  # a softmax over the chosen ones alone
            r = torch.softmax(x.gather(1, ids), 1)
            return torch.zeros_like(x).scatter_(1, ids, r * (g - (g * r).sum(1, keepdim=True)))
        p = torch.softmax(x, 1)
        v = p.gather(1, ids)
        return (torch.zeros_like(x).scatter_(1, ids, g * v) - p * (g * v).sum(1, keepdim=True))
    if op == "experts":
        parts = []
        for e, (a, b) in enumerate(zip(s["bounds"], s["bounds"][1:])):
            xe = s["x"][s["rows"][a:b].long()].to(d) * s["sx"][s["rows"][a:b].long()].to(d)[:, None]
            zg, zu = (torch.mm(xe, (w[e].to(d) * sw[e].to(d)[:, None]).t()) for w, sw in ((s["wg"], s["sg"]), (s["wu"], s["su"])))
            if case["act"] == "silu":
                f = zg * torch.sigmoid(zg)
            elif case["act"] == "gelu":
                f = zg * torch.special.ndtr(zg)
            else:
                f = zg * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (zg + 0.044715 * zg ** 3))
            parts.append(f * zu)
        return torch.cat(parts)
    w = s["w"].to(d)
    if op == "combine":
        out = s["res"].to(d) if case["residual"] else torch.zeros(case["T"], case["K"], dtype=d, device=DEV)
        for j in range(case["k"]):
            out = out + w[:, j:j + 1] * s["y"][s["places"][:, j].long()].to(d)
        return out
    dout, dy = s["dout"].to(d), torch.zeros(s["y"].shape, dtype=d, device=DEV)
    dw = []
    for j in range(case["k"]):
        at = s["places"][:, j].long()
        dy[at] = w[:, j:j + 1] * dout
        dw.append(torch.linalg.vecdot(s["y"][at].to(d), dout))
    return {"dy": dy, "dweights": torch.stack(dw, 1)}
