"""Measured cases of routing by scores and of products in microscaled 4-bit floating point.

Seven entry points of expert_ffn_moe_amd, in four groups:

  route       route_scored: softmax or sigmoid scores of the logits, experts chosen by
              score + bias under a group limit, weights = scale * score (renormalised or not),
              an optional capacity; an expert with a logit of -inf is out
  route_grad  route_scored_backward: dlogits from the gradient of the weights
  quantize    quantize_fp4 (rows) or quantize_fp4_weights ([E, K, N] along K) and back
              (dequantize_fp4): E2M1 codes, two to a byte, one power-of-two scale per 32
  linear      grouped_linear_fp4: y[r] = act(x[r] W[e] + b[e]) (* (x[r] U[e] + c[e]) with a
              second weight set) + residual[r] over expert-contiguous rows; W, U in 4 bits,
              x in 4 (E2M1) or 8 bits (E4M3), each with one power-of-two scale per 32 of K

Rows behind the last expert's are left as they were: y is a buffer of the state.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
QB = 32  # values per scale
INF = float("inf")
BIG = torch.finfo(F32).max


# ---------------------------------------------------------------------------- the cases
def _route(name, op, T, E, k, score, groups=1, taken=1, group_score="max", bias=False,
           renorm=True, scale=1.0, cap=0, masked=0):
    c = dict(op=op, T=T, E=E, k=k, score=score, groups=groups, taken=taken,
             group_score=group_score, bias=bias, renorm=renorm, scale=scale, cap=cap,
             masked=masked)
    return dict(c, name=name) if name else c


def _quant(name, rows, cols, E=0):  # E > 0: weights [E, cols, rows], blocks along cols
    c = dict(op="quantize", rows=rows, cols=cols, E=E)
    return dict(c, name=name) if name else c


def _linear(name, T, E, k, K, N, x="fp4", act="none", gated=False, bias=False, residual=False,
            skew="even", cap=0):
    c = dict(op="linear", T=T, E=E, k=k, K=K, N=N, x=x, act=act, gated=gated, bias=bias,
             residual=residual, skew=skew, cap=cap)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a serving loop, sigmoid scores with a balance bias and group limit
        _route("route one token", "route", 1, 256, 8, "sigmoid", 8, 4, "top2", True, scale=2.5),
        # a prefill of the same layer
        _route("route prefill", "route", 16384, 256, 8, "sigmoid", 8, 4, "top2", True, scale=2.5),
        # softmax over all experts, some of them out of service, under a capacity
        _route("route capacity odd", "route", 4099, 160, 6, "softmax", bias=True, renorm=False,
               cap=200, masked=13),
        # training: the router's gradient of a large batch, and of a small one over all experts
        _route("route_grad batch", "route_grad", 16384, 256, 8, "sigmoid", scale=2.5),
        _route("route_grad odd", "route_grad", 61, 72, 4, "softmax", renorm=False),
        # a prefill's activations to 4 bits and back
        _quant("quantize rows", 16384, 7168),
        # loading a layer of many small experts: its bf16 weights to 4 bits and back
        _quant("quantize weights", 768, 2048, E=128),
        # one token of a serving loop through its 8 experts' gate and up products: latency
        _linear("linear one token", 1, 128, 8, 2048, 768, act="silu", gated=True),
        # a decode batch on 8-bit activations: nearly every expert's weights, for a few rows
        _linear("linear decode batch", 128, 256, 8, 7168, 2048, x="fp8", act="silu", gated=True),
        # prefill of a layer with many small experts, skewed routing
        _linear("linear prefill", 4096, 128, 8, 2048, 768, act="silu", gated=True, skew="bias"),
        # a dense projection on a batch and widths that fill no tile, with everything behind it
        _linear("linear dense odd", 1003, 1, 1, 1440, 2056, x="fp8", act="gelu_tanh", bias=True,
                residual=True),
        # the largest: prefill of a wide layer's gate and up products
        _linear("linear wide", 16384, 256, 8, 7168, 2048, act="silu", gated=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["route", "route_grad", "quantize", "linear", "linear", "linear", "linear"])
    if op in ("route", "route_grad"):
        groups = rng.choice([1, 1, 4, 8])
        E = groups * _log(rng, max(1, 8 // groups), 512 // groups)
        taken = 1 if groups == 1 else rng.randint(groups // 4 + 1, groups)
        k = min(rng.choice([2, 4, 6, 8]), taken * (E // groups))
        T = _log(rng, 1, 16384)
        cap = max(1, 3 * T * k // (2 * E)) if op == "route" and rng.random() < 0.3 else 0
        return _route("", op, T, E, k, rng.choice(["softmax", "sigmoid"]), groups, taken,
                      rng.choice(["max", "top2"]), rng.random() < 0.6, rng.random() < 0.6,
                      rng.choice([1.0, 2.5]), cap, rng.choice([0, 0, E // 8]))
    if op == "quantize":
        cols = 32 * _log(rng, 2, 256)
        if rng.random() < 0.5:
            E = _log(rng, 1, 128)
            rows = 8 * _log(rng, 8, 512)
            while E * rows * cols > 1 << 28:
                E = max(1, E // 2)
            return _quant("", rows, cols, E=E)
        return _quant("", _log(rng, 1, 16384), cols)
    E = rng.choice([1, _log(rng, 2, 256), _log(rng, 2, 256)])
    k = 1 if E == 1 else min(E, rng.choice([1, 2, 4, 8]))
    K, N = 32 * _log(rng, 2, 224), 8 * _log(rng, 8, 512)
    T = _log(rng, 1, 16384)
    gated = rng.random() < 0.5
    while E * K * N > 1 << 30:
        E = max(1, E // 2)
    k = min(k, E)
    while T > 1 and 2.0 * T * k * K * N > 2e12:
        T //= 2
    skew = "even" if E == 1 else rng.choice(["even", "bias", "zipf"])
    return _linear("", T, E, k, K, N, x=rng.choice(["fp4", "fp4", "fp8"]),
                   act="silu" if gated else rng.choice(["none", "relu2", "silu", "gelu_tanh"]),
                   gated=gated, bias=rng.random() < 0.4, residual=rng.random() < 0.3, skew=skew,
                   cap=max(1, 2 * T * k // E) if skew == "zipf" else 0)


# ---------------------------------------------------------------------------- the inputs
def _layout(c, g):
    """Routing of T tokens to k of E experts: the sorted rows' tokens, offsets and counts."""
    T, E, k = c["T"], c["E"], c["k"]
    score = torch.randn(T, E, generator=g, device=DEV)
    if c["skew"] == "bias":
        score += 0.5 * torch.randn(E, generator=g, device=DEV)
    elif c["skew"] == "zipf":
        score -= 1.2 * torch.log(torch.randperm(E, generator=g, device=DEV).float() + 1)
    ids = score.topk(k, dim=1).indices.reshape(-1)
    experts, order = torch.sort(ids, stable=True)
    counts = torch.bincount(ids, minlength=E)
    first = torch.cumsum(counts, 0) - counts
    if c["cap"] > 0:  # an expert keeps its first `cap` rows
        keep = torch.arange(T * k, device=DEV) - first[experts] < c["cap"]
        experts, order = experts[keep], order[keep]
        counts = counts.clamp(max=c["cap"])
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    row_token = torch.zeros(T * k, dtype=torch.int32, device=DEV)
    row_token[:order.numel()] = (order // k).to(torch.int32)
    return row_token, offsets, counts


def _scale_exp(amax, top, bits):
    """The smallest e with amax <= top * 2^e, top = m * 2^bits, m in [0.5, 1) (0 for 0)."""
    m, x = torch.frexp(amax)
    e = x - bits + (m > top / 2.0 ** bits)
    return torch.where(amax > 0, e, torch.zeros_like(e)).clamp(-127, 127)


def _nibbles(b):
    """The E2M1 codes of scaled values: 0, 0.5, 1, 1.5, 2, 3, 4, 6, ties to the even code, and
    the sign in bit 3."""
    a = b.abs()
    q = torch.signbit(b).to(torch.uint8) << 3
    code = (a > 0.25).to(torch.uint8)
    for edge, up in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True),
                     (5.0, False)):
        code += (a >= edge) if up else (a > edge)
    return q | code


def _to_fp4(x):
    """[..., C] -> codes [..., C / 2] (value 2 i in the low half of byte i), scales [..., C / 32]."""
    b = x.float().reshape(*x.shape[:-1], x.shape[-1] // QB, QB)
    e = _scale_exp(b.abs().amax(-1), 6.0, 3)
    q = _nibbles(torch.ldexp(b, -e[..., None])).reshape(x.shape)
    return q[..., 0::2] | (q[..., 1::2] << 4), (e + 127).to(torch.uint8)


def _to_fp8(x):
    b = x.float().reshape(*x.shape[:-1], x.shape[-1] // QB, QB)
    e = _scale_exp(b.abs().amax(-1), 448.0, 9)
    q = torch.ldexp(b, -e[..., None]).to(torch.float8_e4m3fn).reshape(x.shape)
    return q.view(torch.uint8), (e + 127).to(torch.uint8)


def _weights(g, E, K, N):
    """Codes [E, N, K / 2] and scales [E, N, K / 32] of normal weights [E, N, K]."""
    codes = torch.empty(E, N, K // 2, dtype=torch.uint8, device=DEV)
    scales = torch.empty(E, N, K // QB, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 27) // (K * N))
    for e in range(0, E, step):
        n = min(step, E - e)
        w = torch.randn(n, N, K, generator=g, device=DEV).mul_(K ** -0.5)
        codes[e:e + n], scales[e:e + n] = _to_fp4(w)
    return codes, scales


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 29)
    s = dict(c=c)
    if own:
        import expert_ffn_moe_amd as moe
        s["moe"] = moe
    op = c["op"]

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=g, device=DEV, dtype=F32).mul_(scale)

    if op in ("route", "route_grad"):
        T, E, k = c["T"], c["E"], c["k"]
        logits = normal(T, E)
        logits += normal(E, scale=0.5)
        if c["masked"]:
            logits[:, torch.randperm(E, generator=g, device=DEV)[:c["masked"]]] = -INF
        s["logits"] = logits
        s["bias"] = normal(E, scale=0.1) if c["bias"] else None
        if own:
            s["p"] = s["moe"].Problem(T=T, H=64, E=E, k=k, I=64, capacity=c["cap"],
                                      renormalize=int(c["renorm"]))
            s["scoring"] = s["moe"].Scoring(score=c["score"], n_group=c["groups"],
                                            topk_group=c["taken"],
                                            group_score=c["group_score"], scale=c["scale"])
        if op == "route":
            s["out"] = (torch.zeros(T, k, dtype=torch.int32, device=DEV),
                        torch.zeros(T, k, dtype=F32, device=DEV),
                        torch.zeros(T, k, dtype=torch.uint8, device=DEV))
            if own:
                s["ws"] = s["moe"].workspace(s["p"], s["moe"].OP_ROUTE, DEV)
        else:  # the forward's routing
            s["ids"], s["w"], _ = _plain_route(c, logits, s["bias"])
            s["dw"] = normal(T, k)
            s["grad"] = torch.zeros(T, E, dtype=F32, device=DEV)
        return s
    if op == "quantize":
        E, rows, cols = c["E"], c["rows"], c["cols"]
        shape = (E, cols, rows) if E else (rows, cols)
        x = torch.randn(*shape, generator=g, device=DEV, dtype=BF16)
        if not E:  # activations: a few columns are far larger than the others
            x *= torch.exp(normal(cols)).to(BF16)
        s["x"] = x
        lead = (E, rows) if E else (rows,)
        s["codes"] = torch.zeros(*lead, cols // 2, dtype=torch.uint8, device=DEV)
        s["scales"] = torch.zeros(*lead, cols // QB, dtype=torch.uint8, device=DEV)
        s["values"] = torch.zeros(*lead, cols, dtype=BF16, device=DEV)
        return s
    T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
    R = T * k
    row_token, offsets, counts = _layout(c, g)
    host = counts.tolist()
    s["R"], s["live"] = R, sum(host)
    s["offsets"] = offsets
    s["row_token"] = row_token if E > 1 else None
    # the plan of a program that pads: the experts with rows, and each row's place
    active = [e for e in range(E) if host[e]]
    s["cmax"] = max(host)
    s["active"] = torch.tensor(active, dtype=torch.int64, device=DEV)
    per = torch.tensor([host[e] for e in active], dtype=torch.int64, device=DEV)
    s["row_slot"] = torch.repeat_interleave(torch.arange(len(active), device=DEV), per)
    s["row_pos"] = (torch.arange(s["live"], device=DEV)
                    - offsets[:-1].long()[s["active"]][s["row_slot"]])
    x = normal(T, K)
    s["x"] = _to_fp4(x) if c["x"] == "fp4" else _to_fp8(x)
    s["w"] = _weights(g, E, K, N)
    s["up"] = _weights(g, E, K, N) if c["gated"] else None
    s["bias"] = normal(E, N, scale=0.5).to(BF16) if c["bias"] else None
    s["up_bias"] = normal(E, N, scale=0.5).to(BF16) if c["bias"] and c["gated"] else None
    s["residual"] = normal(R, N).to(BF16) if c["residual"] else None
    s["y"] = torch.zeros(R, N, dtype=BF16, device=DEV)
    if own:
        s["p"] = s["moe"].GroupedProblem(R=R, K=K, N=N, E=E, T=T if E > 1 else R)
        s["ws"] = s["moe"].grouped_workspace(s["p"], s["moe"].OP_GROUPED_FP4, DEV)
    return s


# --------------------------------------------------------------------- the plain forms
def _scores(c, logits):
    """(scores, in service) in 64 bits: a choice next to a border needs them."""
    l = logits.double()
    there = l > -INF  # false for NaN too
    l = torch.where(there, l.clamp(max=BIG), torch.full_like(l, -BIG))
    if c["score"] == "sigmoid":
        s = 1 / (1 + torch.exp(-l))
    else:
        s = torch.exp(l - l.amax(1, keepdim=True)) * there
        s = s / s.sum(1, keepdim=True).clamp(min=1e-300)
    return torch.where(there, s, torch.zeros_like(s)), there


def _plain_route(c, logits, bias):
    T, E, k = c["T"], c["E"], c["k"]
    s, there = _scores(c, logits)
    # without a bias the order is that of the logits
    order = logits.double().clamp(max=BIG) if bias is None else s + bias.double()
    order = torch.where(there, order, torch.full_like(s, -INF))
    if c["groups"] > 1 and c["taken"] < c["groups"]:
        size = E // c["groups"]
        of = order.reshape(T, c["groups"], size)
        best = torch.sort(of, dim=2, descending=True).values
        rank = best[..., 0]
        if c["group_score"] == "top2":
            by = s if bias is None else s + bias.double()
            by = torch.where(there, by, torch.full_like(s, -INF)).reshape(of.shape)
            by = torch.sort(by, dim=2, descending=True).values
            rank = by[..., 0]
            if size > 1:
                rank = rank + torch.where(by[..., 1] > -INF, by[..., 1], torch.zeros_like(rank))
        first = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :c["taken"]]
        inside = torch.zeros(T, c["groups"], dtype=torch.bool, device=DEV)
        inside.scatter_(1, first, True)
        inside = inside.repeat_interleave(size, 1)
    else:
        inside = torch.ones_like(there)
    # 2: can be chosen, 1: out of service in a taken group, 0: in a group not taken
    place = inside.long() + (inside & there).long()
    by = torch.sort(order, dim=1, descending=True, stable=True).indices
    by = by.gather(1, torch.sort(place.gather(1, by), dim=1, descending=True,
                                 stable=True).indices)
    ids = by[:, :k]
    live = there.gather(1, ids)
    w = torch.where(live, s.gather(1, ids), torch.zeros((), dtype=F64, device=DEV))
    if c["renorm"]:
        total = w.sum(1, keepdim=True)
        w = torch.where(total > 0, w / torch.where(total > 0, total, torch.ones_like(total)), w)
    w = (w * c["scale"]).float()
    keep = live.to(torch.uint8)
    if c["cap"] > 0:  # an expert keeps its `cap` largest weights, ties to the earlier token
        flat, fw = ids.reshape(-1), w.reshape(-1)
        q = torch.sort(fw, descending=True, stable=True).indices
        q = q[torch.sort(flat[q] + E * (1 - keep.reshape(-1)[q].long()), stable=True).indices]
        q = q[:int(keep.sum())]  # those out of service are behind all others
        n = torch.bincount(flat[q], minlength=E)
        pos = torch.arange(q.numel(), device=DEV) - (torch.cumsum(n, 0) - n)[flat[q]]
        keep.view(-1)[q[pos >= c["cap"]]] = 0
    return ids.to(torch.int32), w, keep


def _plain_route_grad(s):
    c = s["c"]
    p, _ = _scores(c, s["logits"])
    ids, w, dw = s["ids"].long(), s["w"].double(), s["dw"].double()
    dot = (w * dw).sum(1, keepdim=True)  # cancels against dw below: in 64 bits
    if c["renorm"]:
        dot = dot / w.sum(1, keepdim=True).clamp(min=1e-300)
    chosen = p.gather(1, ids)
    if c["score"] == "sigmoid":
        d = w * (1 - chosen) * (dw - dot if c["renorm"] else dw)
        return torch.zeros_like(p).scatter_(1, ids, d).float()
    if c["renorm"]:
        return torch.zeros_like(p).scatter_(1, ids, w * (dw - dot)).float()
    return (-p * dot).scatter_add_(1, ids, w * dw).float()


_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def _from_fp4(codes, scales):
    table = torch.tensor(_LEVELS + tuple(-v for v in _LEVELS), device=DEV)
    v = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1)
    v = v.reshape(*codes.shape[:-1], -1, QB)
    f = torch.ldexp(torch.ones((), device=DEV), scales.int() - 127)
    return (v * f[..., None]).reshape(*codes.shape[:-1], -1)


def _x_values(s, n):
    """The n live rows of x in 32 bits."""
    codes, scales = s["x"]
    if s["row_token"] is not None:
        t = s["row_token"][:n].long()
        codes, scales = codes[t], scales[t]
    if s["c"]["x"] == "fp4":
        return _from_fp4(codes, scales)
    v = codes.view(torch.float8_e4m3fn).float().reshape(n, -1, QB)
    return (v * torch.ldexp(torch.ones((), device=DEV), scales.int() - 127)[..., None]).reshape(
        n, -1)


def _act(z, act):
    if act == "relu2":
        return z * z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
        return z / (1 + torch.exp(-2 * u))
    return z


def _plain_linear(s):
    c, n = s["c"], s["live"]
    at = (s["row_slot"], s["row_pos"])
    x = torch.zeros(len(s["active"]), s["cmax"], c["K"], device=DEV)
    x[at] = _x_values(s, n)
    total = torch.empty(n, c["N"], device=DEV)

    def product(w, bias):
        step = max(1, (1 << 29) // (c["K"] * c["N"]))  # experts whose weights are expanded
        z = torch.empty(x.shape[0], x.shape[1], c["N"], device=DEV)
        for i in range(0, x.shape[0], step):
            e = s["active"][i:i + step]
            we = _from_fp4(w[0][e], w[1][e]).transpose(1, 2).contiguous()
            torch.bmm(x[i:i + step], we, out=z[i:i + step])
        z = z[at]
        return z if bias is None else z + bias.float()[s["active"]][s["row_slot"]]

    y = _act(product(s["w"], s["bias"]), c["act"])
    if s["up"] is not None:
        y = y * product(s["up"], s["up_bias"])
    if s["residual"] is not None:
        y = y + s["residual"][:n].float()
    s["y"][:n] = y.to(BF16)


def run(s):
    c = s["c"]
    op = c["op"]
    if op == "route":
        if own:
            s["moe"].route_scored(s["p"], s["logits"], s["scoring"], bias=s["bias"],
                                  out=s["out"], ws=s["ws"])
            ids, w, keep = s["out"]
        else:
            ids, w, keep = _plain_route(c, s["logits"], s["bias"])
        return dict(ids=ids, w=w, keep=keep)
    if op == "route_grad":
        if own:
            return dict(dlogits=s["moe"].route_scored_backward(
                s["p"], s["logits"], s["scoring"], s["ids"], s["w"], s["dw"], out=s["grad"]))
        return dict(dlogits=_plain_route_grad(s))
    if op == "quantize":
        if own:
            out = (s["codes"], s["scales"])
            if c["E"]:
                s["moe"].quantize_fp4_weights(s["x"], out=out)
            else:
                s["moe"].quantize_fp4(s["x"], out=out)
            s["moe"].dequantize_fp4(*out, out=s["values"])
            values, scales = s["values"], s["scales"]
        else:
            x = s["x"].transpose(1, 2).contiguous() if c["E"] else s["x"]
            codes, scales = _to_fp4(x)
            values = _from_fp4(codes, scales).to(BF16)
        return dict(values=values, scales=scales.view(torch.float8_e8m0fnu))
    if own:
        s["moe"].grouped_linear_fp4(s["p"], s["x"], s["w"],
                                    s["offsets"] if c["E"] > 1 else None, up=s["up"],
                                    bias=s["bias"], up_bias=s["up_bias"], act=c["act"],
                                    residual=s["residual"], row_token=s["row_token"], out=s["y"],
                                    ws=s["ws"])
    else:
        _plain_linear(s)
    return dict(y=s["y"])


# ------------------------------------------------------------------------ what is needed
def work(c):
    op = c["op"]
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return dict(bytes=4 * T * E + 9 * T * k + (4 * E if c["bias"] else 0), flops=20 * T * E)
    if op == "route_grad":
        T, E, k = c["T"], c["E"], c["k"]
        dense = c["score"] == "softmax" and not c["renorm"]  # the others read k logits a token
        return dict(bytes=4 * T * E + 12 * T * k + 4 * T * (E if dense else k),
                    flops=(20 if dense else 1) * T * E)
    if op == "quantize":  # 2 bytes in, codes and scales out and in again, 2 bytes out
        n = max(1, c["E"]) * c["rows"] * c["cols"]
        return dict(bytes=n * (4 + 2 * (0.5 + 1 / QB)), flops=8 * n)
    T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
    R = T * k
    share = 1.0
    if c["skew"] == "zipf" and c["cap"] > 0 and E > 1:  # rows that the capacity leaves
        p = [r ** -1.2 for r in range(1, E + 1)]
        share = sum(min(c["cap"], R * v / sum(p)) for v in p) / R
    n = R * share
    active = E * (1 - (1 - k / E) ** T) if k < E else E
    mats = 2 if c["gated"] else 1
    per = (0.5 if c["x"] == "fp4" else 1) + 1 / QB
    b = min(T, n) * K * per + mats * active * K * N * (0.5 + 1 / QB)
    b += 2 * n * N * (2 if c["residual"] else 1) + (2 * mats * active * N if c["bias"] else 0)
    return dict(bytes=b, flops=2 * mats * n * K * N)


# --------------------------------------------------------------- the definition in 64 bits
def _exact_route(c, s):
    import numpy as np
    T, E, k = c["T"], c["E"], c["k"]
    l = s["logits"].double().cpu().numpy()
    out = ~(l > -np.inf)
    l = np.where(out, 0.0, np.minimum(l, BIG))
    if c["score"] == "sigmoid":
        p = np.exp(-np.logaddexp(0.0, -l))
    else:
        m = np.where(out, -np.inf, l).max(1, keepdims=True)
        m = np.where(np.isfinite(m), m, 0.0)
        p = np.where(out, 0.0, np.exp(l - m))
        p /= np.maximum(p.sum(1, keepdims=True), 1e-300)
    p = np.where(out, 0.0, p)
    choice = p if s["bias"] is None else p + s["bias"].double().cpu().numpy()
    key = l if s["bias"] is None else choice
    away = np.zeros((T, E), dtype=bool)
    G, n = c["groups"], E // c["groups"]
    if c["taken"] < G:
        value = np.empty((T, G))
        for i in range(G):
            sl = slice(i * n, (i + 1) * n)
            v = np.where(out[:, sl], -np.inf,
                         (key if c["group_score"] == "max" else choice)[:, sl])
            top = np.partition(v, n - 1, axis=1)[:, n - 1]
            if c["group_score"] == "top2" and n > 1:
                second = np.partition(v, n - 2, axis=1)[:, n - 2]
                top = top + np.where(np.isfinite(second), second, 0.0)
            value[:, i] = top
        ahead = ((value[:, None, :] > value[:, :, None]).sum(2)
                 + np.tril((value[:, None, :] == value[:, :, None]), -1).sum(2))
        away = np.repeat(ahead >= c["taken"], n, axis=1)
    index = np.broadcast_to(np.arange(E), (T, E))
    ids = np.lexsort((index, np.where(out, 0.0, -key), 2 * away + out), axis=1)[:, :k]
    row = np.arange(T)[:, None]
    dead = out[row, ids]
    w = p[row, ids]
    if c["renorm"]:
        total = w.sum(1, keepdims=True)
        w = np.divide(w, total, out=np.zeros_like(w), where=total > 0)
    w *= c["scale"]
    keep = (~dead).astype(np.uint8)
    if c["cap"] > 0:
        w32 = w.astype(np.float32)
        for e in range(E):
            t, j = np.nonzero((ids == e) & (keep > 0))
            rest = np.lexsort((t, -w32[t, j]))[c["cap"]:]
            keep[t[rest], j[rest]] = 0
    to = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(DEV)  # noqa: E731
    return dict(ids=to(ids.astype(np.int32)), w=to(w), keep=to(keep))


def _exact_route_grad(c, s):
    """Through the scores: dL/dscore by the quotient rule, then the score's own derivative."""
    l, ids, g = s["logits"].to(F64), s["ids"].long(), s["dw"].to(F64)
    alive = torch.isfinite(l)
    if c["score"] == "sigmoid":
        p = torch.sigmoid(l) * alive
    else:
        p = torch.softmax(l, 1).nan_to_num(0.0)
    ok = torch.gather(alive, 1, ids) & (s["w"] > 0)
    v = torch.gather(p, 1, ids) * ok
    g = g * ok * c["scale"]
    if c["renorm"]:
        total = v.sum(1, keepdim=True)
        g = torch.where(total > 0, (g * total - (g * v).sum(1, keepdim=True)) / total ** 2, 0.0)
        g = g * ok
    if c["score"] == "sigmoid":
        return dict(dlogits=torch.zeros_like(l).scatter(1, ids, g * v * torch.sigmoid(
            -torch.gather(l, 1, ids)) * ok))
    dp = torch.zeros_like(l).scatter(1, ids, g)
    return dict(dlogits=p * (dp - (dp * p).sum(1, keepdim=True)))


def _exact_fp4(x):
    """Values and scales of the 4-bit form of x [rows, cols], by distance to the 8 levels."""
    rows, cols = x.shape
    b = x.to(F64).reshape(rows, cols // QB, QB)
    top = b.abs().amax(-1)
    e = torch.ceil(torch.log2(top / 6))
    e = torch.where(top > 6 * torch.exp2(e), e + 1, e)  # a log2 on the wrong side
    e = torch.where(top <= 6 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 0, e, torch.zeros_like(e)).clamp(min=-127)
    v = b * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=1.0)))) / 2
    q = torch.round(v / step) * step
    return (q * torch.exp2(e)[..., None]).reshape(rows, cols), torch.exp2(e)


def _exact_values(codes, scales, eight):
    c = codes.long()
    if eight:
        v = codes.view(torch.float8_e4m3fn).to(F64)
    else:
        n = torch.stack((c % 16, c // 16), -1).flatten(-2)
        m, x = (n % 2).to(F64), ((n % 8) // 2).to(F64)
        v = torch.where(x > 0, torch.exp2(x - 1) * (1 + m / 2), m / 2)
        v = torch.where(n >= 8, -v, v)
    return v * torch.exp2(scales.to(F64) - 127).repeat_interleave(QB, -1)


def exact(c, seed):
    s = prepare(c, seed)
    op = c["op"]
    if op == "route":
        return _exact_route(c, s)
    if op == "route_grad":
        return _exact_route_grad(c, s)
    if op == "quantize":
        if not c["E"]:
            v, f = _exact_fp4(s["x"])
        else:
            got = [_exact_fp4(s["x"][e].t().contiguous()) for e in range(c["E"])]
            v, f = torch.stack([a for a, _ in got]), torch.stack([b for _, b in got])
        return dict(values=v, scales=f)
    off = s["offsets"].tolist()
    y = torch.zeros(s["R"], c["N"], dtype=F64, device=DEV)
    for e in range(c["E"]):
        lo, hi = off[e], off[e + 1]
        if lo == hi:
            continue
        rows = s["row_token"][lo:hi].long() if s["row_token"] is not None else slice(lo, hi)
        x = _exact_values(s["x"][0][rows], s["x"][1][rows], c["x"] == "fp8")
        z = x @ _exact_values(s["w"][0][e], s["w"][1][e], False).t()
        if c["bias"]:
            z += s["bias"][e].to(F64)
        if c["act"] == "relu2":
            z = z.clamp(min=0) ** 2
        elif c["act"] == "silu":
            z = z * torch.sigmoid(z)
        elif c["act"] == "gelu_tanh":
            z = 0.5 * z * (1 + torch.tanh((2 / math.pi) ** 0.5 * (z + 0.044715 * z ** 3)))
        if c["gated"]:
            u = x @ _exact_values(s["up"][0][e], s["up"][1][e], False).t()
            z = z * (u + s["up_bias"][e].to(F64) if c["bias"] else u)
        y[lo:hi] = z
    if c["residual"]:
        n = off[-1]
        y[:n] += s["residual"][:n].to(F64)
    return dict(y=y)
