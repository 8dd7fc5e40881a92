"""Measured cases of the grouped-linear operators and the 8-bit activation checkpoints.

Four entry points of expert_ffn_moe_amd, on the expert-contiguous row layout of the layer
(rows of expert e are offsets[e] .. offsets[e + 1] - 1; E = 1 without offsets is a dense
product):

  linear        y[r] = act(x[r] W[e] + b[e]) + residual[r], with z = x W + b optionally saved
                as an 8-bit checkpoint (E4M3 codes, one power-of-two scale per 32 columns)
  dx            dx[r] = (dz[r] W[e]^T) * act'(z[r]) and a[r] = act(z[r]), z from a checkpoint
  dw            dW[e] = x_e^T dz_e, db[e] = the column sums of dz_e (fp32)
  act_backward  dz[r] = dy[r] * act'(z[r]) and a[r] = act(z[r]), z from a checkpoint

Rows behind the last expert's are left as they were: the outputs are buffers of the state.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64
QB = 32  # columns per scale of a checkpoint


# ---------------------------------------------------------------------------- the cases
def _case(name, op, T, E, k, K, N, act="none", skew="even", cap=0, gather=False, bias=False,
          residual=False, ckpt=False):
    c = dict(op=op, T=T, E=E, k=k, K=K, N=N, act=act, skew=skew, cap=cap, gather=gather,
             bias=bias, residual=residual, ckpt=ckpt)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one token of a serving loop through its 8 experts: latency
        _case("linear one token", "linear", 1, 128, 8, 2048, 768, act="silu", bias=True,
              gather=True),
        # a decode batch: nearly every expert's weights are read for a few rows
        _case("linear decode batch", "linear", 128, 256, 8, 7168, 2048, act="silu", bias=True,
              gather=True),
        # prefill of a layer with many small experts
        _case("linear prefill", "linear", 4096, 128, 8, 2048, 768, act="gelu_tanh",
              skew="bias", bias=True, gather=True),
        # a dense projection with residual on a batch and widths that fill no tile
        _case("linear dense odd", "linear", 1003, 1, 1, 1416, 2056, act="gelu_tanh", bias=True,
              residual=True),
        # training forward, skewed routing under a capacity, pre-activations kept in 8 bits
        _case("linear checkpoint skew", "linear", 8192, 64, 4, 4096, 1408, act="silu",
              skew="zipf", cap=1024, bias=True, gather=True, ckpt=True),
        # the largest: training forward of a wide layer, pre-activations kept in 8 bits
        _case("linear checkpoint wide", "linear", 16384, 256, 8, 7168, 2048, act="silu",
              gather=True, ckpt=True),
        # data gradient of the second product, through the activation read back from 8 bits
        _case("dx checkpoint skew", "dx", 8192, 64, 4, 1408, 4096, act="silu", skew="zipf",
              cap=1024, ckpt=True),
        # data gradient of a plain product, few rows per expert and odd widths
        _case("dx odd", "dx", 333, 16, 2, 1096, 520),
        # weight and bias gradients of the prefill shape, rows gathered from the tokens
        _case("dw prefill", "dw", 4096, 128, 8, 2048, 768, skew="bias", bias=True, gather=True),
        # weight gradient of one dense projection: a long sum for few tiles
        _case("dw dense long", "dw", 16384, 1, 1, 2048, 768, bias=True),
        # elementwise: the activation's gradient from an 8-bit checkpoint
        _case("act backward", "act_backward", 8192, 64, 4, 4096, 1408, act="gelu_tanh",
              skew="zipf", cap=1024, ckpt=True),
        _case("act backward small", "act_backward", 61, 8, 2, 128, 768, act="silu", ckpt=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["linear", "linear", "linear", "dx", "dx", "dw", "dw", "act_backward"])
    E = rng.choice([1, _log(rng, 2, 256), _log(rng, 2, 256)])
    k = 1 if E == 1 else min(E, rng.choice([1, 2, 4, 8]))
    K, N = 8 * _log(rng, 8, 896), 8 * _log(rng, 8, 512)
    ckpt = op == "act_backward" or (op in ("linear", "dx") and rng.random() < 0.5)
    act = rng.choice(["relu", "relu2", "silu", "gelu_tanh"]) if op != "dw" else "none"
    if op == "dx" and not ckpt:
        act = "none"
    if op == "linear" and not ckpt and rng.random() < 0.25:
        act = "none"
    if ckpt:  # the checkpoint's width is a multiple of 32
        if op == "dx":
            K = max(32, K // 32 * 32)
        else:
            N = max(32, N // 32 * 32)
    T = _log(rng, 1, 16384)
    while E * K * N > 1 << 30:
        E = max(1, E // 2)
    k = min(k, E)
    while T > 1 and 2.0 * T * k * K * N > 1.5e12:
        T //= 2
    skew = "even" if E == 1 else rng.choice(["even", "bias", "zipf"])
    cap = max(1, 2 * T * k // E) if skew == "zipf" else 0
    return _case("", op, T, E, k, K, N, act=act, skew=skew, cap=cap,
                 gather=op in ("linear", "dw") and E > 1 and rng.random() < 0.5,
                 bias=op in ("linear", "dw") and rng.random() < 0.5,
                 residual=op == "linear" and rng.random() < 0.3, ckpt=ckpt)


# ---------------------------------------------------------------------------- the inputs
def _layout(c, g):
    """Routing of T tokens to k of E experts: the sorted rows' tokens, offsets and counts."""
    T, E, k = c["T"], c["E"], c["k"]
    score = torch.randn(T, E, generator=g, device=DEV)
    if c["skew"] == "bias":
        score += 0.5 * torch.randn(E, generator=g, device=DEV)
    elif c["skew"] == "zipf":
        rank = torch.randperm(E, generator=g, device=DEV).float() + 1
        score -= 1.2 * torch.log(rank)
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


def _quantize(z):
    """E4M3 codes and power-of-two scales of 32-column blocks: the smallest 2^e with
    max|z| <= 448 * 2^e (2^0 for a block of zeros)."""
    R, N = z.shape
    b = z.reshape(R, N // QB, QB)
    m, x = torch.frexp(b.abs().amax(-1))
    e = torch.where(m > 0, x - 9 + (m > 0.875), torch.zeros_like(x)).clamp(-127, 127)
    codes = torch.ldexp(b, -e[..., None]).float().to(torch.float8_e4m3fn).reshape(R, N)
    return codes, torch.ldexp(torch.ones_like(m), e).float().to(torch.float8_e8m0fnu)


def _bytes(t):
    return t.view(torch.uint8)


def prepare(c, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 1000003 + 17)
    T, E, K, N = c["T"], c["E"], c["K"], c["N"]
    R = T * c["k"]

    def draw_(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=BF16)
                .mul_(scale) if scale != 1.0 else
                torch.randn(*shape, generator=g, device=DEV, dtype=BF16))

    row_token, offsets, counts = _layout(c, g)
    host = counts.tolist()
    live = sum(host)
    s = dict(c=c, R=R, live=live, offsets=offsets, row_token=row_token if c["gather"] else None)
    # the plan of a program that pads: the experts with rows, and each row's place
    active = [e for e in range(E) if host[e]]
    slot = {e: i for i, e in enumerate(active)}
    s["cmax"] = max(host) if active else 0
    s["active"] = torch.tensor(active, dtype=torch.int64, device=DEV)
    per = torch.tensor([host[e] for e in active], dtype=torch.int64, device=DEV)
    s["row_slot"] = torch.repeat_interleave(torch.arange(len(slot), device=DEV), per)
    s["row_pos"] = torch.arange(live, device=DEV) - offsets[:-1].long()[s["active"]][s["row_slot"]]

    op = c["op"]
    if op in ("linear", "dw"):
        s["x"] = draw_(T if c["gather"] else R, K)
    if op in ("dx", "dw"):
        s["dz"] = draw_(R, N)
    if op in ("linear", "dx"):
        s["w"] = draw_(E, K, N, scale=(K if op == "linear" else N) ** -0.5)
    if op == "linear":
        s["bias"] = draw_(E, N, scale=0.5) if c["bias"] else None
        s["residual"] = draw_(R, N) if c["residual"] else None
        s["y"] = torch.zeros(R, N, dtype=BF16, device=DEV)
    if op == "act_backward":
        s["dy"] = draw_(R, N)
    width = K if op == "dx" else N
    if c["ckpt"]:
        if op == "linear":  # written by the call
            s["codes"] = torch.zeros(R, width, dtype=torch.uint8, device=DEV)
            s["scales"] = torch.zeros(R, width // QB, dtype=torch.uint8, device=DEV)
        else:  # the forward's
            z = torch.randn(R, width, generator=g, device=DEV)
            codes, scales = _quantize(z)
            s["codes"], s["scales"] = _bytes(codes), _bytes(scales)
    if op in ("dx", "act_backward"):
        s["grad"] = torch.zeros(R, width, dtype=BF16, device=DEV)
        s["a"] = torch.zeros(R, width, dtype=BF16, device=DEV) if c["ckpt"] else None
    if own:
        import expert_ffn_moe_amd as moe
        s["moe"] = moe
        s["p"] = moe.GroupedProblem(R=R, K=K, N=N, E=E, T=T if c["gather"] else R)
        s["ws"] = {"linear": moe.OP_GROUPED_LINEAR, "dx": moe.OP_GROUPED_DX,
                   "dw": moe.OP_GROUPED_DW}.get(op)
        if s["ws"] is not None:
            s["ws"] = moe.grouped_workspace(s["p"], s["ws"], DEV)
    return s


# --------------------------------------------------------------------- the plain forms
def _act(z, act):
    if act == "relu":
        return z * (z > 0)
    if act == "relu2":
        return z * z * (z > 0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu_tanh":
        u = math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)
        return z / (1 + torch.exp(-2 * u))
    return z


def _act_grad(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "relu2":
        return 2 * z * (z > 0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    if act == "gelu_tanh":
        r = math.sqrt(2 / math.pi)
        s = 1 / (1 + torch.exp(-2 * r * (z + 0.044715 * z * z * z)))
        return s + z * s * (1 - s) * 2 * r * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _padded(s, rows):
    """[live, C] rows as [active experts, cmax, C] in 32 bits, zeros behind each expert's."""
    p = torch.zeros(len(s["active"]), s["cmax"], rows.shape[1], device=DEV)
    p[s["row_slot"], s["row_pos"]] = rows.float()
    return p


def _x_rows(s):
    n = s["live"]
    return s["x"][:n] if s["row_token"] is None else s["x"][s["row_token"][:n].long()]


def _checkpoint(s):
    n = s["live"]
    codes = s["codes"][:n].view(torch.float8_e4m3fn).float()
    scales = s["scales"][:n].view(torch.float8_e8m0fnu).float()
    return (codes.reshape(n, -1, QB) * scales[..., None]).reshape(n, -1)


def _plain_linear(s):
    c, n = s["c"], s["live"]
    z = torch.bmm(_padded(s, _x_rows(s)), s["w"][s["active"]].float())
    z = z[s["row_slot"], s["row_pos"]]
    if s["bias"] is not None:
        z = z + s["bias"].float()[s["active"]][s["row_slot"]]
    if c["ckpt"]:
        codes, scales = _quantize(z)
        s["codes"][:n] = _bytes(codes)
        s["scales"][:n] = _bytes(scales)
    y = _act(z, c["act"])
    if s["residual"] is not None:
        y = y + s["residual"][:n].float()
    s["y"][:n] = y.to(BF16)


def _plain_dx(s):
    c, n = s["c"], s["live"]
    w = s["w"][s["active"]].float().transpose(1, 2).contiguous()
    d = torch.bmm(_padded(s, s["dz"][:n]), w)[s["row_slot"], s["row_pos"]]
    if c["ckpt"]:
        z = _checkpoint(s)
        d = d * _act_grad(z, c["act"])
        s["a"][:n] = _act(z, c["act"]).to(BF16)
    s["grad"][:n] = d.to(BF16)


def _plain_dw(s):
    c, n = s["c"], s["live"]
    dw = torch.zeros(c["E"], c["K"], c["N"], device=DEV)
    dz = _padded(s, s["dz"][:n])
    dw[s["active"]] = torch.bmm(_padded(s, _x_rows(s)).transpose(1, 2).contiguous(), dz)
    if not c["bias"]:
        return dw, None
    db = torch.zeros(c["E"], c["N"], device=DEV)
    db[s["active"]] = dz.sum(1)
    return dw, db


def _plain_act_backward(s):
    c, n = s["c"], s["live"]
    z = _checkpoint(s)
    s["grad"][:n] = (s["dy"][:n].float() * _act_grad(z, c["act"])).to(BF16)
    s["a"][:n] = _act(z, c["act"]).to(BF16)


def run(s):
    c = s["c"]
    op = c["op"]
    offsets = s["offsets"] if c["E"] > 1 else None
    if op == "linear":
        if own:
            s["moe"].grouped_linear(s["p"], s["x"], s["w"], offsets, bias=s["bias"],
                                    act=c["act"], residual=s["residual"],
                                    row_token=s["row_token"], out=s["y"],
                                    checkpoint=(s["codes"], s["scales"]) if c["ckpt"] else None,
                                    ws=s["ws"])
        else:
            _plain_linear(s)
        if c["ckpt"]:
            return dict(y=s["y"], codes=s["codes"].view(torch.float8_e4m3fn),
                        scales=s["scales"].view(torch.float8_e8m0fnu))
        return dict(y=s["y"])
    if op == "dx":
        if own:
            s["moe"].grouped_linear_dx(s["p"], s["dz"], s["w"], offsets, act=c["act"],
                                       checkpoint=(s["codes"], s["scales"]) if c["ckpt"] else None,
                                       out=s["grad"], a=s["a"], ws=s["ws"])
        else:
            _plain_dx(s)
        return dict(dx=s["grad"], a=s["a"]) if c["ckpt"] else dict(dx=s["grad"])
    if op == "dw":
        if own:
            dw, db = s["moe"].grouped_linear_dw(s["p"], s["x"], s["dz"], offsets,
                                                row_token=s["row_token"], want_bias=c["bias"],
                                                ws=s["ws"])
        else:
            dw, db = _plain_dw(s)
        return dict(dw=dw, db=db) if c["bias"] else dict(dw=dw)
    if own:
        s["moe"].activation_backward(s["dy"], (s["codes"], s["scales"]), c["act"],
                                     live_rows=s["offsets"][-1:], out=s["grad"], a=s["a"])
    else:
        _plain_act_backward(s)
    return dict(dz=s["grad"], a=s["a"])


# ------------------------------------------------------------------------ what is needed
def work(c):
    T, E, k, K, N = c["T"], c["E"], c["k"], c["K"], c["N"]
    R = T * k
    share = 1.0
    if c["skew"] == "zipf" and c["cap"] > 0 and E > 1:  # rows that the capacity leaves
        p = [r ** -1.2 for r in range(1, E + 1)]
        share = sum(min(c["cap"], R * v / sum(p)) for v in p) / R
    n = R * share
    active = E * (1 - (1 - k / E) ** T) if k < E else E
    x_rows = min(T, n) if c["gather"] else n
    op = c["op"]
    ck = 1 + 1 / QB
    if op == "linear":
        b = 2 * x_rows * K + 2 * active * K * N + 2 * n * N * (2 if c["residual"] else 1)
        b += n * N * ck if c["ckpt"] else 0
        b += 2 * active * N if c["bias"] else 0
        return dict(bytes=b, flops=2 * n * K * N)
    if op == "dx":
        b = 2 * n * N + 2 * active * K * N + 2 * n * K
        b += n * K * (ck + 2) if c["ckpt"] else 0
        return dict(bytes=b, flops=2 * n * K * N)
    if op == "dw":
        b = 2 * x_rows * K + 2 * n * N + 4 * E * K * N + (4 * E * N if c["bias"] else 0)
        return dict(bytes=b, flops=2 * n * K * N)
    return dict(bytes=n * N * (2 + 2 + 2 + ck), flops=20 * n * N)


# --------------------------------------------------------------- the definition in 64 bits
def _exact_act(z, name):
    sig = torch.sigmoid
    if name == "relu":
        return z.clamp(min=0), torch.heaviside(z, torch.zeros_like(z))
    if name == "relu2":
        return z.clamp(min=0) ** 2, 2 * z.clamp(min=0)
    if name == "silu":
        return z * sig(z), sig(z) + z * sig(z) * sig(-z)
    if name == "gelu_tanh":
        r = (2 / math.pi) ** 0.5
        t = torch.tanh(r * (z + 0.044715 * z ** 3))
        return (0.5 * z * (1 + t),
                0.5 * (1 + t) + 0.5 * z * (1 - t ** 2) * r * (1 + 0.134145 * z ** 2))
    return z, torch.ones_like(z)


def _exact_blocks(z):
    """The values that the codes and scales of z stand for, rounded by hand in 64 bits."""
    R, N = z.shape
    b = z.reshape(R, N // QB, QB)
    top = b.abs().amax(-1)
    e = torch.ceil(torch.log2(top / 448))
    e = torch.where(top > 448 * torch.exp2(e), e + 1, e)  # a log2 on the wrong side
    e = torch.where(top <= 448 * torch.exp2(e - 1), e - 1, e)
    e = torch.where(top > 0, e, torch.zeros_like(e))
    v = b * torch.exp2(-e)[..., None]
    step = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / step) * step).reshape(R, N), torch.exp2(e)


def exact(c, seed):
    s = prepare(c, seed)
    op, E, K, N, R = c["op"], c["E"], c["K"], c["N"], s["R"]
    off = s["offsets"].tolist()
    n = off[-1]
    if c["ckpt"] and op != "linear":
        codes = s["codes"].view(torch.float8_e4m3fn).to(F64)
        scales = s["scales"].view(torch.float8_e8m0fnu).to(F64)
        z = codes * scales.repeat_interleave(QB, 1)
        f, df = _exact_act(z, c["act"])
    if op == "act_backward":
        dz, a = torch.zeros(R, N, dtype=F64, device=DEV), torch.zeros(R, N, dtype=F64, device=DEV)
        dz[:n], a[:n] = (s["dy"].to(F64) * df)[:n], f[:n]
        return dict(dz=dz, a=a)
    if op == "dw":
        out = dict(dw=torch.zeros(E, K, N, dtype=F64, device=DEV))
        if c["bias"]:
            out["db"] = torch.zeros(E, N, dtype=F64, device=DEV)
        for e in range(E):
            lo, hi = off[e], off[e + 1]
            rows = torch.arange(lo, hi, device=DEV)
            x = s["x"][s["row_token"][lo:hi].long() if c["gather"] else rows].to(F64)
            d = s["dz"][lo:hi].to(F64)
            out["dw"][e] = x.t() @ d
            if c["bias"]:
                out["db"][e] = d.sum(0)
        return out
    if op == "dx":
        dx = torch.zeros(R, K, dtype=F64, device=DEV)
        for e in range(E):
            dx[off[e]:off[e + 1]] = s["dz"][off[e]:off[e + 1]].to(F64) @ s["w"][e].to(F64).t()
        if not c["ckpt"]:
            return dict(dx=dx)
        a = torch.zeros(R, K, dtype=F64, device=DEV)
        a[:n] = f[:n]
        dx[:n] *= df[:n]
        return dict(dx=dx, a=a)
    z = torch.zeros(n, N, dtype=F64, device=DEV)
    for e in range(E):
        lo, hi = off[e], off[e + 1]
        if lo < hi:
            x = s["x"][s["row_token"][lo:hi].long()] if c["gather"] else s["x"][lo:hi]
            z[lo:hi] = x.to(F64) @ s["w"][e].to(F64)
            if c["bias"]:
                z[lo:hi] += s["bias"][e].to(F64)
    y = torch.zeros(R, N, dtype=F64, device=DEV)
    y[:n] = _exact_act(z, c["act"])[0]
    if c["residual"]:
        y[:n] += s["residual"][:n].to(F64)
    if not c["ckpt"]:
        return dict(y=y)
    codes = torch.zeros(R, N, dtype=F64, device=DEV)
    scales = torch.full((R, N // QB), 2.0 ** -127, dtype=F64, device=DEV)
    codes[:n], scales[:n] = _exact_blocks(z)
    return dict(y=y, codes=codes, scales=scales)
