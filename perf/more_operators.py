"""Linear layers in 8-bit integers and linear layers grouped by expert, as
cases to measure.

* ``quantise``     symmetric 8-bit integers with a scale per token, or per
                   output channel of a transposed weight (which it transposes);
* ``int8``         y = act(sx sw (xq Wq^T) + bias) + residual from 16-bit
                   activations (quantised within the call) or 8-bit ones;
* ``grouped``      rows offsets[e] .. offsets[e + 1] - 1 through expert e's
                   projection: y = act(x We^T + be) + residual, or the gated
                   pair h = act(x Wge^T) * (x Wue^T);
* ``grouped_bwd``  the gradients of either: dx, every expert's weights' and
                   biases'.

Expert weights are ``wt[e][d_in][d_out]``, 8-bit weights ``wq[d_out][d_in]``.
Sizes are those of the Llama-2-7B layer (4096, 11008), the Llama-3-8B layer
(4096, 14336; k/v projection 4096 to 1024) and generic smaller ones.  Rows per
expert are ragged, as a router leaves them, and some experts have none.  With
``own`` false ``run`` computes the plain form in fp32 (quotients in fp64);
with ``own`` true it calls this package.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("relu", "relu2", "silu", "gelu", "gelu_tanh")
DEVICE = "cuda"


def listed():
    def quantise(name, t, d, dtype, kind):
        return {"name": name, "op": "quantise", "t": t, "d_in": d, "d_out": 0, "dtype": dtype, "kind": kind}

    def int8(name, t, d_in, d_out, dtype, **more):
        return {"name": name, "op": "int8", "t": t, "d_in": d_in, "d_out": d_out, "dtype": dtype,
                "act": "none", "bias": False, "residual": False, "quantised": False, **more}

    def grouped(name, t, e, d_in, d_out, dtype, **more):
        return {"name": name, "op": "grouped", "t": t, "e": e, "d_in": d_in, "d_out": d_out, "dtype": dtype,
                "act": "none", "gated": False, "bias": False, "residual": False, "save": False, "spare": 0, **more}

    return [
        # eight decoding sequences' input of an 8-bit projection
        quantise("quantise 8 tokens", 8, 4096, "fp16", "token"),
        # a training or prefill batch's hidden activations
        quantise("quantise 8192 tokens", 8192, 14336, "bf16", "token"),
        # a checkpoint's down projection, quantised when it is loaded
        quantise("quantise a weight", 11008, 4096, "fp16", "channel"),
        # one decoded token through an up projection
        int8("int8 up, 1 token", 1, 4096, 11008, "fp16"),
        # thirty-three sequences decoding together through the down projection
        int8("int8 down, 33 tokens", 33, 11008, 4096, "bf16", residual=True),
        # a prefill batch of 8-bit activations through a biased, activated up projection
        int8("int8 up, 8192 tokens", 8192, 4096, 14336, "bf16", bias=True, act="silu", quantised=True),
        # eight sequences decoding together, two of eight experts each: gate and up, room for more rows
        grouped("experts gate|up, 16 rows", 16, 8, 4096, 14336, "bf16", gated=True, act="silu", spare=5),
        # a short prompt through many small biased, activated experts
        grouped("64 small experts, 1000 rows", 1000, 64, 1024, 4096, "fp16", bias=True, act="gelu"),
        # a training batch's gate and up, both projections kept
        grouped("experts gate|up, 4096 rows", 4096, 8, 4096, 11008, "bf16", gated=True, act="silu", save=True),
        # a prefill batch through the experts' down projections
        grouped("experts down, 8192 rows", 8192, 8, 14336, 4096, "bf16"),
        # a small training step of biased squared-ReLU experts
        grouped("small experts backward", 509, 16, 1024, 4096, "fp16", op="grouped_bwd", bias=True, act="relu2"),
        # a training step of the gated experts
        grouped("experts gate|up backward", 4096, 8, 4096, 11008, "bf16", op="grouped_bwd", gated=True, act="silu"),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    op = rng.choice(("quantise", "int8", "int8", "grouped", "grouped", "grouped", "grouped_bwd", "grouped_bwd"))
    t = max(1, min(8192, int(_log(rng, 1, 8192))))
    dtype = rng.choice(("fp16", "bf16"))
    if op == "quantise":
        kind = rng.choice(("token", "token", "channel"))
        if kind == "channel":
            return {"op": op, "t": 16 * int(_log(rng, 16, 700)), "d_in": 8 * int(_log(rng, 32, 1700)), "d_out": 0,
                    "dtype": dtype, "kind": kind}
        return {"op": op, "t": t, "d_in": 16 * int(_log(rng, 16, 900)), "d_out": 0, "dtype": dtype, "kind": kind}
    if op == "int8":
        case = {"op": op, "t": t, "d_in": 16 * int(_log(rng, 16, 900)), "d_out": 8 * int(_log(rng, 32, 1700)),
                "dtype": dtype, "act": rng.choice(("none",) + ACTS), "bias": rng.random() < 0.5,
                "residual": rng.random() < 0.5, "quantised": rng.random() < 0.5}
    else:
        gated = rng.random() < 0.5
        back = op == "grouped_bwd"
        d_in, d_out = 8 * int(_log(rng, 32, 1024)), 8 * int(_log(rng, 32, 1400))
        most = max(1, min(128, int(5e8 / (d_in * d_out * (1 + gated)))))  # a gigabyte of weights
        case = {"op": op, "t": max(2, t // 2) if back else t, "e": max(1, int(_log(rng, 1, most + 1))),
                "d_in": d_in, "d_out": d_out, "dtype": dtype,
                "act": rng.choice(ACTS) if gated else rng.choice(("none",) + ACTS), "gated": gated,
                "bias": not gated and rng.random() < 0.5,
                "residual": not gated and not back and rng.random() < 0.5,
                "save": not back and rng.random() < 0.3, "spare": rng.choice((0, 0, 3, 100))}
    top = max(work(c)["flops"] for c in listed() if c["op"] == op)
    case["t"] = max(1, min(case["t"], int(case["t"] * top / work(case)["flops"])))
    return case


def _generator(seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    return gen


def _offsets(t, e, gen):
    """Rows per expert as a router's skewed choice leaves them, and their
    largest number, which sizes the plain form's batches."""
    liking = torch.randn(e, generator=gen, device=DEVICE) * 0.7
    noise = torch.rand(t, e, generator=gen, device=DEVICE).clamp_(1e-9, 1 - 1e-7)
    chosen = (liking - torch.log(-torch.log(noise))).argmax(1)
    counts = torch.zeros(e, dtype=torch.int64, device=DEVICE)
    counts.scatter_add_(0, chosen, torch.ones_like(chosen))
    off = torch.zeros(e + 1, dtype=torch.int32, device=DEVICE)
    off[1:] = counts.cumsum(0)
    return off, int(counts.max())


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    gen = _generator(seed)

    def normal(*shape, std=1.0):
        out = torch.empty(shape, dtype=dt, device=DEVICE)
        return out.normal_(0.0, std, generator=gen)

    def spiky(*shape):  # activations with a few large channels
        x = torch.randn(*shape, generator=gen, device=DEVICE)
        loud = torch.rand(shape[-1], generator=gen, device=DEVICE) < 0.005
        return (x * torch.where(loud, 12.0, 1.0)).to(dt)

    t, d_in, d_out, op = case["t"], case["d_in"], case["d_out"], case["op"]
    if op == "quantise":
        if case["kind"] == "token":
            return {"op": op, "kind": "token", "x": spiky(t, d_in)}
        return {"op": op, "kind": "channel", "x": normal(t, d_in, std=0.02)}
    if op == "int8":
        s = {"op": op, "act": case["act"], "x": spiky(t, d_in), "sx": None, "dtype": dt,
             "wq": torch.randint(-127, 128, (d_out, d_in), generator=gen, device=DEVICE, dtype=torch.int8),
             "sw": (1 + torch.rand(d_out, generator=gen, device=DEVICE)) * (0.02 / 110),
             "bias": normal(d_out, std=0.1) if case["bias"] else None,
             "residual": normal(t, d_out) if case["residual"] else None}
        if case["quantised"]:
            s["x"], s["sx"] = _codes64(s["x"])
        return s
    e, room, gated = case["e"], t + case["spare"], case["gated"]
    s = {"op": op, "act": case["act"], "gated": gated, "x": normal(room, d_in)}
    s["offsets"], s["most"] = _offsets(t, e, gen)
    pre_std = 0.02 * math.sqrt(d_in)  # of x W^T for x ~ N(0, 1), W ~ N(0, 0.02)
    for k in ("wgt", "wut") if gated else ("wt",):
        s[k] = normal(e, d_in, d_out, std=0.02)
    # rows that no expert takes keep what these hold
    if op == "grouped":
        s["save"] = case["save"]
        s["bias"] = normal(e, d_out, std=0.1) if case["bias"] else None
        s["residual"] = normal(room, d_out) if case["residual"] else None
        for k in (("y",) if not gated else ("h",)) + (() if not case["save"] else ("g", "u") if gated else ("pre",)):
            s[k] = torch.zeros(room, d_out, dtype=dt, device=DEVICE)
        return s
    s["bias"] = case["bias"]
    s["dx"] = torch.zeros(room, d_in, dtype=dt, device=DEVICE)
    s["dy"] = normal(room, d_out, std=0.05)
    if gated:
        s["g"], s["u"] = normal(room, d_out, std=pre_std), normal(room, d_out, std=pre_std)
    else:
        s["pre"] = normal(room, d_out, std=pre_std) if case["act"] != "none" else None
    return s


# ---- the plain forms ------------------------------------------------------------

C_TANH = math.sqrt(2.0 / math.pi)


def _act(v, act):
    if act == "none":
        return v
    if act == "relu":
        return torch.where(v > 0, v, 0.0)
    if act == "relu2":
        return torch.where(v > 0, v * v, 0.0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    return 0.5 * v * (1 + torch.tanh(C_TANH * (v + 0.044715 * v * v * v)))


def _slope(v, act):
    if act == "none":
        return torch.ones_like(v)
    if act == "relu":
        return torch.where(v > 0, 1.0, 0.0)
    if act == "relu2":
        return torch.where(v > 0, 2 * v, 0.0)
    if act == "silu":
        s = 1 / (1 + torch.exp(-v))
        return s * (1 + v * (1 - s))
    if act == "gelu":
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) * (0.5 * math.sqrt(2 / math.pi))
    th = torch.tanh(C_TANH * (v + 0.044715 * v * v * v))
    return 0.5 * (1 + th) + 0.5 * v * (1 - th * th) * C_TANH * (1 + 3 * 0.044715 * v * v)


def _codes64(x):
    """8-bit codes and scales of x's rows.  The scale is the fp32 quotient; a
    product by the reciprocal of 127 may differ from it, and a value's quotient
    may lie next to half a step, so both are taken in fp64."""
    s = (x.float().abs().amax(1).double() / 127).float()
    by = torch.where(s > 0, s, 1.0).double()
    return torch.round(x.double() / by[:, None]).clamp(-127, 127).to(torch.int8), s


def _slots(s):
    """Each expert's rows, its slots past them, and which slots are rows:
    [experts][most rows of one]."""
    off = s["offsets"].long()
    row = off[:-1, None] + torch.arange(s["most"], device=off.device)[None]
    return row, row < off[1:, None]


def _by_expert(v, row, there):
    """v's rows as fp32 batches [experts][most][columns], zeros past each end."""
    return torch.where(there[..., None], v.float()[row.clamp(max=v.shape[0] - 1)], 0.0)


def _rows_of(b, row, there, out):
    """The batches' rows in their places of a matrix like `out`, zeros elsewhere."""
    flat = torch.zeros(out.shape[0] + 1, out.shape[1], dtype=torch.float32, device=b.device)
    flat[torch.where(there, row, out.shape[0]).reshape(-1)] = b.reshape(-1, b.shape[-1])
    return flat[:-1].to(out.dtype)


def _plain_grouped(s):
    row, there = _slots(s)
    x, act = _by_expert(s["x"], row, there), s["act"]
    if s["gated"]:
        g, u = torch.bmm(x, s["wgt"].float()), torch.bmm(x, s["wut"].float())
        out = {"h": _rows_of(_act(g, act) * u, row, there, s["h"])}
        if s["save"]:
            out.update(g=_rows_of(g, row, there, s["g"]), u=_rows_of(u, row, there, s["u"]))
        return out
    pre = torch.bmm(x, s["wt"].float())
    if s["bias"] is not None:
        pre = pre + s["bias"].float()[:, None]
    y = _act(pre, act)
    if s["residual"] is not None:
        y = y + _by_expert(s["residual"], row, there)
    out = {"y": _rows_of(y, row, there, s["y"])}
    if s["save"]:
        out["pre"] = _rows_of(pre, row, there, s["pre"])
    return out


def _plain_grouped_bwd(s):
    row, there = _slots(s)
    dt, act = s["x"].dtype, s["act"]
    xt = _by_expert(s["x"], row, there).transpose(1, 2).contiguous()
    d = _by_expert(s["dy"], row, there)

    def times_w(v, w):  # v W of each expert
        return torch.bmm(v, w.float().transpose(1, 2).contiguous())

    if s["gated"]:
        g, u = _by_expert(s["g"], row, there), _by_expert(s["u"], row, there)
        dg, du = d * u * _slope(g, act), d * _act(g, act)
        dx = times_w(dg, s["wgt"]) + times_w(du, s["wut"])
        return {"dx": _rows_of(dx, row, there, s["dx"]), "dwgt": torch.bmm(xt, dg).to(dt), "dwut": torch.bmm(xt, du).to(dt)}
    if s["pre"] is not None:
        d = d * _slope(_by_expert(s["pre"], row, there), act)
    out = {"dx": _rows_of(times_w(d, s["wt"]), row, there, s["dx"]), "dwt": torch.bmm(xt, d).to(dt)}
    if s["bias"]:
        out["dbias"] = d.sum(1).to(dt)
    return out


def _plain(s):
    if s["op"] == "quantise":
        q, scale = _codes64(s["x"] if s["kind"] == "token" else s["x"].t().contiguous())
        return {"q": q, "s": scale}
    if s["op"] == "grouped":
        return _plain_grouped(s)
    if s["op"] == "grouped_bwd":
        return _plain_grouped_bwd(s)
    q, sx = (s["x"], s["sx"]) if s["sx"] is not None else _codes64(s["x"])
    y = (q.float() @ s["wq"].float().t()) * sx[:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    y = _act(y, s["act"])
    if s["residual"] is not None:
        y = y + s["residual"].float()
    return {"y": y.to(s["dtype"])}


# ---- the package's operators ------------------------------------------------------

def _own(s):
    import sparse_input_gemv_amd as sa

    op = s["op"]
    if op == "quantise":
        q, scale = sa.act_quantize_int8(s["x"]) if s["kind"] == "token" else sa.weight_quantize_int8(s["x"])
        return {"q": q, "s": scale}
    if op == "int8":
        return {"y": sa.int8_linear(s["x"], s["wq"], s["sw"], sx=s["sx"], bias=s["bias"], act=s["act"],
                                    residual=s["residual"], dtype=s["dtype"])}
    if op == "grouped" and s["gated"]:
        if not s["save"]:
            return {"h": sa.grouped_gated_linear(s["x"], s["wgt"], s["wut"], s["offsets"], act=s["act"], h=s["h"])}
        h, g, u = sa.grouped_gated_linear(s["x"], s["wgt"], s["wut"], s["offsets"], act=s["act"], h=s["h"],
                                          g=s["g"], u=s["u"])
        return {"h": h, "g": g, "u": u}
    if op == "grouped":
        got = sa.grouped_linear(s["x"], s["wt"], s["offsets"], bias=s["bias"], act=s["act"],
                                residual=s["residual"], y=s["y"], pre=s["pre"] if s["save"] else None)
        return {"y": got[0], "pre": got[1]} if s["save"] else {"y": got}
    if s["gated"]:
        dx, dwgt, dwut = sa.grouped_gated_linear_backward(s["dy"], s["x"], s["wgt"], s["wut"], s["offsets"],
                                                          s["g"], s["u"], act=s["act"], dx=s["dx"])
        return {"dx": dx, "dwgt": dwgt, "dwut": dwut}
    dx, dwt, dbias = sa.grouped_linear_backward(s["dy"], s["x"], s["wt"], s["offsets"], act=s["act"],
                                                pre=s["pre"], with_dbias=s["bias"], dx=s["dx"])
    return {"dx": dx, "dwt": dwt, **({"dbias": dbias} if s["bias"] else {})}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """What one pass cannot do without: every input read and every output
    written once, and the products' operations.  Of the experts' weights a
    forward pass reads those of experts with rows: the expected number of
    them for an even choice, at most the rows."""
    t, d_in, d_out, op = case["t"], case["d_in"], case["d_out"], case["op"]
    if op == "quantise":
        return {"bytes": 3 * t * d_in + 4 * (t if case["kind"] == "token" else d_in), "flops": 2 * t * d_in}
    x, o = t * d_in, t * d_out
    if op == "int8":
        read = x * (1 if case["quantised"] else 2) + 4 * t * case["quantised"] + d_in * d_out + 4 * d_out
        return {"bytes": read + 2 * (o * (1 + case["residual"]) + d_out * case["bias"]), "flops": 2 * t * d_in * d_out}
    e, pair = case["e"], 2 if case["gated"] else 1
    w = pair * d_in * d_out
    used = e * (1 - (1 - 1 / e) ** t)
    if op == "grouped":
        outs = (1 + 2 * case["save"] if case["gated"] else 1 + case["save"] + case["residual"]) * o
        return {"bytes": 2 * (x + used * (w + d_out * case["bias"]) + outs) + 4 * (e + 1),
                "flops": 2 * pair * t * d_in * d_out}
    reads = (3 if case["gated"] else 1 + (case["act"] != "none")) * o + x + used * w
    return {"bytes": 2 * (reads + x + e * (w + d_out * case["bias"])) + 4 * (e + 1),
            "flops": 4 * pair * t * d_in * d_out}


# ---- the definition in 64 bits ------------------------------------------------------

def _fn64(kind, z):
    """(f(z), f'(z)) of an activation, by its definition, in fp64."""
    one = torch.ones_like(z)
    if kind == "none":
        return z, one
    if kind in ("relu", "relu2"):
        p = z.clamp(min=0)
        return (p, (z > 0).to(z.dtype)) if kind == "relu" else (p.square(), 2 * p)
    if kind == "silu":
        sg = torch.reciprocal(one + (-z).exp())
        return z * sg, sg + z * sg * (one - sg)
    if kind == "gelu":
        cdf = torch.erfc(-z / math.sqrt(2.0)) / 2
        pdf = (-z.square() / 2).exp() / math.sqrt(2.0 * math.pi)
        return z * cdf, cdf + z * pdf
    a = math.sqrt(2.0 / math.pi) * (z + 0.044715 * z.pow(3))
    da = math.sqrt(2.0 / math.pi) * (one + 0.134145 * z.square())
    # (1 + tanh a) / 2 is the logistic function of 2a
    lg = torch.reciprocal(one + (-2 * a).exp())
    return z * lg, lg + z * 2 * lg * (one - lg) * da


def exact(case, seed):
    s = prepare(case, seed)
    kind, op = case.get("act"), case["op"]
    if op == "quantise":
        # whole numbers: the largest magnitude through the stored scale
        rows = s["x"].double() if case["kind"] == "token" else s["x"].double().T
        scale = (rows.abs().max(dim=1).values / 127.0).float()  # the fp32 quotient: 127 and a 16-bit value fit fp64
        q = (rows / scale.double().masked_fill(scale == 0, 1.0).unsqueeze(1)).round()
        return {"q": q.to(torch.int8), "s": scale.double()}
    if op == "int8":
        q, sx = s["x"].double(), s["sx"]
        if not case["quantised"]:
            sx = (q.abs().max(dim=1).values / 127.0).float()
            q = (q / sx.double().masked_fill(sx == 0, 1.0).unsqueeze(1)).round()
        z = torch.mm(q, s["wq"].double().T).mul_(torch.outer(sx.double(), s["sw"].double()))
        if case["bias"]:
            z += s["bias"].double()
        y = _fn64(kind, z)[0]
        return {"y": y + s["residual"].double() if case["residual"] else y}
    ends = s["offsets"].tolist()
    parts = [slice(a, b) for a, b in zip(ends, ends[1:])]
    room, d_in, d_out = s["x"].shape[0], case["d_in"], case["d_out"]

    def nothing(*shape):
        return torch.zeros(shape, dtype=torch.float64, device=DEVICE)

    if op == "grouped":
        names = (["h"] + ["g", "u"] * case["save"]) if case["gated"] else (["y"] + ["pre"] * case["save"])
        res = {k: nothing(room, d_out) for k in names}
        for e, rows in enumerate(parts):
            x = s["x"][rows].double()
            if case["gated"]:
                g, u = x @ s["wgt"][e].double(), x @ s["wut"][e].double()
                found = {"h": _fn64(kind, g)[0] * u, "g": g, "u": u}
            else:
                z = x @ s["wt"][e].double()
                z = z + s["bias"][e].double() if case["bias"] else z
                y = _fn64(kind, z)[0]
                found = {"y": y + s["residual"][rows].double() if case["residual"] else y, "pre": z}
            for k in names:
                res[k][rows] = found[k]
        return res
    pairs = (("dwgt", "wgt"), ("dwut", "wut")) if case["gated"] else (("dwt", "wt"),)
    res = {"dx": nothing(room, d_in), **{k: nothing(case["e"], d_in, d_out) for k, _ in pairs}}
    if case["bias"]:
        res["dbias"] = nothing(case["e"], d_out)
    for e, rows in enumerate(parts):
        x, dy = s["x"][rows].double(), s["dy"][rows].double()
        if case["gated"]:
            f, df = _fn64(kind, s["g"][rows].double())
            ds = (dy * s["u"][rows].double() * df, dy * f)
        else:
            ds = (dy if kind == "none" else dy * _fn64(kind, s["pre"][rows].double())[1],)
        for (dk, wk), d in zip(pairs, ds):
            res["dx"][rows] += d @ s[wk][e].double().T
            res[dk][e] = x.T @ d
        if case["bias"]:
            res["dbias"][e] = ds[0].sum(0)
    return res
