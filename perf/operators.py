"""The dense feed-forward operators, as cases to measure.

Four operators of a transformer's linear layers, forward and backward, for
prompts, training batches and single tokens:

* ``linear``      y = act(x W^T + bias) + residual (and the pre-activation);
* ``linear_bwd``  its gradients: dx, dW^T and dbias;
* ``gated``       h = act(x Wg^T) * (x Wu^T) (and both projections g and u);
* ``gated_bwd``   its gradients: dx, dWg^T and dWu^T.

Weights are stored transposed, ``wt[d_in][d_out]``.  Sizes are those of the
Llama-2-7B layer (4096, 11008), the Llama-3-8B layer (4096, 14336; k/v
projection 4096 to 1024) and generic smaller ones.  With ``own`` false ``run``
computes the plain form in fp32; with ``own`` true it calls this package.
"""

from __future__ import annotations

import math

import torch

own = False

DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
ACTS = ("relu", "relu2", "silu", "gelu", "gelu_tanh")
DEVICE = "cuda"


def listed():
    def linear(name, t, d_in, d_out, dtype, **more):
        return {"name": name, "op": "linear", "t": t, "d_in": d_in, "d_out": d_out, "dtype": dtype,
                "act": "none", "bias": False, "residual": False, "pre": False, **more}

    def gated(name, t, d_in, d_out, dtype, **more):
        return {"name": name, "op": "gated", "t": t, "d_in": d_in, "d_out": d_out, "dtype": dtype,
                "act": "silu", "save": False, "side": False, **more}

    return [
        # one decoded token through the attention output projection, added to the residual
        linear("o, 1 token", 1, 4096, 4096, "fp16", residual=True),
        # eight sequences decoding together through the down projection
        linear("down, 8 tokens", 8, 11008, 4096, "bf16", residual=True),
        # a short prompt through a small biased projection (k or v with grouped queries)
        linear("kv, 33 tokens", 33, 4096, 1024, "fp16", bias=True),
        # a ragged prompt through a biased, activated up projection that keeps its pre-activation
        linear("up, 1000 tokens", 1000, 4096, 11008, "fp16", bias=True, act="gelu_tanh", pre=True),
        # a large prefill batch through the down projection
        linear("down, 8192 tokens", 8192, 14336, 4096, "bf16", residual=True),
        # a small training step of a biased squared-ReLU layer, a ragged batch
        linear("small layer backward", 509, 1024, 4096, "fp16", op="linear_bwd", bias=True, act="relu2"),
        # a training step of the biased, activated up projection
        linear("up backward", 4096, 4096, 11008, "bf16", op="linear_bwd", bias=True, act="gelu"),
        # one decoded token through gate and up
        gated("gate|up, 1 token", 1, 4096, 11008, "fp16"),
        # seventeen sequences decoding together, gate and up stored side by side
        gated("gate|up, 17 tokens", 17, 4096, 14336, "bf16", side=True),
        # a training batch's forward pass, which keeps both projections
        gated("gate|up, 8192 tokens", 8192, 4096, 14336, "bf16", save=True),
        # a small gated layer's training step, a ragged batch
        gated("small gated backward", 300, 1024, 4096, "fp16", op="gated_bwd"),
        # a training step of the Llama-2-7B gate and up projections, stored side by side
        gated("gate|up backward", 4096, 4096, 11008, "bf16", op="gated_bwd", side=True),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    op = rng.choice(("linear", "linear", "linear_bwd", "gated", "gated", "gated_bwd"))
    t = max(1, min(8192, int(_log(rng, 1, 8192))))
    if op.endswith("bwd"):
        t = max(2, t // 2)
    case = {"op": op, "t": t, "d_in": 8 * int(_log(rng, 32, 1024)), "d_out": 8 * int(_log(rng, 32, 1536)),
            "dtype": rng.choice(("fp16", "bf16"))}
    if op.startswith("linear"):
        case.update(act=rng.choice(("none",) + ACTS), bias=rng.random() < 0.5,
                    residual=op == "linear" and rng.random() < 0.5, pre=op == "linear" and rng.random() < 0.25)
    else:
        case.update(act=rng.choice(ACTS), save=op == "gated" and rng.random() < 0.3, side=rng.random() < 0.5)
    most = max(work(c)["flops"] for c in listed())
    case["t"] = max(1, min(t, int(t * most / work(case)["flops"])))
    return case


def prepare(case, seed):
    dt = DTYPES[case["dtype"]]
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)

    def normal(*shape, std=1.0):
        return (torch.randn(*shape, generator=gen, device=DEVICE) * std).to(dt)

    t, d_in, d_out, op = case["t"], case["d_in"], case["d_out"], case["op"]
    pre_std = 0.02 * math.sqrt(d_in)  # of x W^T for x ~ N(0, 1), W ~ N(0, 0.02)
    s = {"op": op, "act": case["act"], "x": normal(t, d_in)}
    if op.startswith("linear"):
        s["wt"] = normal(d_in, d_out, std=0.02)
        s["bias"] = normal(d_out, std=0.1) if case["bias"] else None
    else:
        if case["side"]:
            both = normal(d_in, 2 * d_out, std=0.02)
            s["wgt"], s["wut"] = both[:, :d_out], both[:, d_out:]
        else:
            s["wgt"], s["wut"] = normal(d_in, d_out, std=0.02), normal(d_in, d_out, std=0.02)
    if op == "linear":
        s["residual"] = normal(t, d_out) if case["residual"] else None
        s["with_pre"] = case["pre"]
    elif op == "linear_bwd":
        s["dy"] = normal(t, d_out, std=0.05)
        s["pre"] = normal(t, d_out, std=pre_std) if case["act"] != "none" else None
        s["with_dbias"] = case["bias"]
    elif op == "gated":
        s["with_gu"] = case["save"]
    else:
        s["dh"] = normal(t, d_out, std=0.05)
        s["g"], s["u"] = normal(t, d_out, std=pre_std), normal(t, d_out, std=pre_std)
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


def _plain(s):
    op, act, x = s["op"], s["act"], s["x"]
    dt = x.dtype
    xf = x.float()
    if op == "linear":
        pre = xf @ s["wt"].float()
        if s["bias"] is not None:
            pre = pre + s["bias"].float()
        y = _act(pre, act)
        if s["residual"] is not None:
            y = y + s["residual"].float()
        return {"y": y.to(dt), **({"pre": pre.to(dt)} if s["with_pre"] else {})}
    if op == "linear_bwd":
        d = s["dy"].float()
        if s["pre"] is not None:
            d = d * _slope(s["pre"].float(), act)
        out = {"dx": (d @ s["wt"].float().t()).to(dt), "dwt": (xf.t() @ d).to(dt)}
        if s["with_dbias"]:
            out["dbias"] = d.sum(0).to(dt)
        return out
    if op == "gated":
        g, u = xf @ s["wgt"].float(), xf @ s["wut"].float()
        h = _act(g, act) * u
        return {"h": h.to(dt), **({"g": g.to(dt), "u": u.to(dt)} if s["with_gu"] else {})}
    dh, g, u = s["dh"].float(), s["g"].float(), s["u"].float()
    dg, du = dh * u * _slope(g, act), dh * _act(g, act)
    dx = dg @ s["wgt"].float().t() + du @ s["wut"].float().t()
    return {"dx": dx.to(dt), "dwgt": (xf.t() @ dg).to(dt), "dwut": (xf.t() @ du).to(dt)}


# ---- the package's operators ------------------------------------------------------

def _own(s):
    import sparse_input_gemv_amd as sa

    op = s["op"]
    if op == "linear":
        got = sa.dense_linear(s["x"], s["wt"], bias=s["bias"], act=s["act"], residual=s["residual"],
                              with_pre=s["with_pre"])
        return {"y": got[0], "pre": got[1]} if s["with_pre"] else {"y": got}
    if op == "linear_bwd":
        dx, dwt, dbias = sa.dense_linear_backward(s["dy"], s["x"], s["wt"], act=s["act"], pre=s["pre"],
                                                  with_dbias=s["with_dbias"])
        return {"dx": dx, "dwt": dwt, **({"dbias": dbias} if s["with_dbias"] else {})}
    if op == "gated":
        got = sa.gated_linear(s["x"], s["wgt"], s["wut"], act=s["act"], with_gu=s["with_gu"])
        return {"h": got[0], "g": got[1], "u": got[2]} if s["with_gu"] else {"h": got}
    dx, dwgt, dwut = sa.gated_linear_backward(s["dh"], s["x"], s["wgt"], s["wut"], s["g"], s["u"], act=s["act"])
    return {"dx": dx, "dwgt": dwgt, "dwut": dwut}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    """What one pass cannot do without: every input read and every output
    written once (two bytes a value), and the products' operations."""
    t, d_in, d_out, op = case["t"], case["d_in"], case["d_out"], case["op"]
    x, w, o = t * d_in, d_in * d_out, t * d_out
    if op == "linear":
        values = x + w + o * (1 + case["residual"] + case["pre"]) + d_out * case["bias"]
        products = 1
    elif op == "linear_bwd":
        values = o * (1 + (case["act"] != "none")) + x + w + x + w + d_out * case["bias"]
        products = 2
    elif op == "gated":
        values = x + 2 * w + o * (3 if case["save"] else 1)
        products = 2
    else:
        values = 3 * o + x + 2 * w + x + 2 * w
        products = 4
    return {"bytes": 2 * values, "flops": 2 * products * t * d_in * d_out}


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
    s = {k: v.double() if isinstance(v, torch.Tensor) else v for k, v in prepare(case, seed).items()}
    kind = s["act"]
    if case["op"] == "linear":
        z = torch.mm(s["x"], s["wt"])
        if case["bias"]:
            z += s["bias"][None, :]
        y = _fn64(kind, z)[0]
        res = {"y": y + s["residual"] if case["residual"] else y}
        if case["pre"]:
            res["pre"] = z
        return res
    if case["op"] == "linear_bwd":
        dz = s["dy"] if kind == "none" else s["dy"] * _fn64(kind, s["pre"])[1]
        res = {"dx": torch.mm(dz, s["wt"].T), "dwt": torch.mm(s["x"].T, dz)}
        if case["bias"]:
            res["dbias"] = torch.mv(dz.T, torch.ones(dz.shape[0], dtype=dz.dtype, device=dz.device))
        return res
    if case["op"] == "gated":
        g, u = torch.mm(s["x"], s["wgt"]), torch.mm(s["x"], s["wut"])
        res = {"h": _fn64(kind, g)[0] * u}
        return {**res, "g": g, "u": u} if case["save"] else res
    f, df = _fn64(kind, s["g"])
    dg, du = s["dh"] * s["u"] * df, s["dh"] * f
    return {"dx": torch.mm(dg, s["wgt"].T).addmm_(du, s["wut"].T),
            "dwgt": torch.mm(s["x"].T, dg), "dwut": torch.mm(s["x"].T, du)}
