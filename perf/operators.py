"""Timed cases of the dense operators around the MoE layer: the gated projection and its
gradients, the norms before and after a block and their gradients, and the product in
8-bit integers.

Each case is one pass through one operator (or through two that are used as a pair), in
its plain form in elementary torch operations, or through the library's entry points when
`own` is true.  Shapes: H = 6144, I = 2048 and 4096 tokens are the layer that bench.py runs;
the others are generic.
"""
import math

import torch

own = False
EPS = 1e-5
DEV = "cuda"


# ------------------------------------------------------------------------------ cases
def listed():
    return [
        # one token through an 8-bit projection: the shape of a decode step, latency counts
        {"name": "int8_T1", "op": "int8", "T": 1, "K": 6144, "N": 4096},
        # a few sequences decoding together, sizes off every tile border
        {"name": "int8_T37_ragged", "op": "int8", "T": 37, "K": 1552, "N": 2040},
        # a prefill batch through an 8-bit projection
        {"name": "int8_T4096", "op": "int8", "T": 4096, "K": 6144, "N": 6144},
        # decoding 64 sequences: the norm hands its rows to the product as 8-bit codes
        {"name": "norm_int8_T64", "op": "norm_int8", "T": 64, "K": 6144, "N": 4096},
        # serving: one token through the gate and up projections
        {"name": "gate_up_T1", "op": "gate_up", "T": 1, "H": 6144, "I": 2048, "act": "silu",
         "save": False},
        # training forward: the pre-activations are kept for the gradients
        {"name": "gate_up_T4096_train", "op": "gate_up", "T": 4096, "H": 6144, "I": 2048,
         "act": "silu", "save": True},
        # gradients of a ragged micro-batch of a small block, GELU gate
        {"name": "gate_up_bwd_T333_gelu", "op": "gate_up_bwd", "T": 333, "H": 1000, "I": 520,
         "act": "gelu"},
        # gradients of a training batch
        {"name": "gate_up_bwd_T4096", "op": "gate_up_bwd", "T": 4096, "H": 6144, "I": 2048,
         "act": "silu"},
        # decode: one row, the norm after a block, the residual sum and the next block's norm
        {"name": "post_norm_T1", "op": "post_norm", "T": 1, "H": 6144, "gate": "none",
         "next": True},
        # prefill of long prompts: the same over many rows with a gate for each channel
        {"name": "post_norm_T16384", "op": "post_norm", "T": 16384, "H": 6144, "gate": "h",
         "next": True},
        # training: the norm after a block with a gate for each token, forward and backward
        {"name": "post_norm_train_T4096", "op": "post_norm_train", "T": 4096, "H": 6144,
         "gate": "t"},
        # training: the norm before a block, forward and backward, an odd batch of short rows
        {"name": "pre_norm_train_T8191", "op": "pre_norm_train", "T": 8191, "H": 1032},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _mult(rng, lo, hi, m):
    return max(m, _log(rng, lo, hi) // m * m)


def draw(rng):
    op = rng.choice(["int8", "norm_int8", "gate_up", "gate_up_bwd", "post_norm",
                     "post_norm_train", "pre_norm_train"])
    T = _log(rng, 1, 4096)
    if op in ("int8", "norm_int8"):
        return {"op": op, "T": T, "K": _mult(rng, 64, 6144, 16), "N": _mult(rng, 64, 6144, 8)}
    if op in ("gate_up", "gate_up_bwd"):
        c = {"op": op, "T": T, "H": _mult(rng, 64, 6144, 8), "I": _mult(rng, 64, 2048, 8),
             "act": rng.choice(["silu", "gelu"])}
        if op == "gate_up":
            c["save"] = rng.choice([False, True])
        return c
    c = {"op": op, "T": _log(rng, 1, 16384) if op == "post_norm" else T,
         "H": _mult(rng, 64, 6144, 8)}
    if op != "pre_norm_train":
        c["gate"] = rng.choice(["none", "1", "t", "h", "th"])
    if op == "post_norm":
        c["next"] = rng.choice([False, True])
    return c


# ------------------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=DEV) * std + mean).to(torch.bfloat16)

    s = dict(case)
    T, op = case["T"], case["op"]
    if op in ("int8", "norm_int8"):
        K, N = case["K"], case["N"]
        # activations with a few channels far above the rest, as hidden states have
        s["x"] = normal(T, K)
        s["x"][:, torch.randint(0, K, (max(1, K // 256),), generator=g, device=DEV)] *= 8
        s["w"] = torch.randint(-127, 128, (N, K), generator=g, device=DEV, dtype=torch.int8)
        s["ws"] = torch.rand((N,), generator=g, device=DEV) * 4e-4 + 1e-4
        if op == "norm_int8":
            s["weight"] = normal(K, std=0.1, mean=1.0)
        return s
    H = case["H"]
    if op in ("gate_up", "gate_up_bwd"):
        I = case["I"]
        s["x"] = normal(T, H)
        s["w_gu"] = normal(2 * I, H, std=1.0 / math.sqrt(H))
        if op == "gate_up_bwd":
            # what the forward pass kept, and the gradient that comes from the layers above
            s["gu"] = torch.matmul(s["x"].float(), s["w_gu"].float().t()).to(torch.bfloat16)
            s["dh"] = normal(T, I, std=0.1)
        return s
    s["x"] = normal(T, H)
    s["x"] *= torch.rand((T, 1), generator=g, device=DEV).mul(2.0).add(0.25).to(torch.bfloat16)
    s["weight"] = normal(H, std=0.1, mean=1.0)
    if op == "pre_norm_train":
        s["dy"], s["dskip"] = normal(T, H, std=0.1), normal(T, H, std=0.1)
        return s
    shape = {"none": None, "1": (1, 1), "t": (T, 1), "h": (1, H), "th": (T, H)}[case["gate"]]
    s["g"] = None if shape is None else normal(*shape, std=0.25, mean=0.5)
    s["residual"] = normal(T, H)
    s["scale"] = 0.875
    if op == "post_norm":
        s["next_weight"] = normal(H, std=0.1, mean=1.0) if case["next"] else None
    else:
        s["dout"] = normal(T, H, std=0.1)
    return s


# ------------------------------------------------------------------------------ plain forms
def _norm(x):
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)


def _int8_product(x, w, ws):
    amax = x.abs().amax(-1, keepdim=True)
    codes = (x * 127 / torch.where(amax > 0, amax, torch.ones_like(amax))).round()
    scale = torch.where(amax > 0, amax / 127, torch.ones_like(amax))
    return (torch.matmul(codes, w.float().t()) * scale * ws).to(torch.bfloat16)


_C = math.sqrt(2.0 / math.pi)


def _act(z, act):
    if act == "silu":
        return z / (1 + torch.exp(-z))
    return 0.5 * z * (1 + torch.tanh(_C * (z + 0.044715 * z * z * z)))


def _act_slope(z, act):
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    t = torch.tanh(_C * (z + 0.044715 * z * z * z))
    return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _C * (1 + 3 * 0.044715 * z * z)


def _norm_grad(dn, n, x):
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return r * (dn - n * (dn * n).mean(-1, keepdim=True))


def _plain(s):
    op, bf = s["op"], torch.bfloat16
    x = s["x"].float()
    if op == "int8":
        return _int8_product(x, s["w"], s["ws"])
    if op == "norm_int8":
        return _int8_product(_norm(x) * s["weight"].float(), s["w"], s["ws"])
    if op == "gate_up":
        gu = torch.matmul(x, s["w_gu"].float().t())
        g, u = gu[:, : s["I"]], gu[:, s["I"]:]
        h = (_act(g, s["act"]) * u).to(bf)
        return {"h": h, "gu": gu.to(bf)} if s["save"] else {"h": h}
    if op == "gate_up_bwd":
        gu, dh = s["gu"].float(), s["dh"].float()
        g, u = gu[:, : s["I"]], gu[:, s["I"]:]
        dgu = torch.cat([dh * u * _act_slope(g, s["act"]), dh * _act(g, s["act"])], 1)
        return {"dx": torch.matmul(dgu, s["w_gu"].float()).to(bf),
                "dw_gu": torch.matmul(dgu.t(), x).to(bf)}
    w, n = s["weight"].float(), _norm(x)
    if op == "pre_norm_train":
        dy = s["dy"].float()
        return {"y": (n * w).to(bf),
                "dx": (s["dskip"].float() + _norm_grad(dy * w, n, x)).to(bf),
                "dweight": (dy * n).sum(0).to(bf)}
    g = 1.0 if s["g"] is None else s["g"].float()
    out = s["scale"] * s["residual"].float() + g * (w * n)
    if op == "post_norm":
        if s["next_weight"] is None:
            return {"out": out.to(bf)}
        return {"out": out.to(bf), "next": (_norm(out) * s["next_weight"].float()).to(bf)}
    dout = s["dout"].float()
    r = {"out": out.to(bf), "dy": _norm_grad(dout * g * w, n, x).to(bf),
         "dweight": (dout * g * n).sum(0).to(bf), "dresidual": (s["scale"] * dout).to(bf)}
    if s["g"] is not None:
        dims = [d for d in (0, 1) if s["g"].shape[d] == 1]
        dg = dout * w * n
        r["dgate"] = (dg.sum(dims, keepdim=True) if dims else dg).to(bf)
    return r


def run(state):
    if not own:
        return _plain(state)
    import bit_quantized_moe_nvfp4_b200 as nv
    s, op = state, state["op"]
    if op in ("int8", "norm_int8"):
        if op == "int8":
            codes, scales = nv.nvfp4_int8_quantize(s["x"])
        else:
            codes, scales = nv.moe_nvfp4_pre_norm_int8(s["x"], s["weight"], EPS)
        return nv.nvfp4_int8_matmul(codes, scales, s["w"], s["ws"])
    if op in ("gate_up", "gate_up_bwd"):
        act = nv.ACT_SILU if s["act"] == "silu" else nv.ACT_GELU
        if op == "gate_up_bwd":
            dx, dw = nv.moe_nvfp4_gate_up_backward(s["dh"], s["x"], s["w_gu"], s["gu"], act=act)
            return {"dx": dx, "dw_gu": dw}
        if not s["save"]:
            return {"h": nv.moe_nvfp4_gate_up(s["x"], s["w_gu"], act=act)}
        gu = torch.empty((s["T"], 2 * s["I"]), dtype=torch.bfloat16, device=DEV)
        return {"h": nv.moe_nvfp4_gate_up(s["x"], s["w_gu"], act=act, gu=gu), "gu": gu}
    if op == "pre_norm_train":
        y = nv.moe_nvfp4_pre_norm(s["x"], s["weight"], EPS)
        dx, dw = nv.moe_nvfp4_pre_norm_backward(s["dy"], s["x"], s["weight"], EPS,
                                                dskip=s["dskip"])
        return {"y": y, "dx": dx, "dweight": dw}
    if op == "post_norm":
        r = nv.moe_nvfp4_post_norm(s["x"], s["weight"], s["residual"], EPS, gate=s["g"],
                                   residual_scale=s["scale"], next_weight=s["next_weight"])
        return {"out": r} if s["next_weight"] is None else {"out": r[0], "next": r[1]}
    out = nv.moe_nvfp4_post_norm(s["x"], s["weight"], s["residual"], EPS, gate=s["g"],
                                 residual_scale=s["scale"])
    dy, dw, dg, dres = nv.moe_nvfp4_post_norm_backward(s["dout"], s["x"], s["weight"], EPS,
                                                       gate=s["g"], residual_scale=s["scale"])
    r = {"out": out, "dy": dy, "dweight": dw, "dresidual": dres}
    if dg is not None:
        r["dgate"] = dg
    return r


# ------------------------------------------------------------------------------ 64 bits
def exact(case, seed):
    """The operators' definitions in 64 bits, gradients by torch's differentiation."""
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float64

    def rms(v, weight):
        return weight.to(f8) * v / ((v ** 2).sum(-1, keepdim=True) / v.shape[-1] + EPS).sqrt()

    def eight_bits(v):
        top = v.abs().max(-1, keepdim=True).values
        step = top / 127
        q = torch.where(top > 0, torch.round(127 * v / top), torch.zeros_like(v))
        prod = torch.einsum("tk,nk->tn", q, s["w"].to(f8))
        return prod * torch.where(top > 0, step, torch.ones_like(step)) * s["ws"].to(f8)

    def gated(g, u):
        if case["act"] == "silu":
            return g * torch.special.expit(g) * u
        inner = (2 / math.pi) ** 0.5 * (g + 0.044715 * g ** 3)
        return g * (0.5 + 0.5 * torch.tanh(inner)) * u

    if op == "int8":
        return eight_bits(s["x"].to(f8))
    if op == "norm_int8":
        return eight_bits(rms(s["x"].to(f8), s["weight"]))
    if op == "gate_up":
        gu = torch.einsum("th,jh->tj", s["x"].to(f8), s["w_gu"].to(f8))
        r = {"h": gated(*gu.chunk(2, 1))}
        return dict(r, gu=gu) if case["save"] else r
    if op == "gate_up_bwd":
        gu = s["gu"].to(f8).requires_grad_()
        d, = torch.autograd.grad(gated(*gu.chunk(2, 1)), gu, s["dh"].to(f8))
        return {"dx": torch.einsum("tj,jh->th", d, s["w_gu"].to(f8)),
                "dw_gu": torch.einsum("tj,th->jh", d, s["x"].to(f8))}
    if op == "pre_norm_train":
        x, w = s["x"].to(f8).requires_grad_(), s["weight"].to(f8).requires_grad_()
        y = rms(x, w)
        dx, dw = torch.autograd.grad(y, (x, w), s["dy"].to(f8))
        return {"y": y.detach(), "dx": dx + s["dskip"].to(f8), "dweight": dw}
    leaves = [s["x"], s["weight"], s["residual"]] + ([] if s["g"] is None else [s["g"]])
    leaves = [t.to(f8).requires_grad_() for t in leaves]
    out = rms(leaves[0], leaves[1])
    if s["g"] is not None:
        out = out * leaves[3]
    out = out + s["scale"] * leaves[2]
    if op == "post_norm":
        r = {"out": out.detach()}
        if s["next_weight"] is not None:
            r["next"] = rms(out.detach(), s["next_weight"])
        return r
    d = torch.autograd.grad(out, leaves, s["dout"].to(f8))
    r = {"out": out.detach(), "dy": d[0], "dweight": d[1], "dresidual": d[2]}
    if s["g"] is not None:
        r["dgate"] = d[3]
    return r


# ------------------------------------------------------------------------------ work
def work(case):
    op, T = case["op"], case["T"]
    if op in ("int8", "norm_int8"):
        K, N = case["K"], case["N"]
        n = 2 * T * K + N * K + 4 * N + 2 * T * N
        return {"bytes": n + (2 * K if op == "norm_int8" else 0), "flops": 2 * T * N * K}
    H = case["H"]
    if op in ("gate_up", "gate_up_bwd"):
        I = case["I"]
        if op == "gate_up":
            return {"bytes": 2 * (T * H + 2 * I * H + T * I + (2 * T * I if case["save"] else 0)),
                    "flops": 4 * T * I * H}
        return {"bytes": 2 * (2 * T * H + 4 * I * H + 3 * T * I), "flops": 8 * T * I * H}
    if op == "pre_norm_train":      # x, dy, dskip read; y, dx written
        return {"bytes": 2 * (5 * T * H + 2 * H), "flops": 14 * T * H}
    gate = {"none": 0, "1": 1, "t": T, "h": H, "th": T * H}[case["gate"]]
    if op == "post_norm":
        n = 3 * T * H + H + gate + ((T * H + H) if case["next"] else 0)
        return {"bytes": 2 * n, "flops": (12 if case["next"] else 7) * T * H}
    # x, residual, dout read; out, dy, dresidual written
    return {"bytes": 2 * (6 * T * H + 2 * H + 2 * gate), "flops": 18 * T * H}
