"""Operators for serving with few tokens: what is measured, on which cases.

Four operators, each in its plain form (elementary torch operations in 32 bits, the
router's logits in 64, rounded once) and as a user calls the library:

  route      w, ids = top-k of softmax(x Wr^T) over E experts, per token
  moe        y = sum over a token's k experts of w_e (SiLU(x Wg_e^T) * (x Wu_e^T)) Wd_e^T, router included,
             with the experts' weights in bf16, fp16, fp32 or 4 bits
  w4_linear  y = x W^T with W held as 4-bit codes, a scale (and a zero point) for each group along K
  mlp_w4     y = (SiLU(x Wg^T) * (x Wu^T)) Wd^T with all three weights in that form

Weights are in the nn.Linear layout (out_features x in_features, row-major). A 4-bit weight is
W[n, k] = scale[n, k / g] * (code[n, k] - zero[n, k / g]), codes 0..15, two to a byte, the even k in
the low half; without zero points, zero = 8.
"""

import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decoded token through a router of 64 experts: latency
        {"name": "route_1", "op": "route", "dtype": "bf16", "T": 1, "E": 64, "k": 8, "D": 2048, "renorm": True},
        # a long prompt's tokens through a wide router, weights not renormalised
        {"name": "route_8192", "op": "route", "dtype": "fp16", "T": 8192, "E": 128, "k": 8, "D": 4096, "renorm": False},
        # one decoded token, 2 of 8 experts of the small configuration: the smallest layer call
        {"name": "moe_1", "op": "moe", "dtype": "bf16", "w4": False, "T": 1, "E": 8, "k": 2, "D": 1024, "H": 2816,
         "renorm": True, "group": 0, "zeros": False},
        # a batch of 16 decoding sequences over many fine experts
        {"name": "moe_16_fine", "op": "moe", "dtype": "bf16", "w4": False, "T": 16, "E": 64, "k": 8, "D": 2048, "H": 1408,
         "renorm": False, "group": 0, "zeros": False},
        # odd sizes: no dimension fills the matrix cores' blocks
        {"name": "moe_37_ragged", "op": "moe", "dtype": "fp16", "w4": False, "T": 37, "E": 20, "k": 3, "D": 1000, "H": 712,
         "renorm": True, "group": 0, "zeros": False},
        # a batch of 64 over 8 large experts: the largest
        {"name": "moe_64_large", "op": "moe", "dtype": "bf16", "w4": False, "T": 64, "E": 8, "k": 2, "D": 4096, "H": 11008,
         "renorm": True, "group": 0, "zeros": False},
        # the IEEE fp32 mode
        {"name": "moe_5_fp32", "op": "moe", "dtype": "fp32", "w4": False, "T": 5, "E": 16, "k": 4, "D": 1024, "H": 704,
         "renorm": True, "group": 0, "zeros": False},
        # the fine experts in 4 bits
        {"name": "moe_8_w4", "op": "moe", "dtype": "bf16", "w4": True, "T": 8, "E": 64, "k": 8, "D": 2048, "H": 1408,
         "renorm": True, "group": 128, "zeros": False},
        # a projection of one decoded token
        {"name": "w4_1", "op": "w4_linear", "dtype": "bf16", "T": 1, "N": 4096, "K": 4096, "group": 128, "zeros": False},
        # speculative or batched decoding, small groups with zero points
        {"name": "w4_33", "op": "w4_linear", "dtype": "fp16", "T": 33, "N": 11008, "K": 4096, "group": 64, "zeros": True},
        # a dense block of the large configuration, one decoded token
        {"name": "mlp_w4_1", "op": "mlp_w4", "dtype": "bf16", "T": 1, "D": 4096, "H": 11008, "group": 128, "zeros": False},
        # a batch of 16 through the middle configuration, the smallest groups
        {"name": "mlp_w4_16", "op": "mlp_w4", "dtype": "fp16", "T": 16, "D": 2048, "H": 5632, "group": 32, "zeros": True},
    ]


def _log(rng, lo, hi, step=1):
    """A whole number in [lo, hi], spread over its logarithm, a multiple of step."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = min(hi // step * step, max(-(-lo // step) * step, round(v / step) * step))
    return v - step if v == 3072 else v  # no configuration here has that width


def draw(rng):
    op = rng.choice(["route", "moe", "moe", "w4_linear", "mlp_w4"])
    if op == "route":
        E = _log(rng, 4, 256)
        return {"op": op, "dtype": rng.choice(["bf16", "fp16", "fp32"]), "T": _log(rng, 1, 8192), "E": E,
                "k": rng.randint(1, min(8, E)), "D": _log(rng, 512, 4096, 8), "renorm": rng.random() < 0.5}
    if op == "moe":
        E = _log(rng, 4, 128)
        k = rng.randint(1, min(8, E))
        w4 = rng.random() < 0.4
        dtype = rng.choice(["bf16", "fp16"] if w4 else ["bf16", "bf16", "fp16", "fp16", "fp32"])
        group = rng.choice([32, 64, 128]) if w4 else 0
        D = _log(rng, 512, 4096, group or 8)
        # the experts of one layer stay below about 1.5 GB as 16-bit numbers
        H = _log(rng, 256, max(256, min(4096, 250_000_000 // (E * D))), group or 8)
        return {"op": op, "dtype": dtype, "w4": w4, "T": _log(rng, 1, 64), "E": E, "k": k, "D": D, "H": H,
                "renorm": rng.random() < 0.5, "group": group, "zeros": w4 and rng.random() < 0.5}
    group = rng.choice([32, 64, 128])
    zeros = rng.random() < 0.5
    dtype = rng.choice(["bf16", "fp16"])
    if op == "w4_linear":
        return {"op": op, "dtype": dtype, "T": _log(rng, 1, 64), "N": _log(rng, 256, 11008, 8),
                "K": _log(rng, 512, 11008, group), "group": group, "zeros": zeros}
    return {"op": op, "dtype": dtype, "T": _log(rng, 1, 64), "D": _log(rng, 1024, 4096, group),
            "H": _log(rng, 2048, 11008, group), "group": group, "zeros": zeros}


# ---- inputs -----------------------------------------------------------------


def _generator(seed):
    return torch.Generator(device=DEVICE).manual_seed(seed)


def _normal(gen, shape, scale, dtype):
    return (torch.randn(shape, generator=gen, device=DEVICE) * scale).to(dtype)


def _tokens(gen, T, D, dtype):
    # tokens share a direction, so a router favours some experts
    return (torch.randn((T, D), generator=gen, device=DEVICE) + 0.5 * torch.randn((1, D), generator=gen, device=DEVICE)).to(dtype)


def _quantised(gen, shape, group, zeros, dtype):
    """(codes [.., N, K/2], scales [.., N, K/g], zeros or None) of normal weights of variance 1/K."""
    *lead, K = shape
    w = torch.randn(shape, generator=gen, device=DEVICE) / math.sqrt(K)
    w = w.view(*lead, K // group, group)
    if zeros:
        lo, hi = w.amin(-1).clamp(max=0), w.amax(-1).clamp(min=0)
        scale = ((hi - lo) / 15).to(dtype)
        zero = (-lo / scale.float()).round().clamp(0, 15)
    else:
        scale = (w.abs().amax(-1) / 7.5).to(dtype)
        zero = torch.full_like(scale, 8, dtype=torch.float32)
    q = (w / scale.float()[..., None] + zero[..., None]).round().clamp(0, 15).to(torch.uint8).view(*lead, K)
    return q[..., 0::2] | (q[..., 1::2] << 4), scale, zero.to(torch.uint8) if zeros else None


def _inputs(case, seed):
    c, dtype, gen = case, TYPES[case["dtype"]], _generator(seed)
    s = {"case": case}
    if c["op"] in ("route", "moe"):
        s["x"] = _tokens(gen, c["T"], c["D"], dtype)
        s["w_router"] = _normal(gen, (c["E"], c["D"]), 1.5 / math.sqrt(c["D"]), dtype)
    if c["op"] == "moe":
        E, D, H = c["E"], c["D"], c["H"]
        shapes = {"wg": (E, H, D), "wu": (E, H, D), "wd": (E, D, H)}
    elif c["op"] == "mlp_w4":
        s["x"] = _tokens(gen, c["T"], c["D"], dtype)
        shapes = {"wg": (c["H"], c["D"]), "wu": (c["H"], c["D"]), "wd": (c["D"], c["H"])}
    elif c["op"] == "w4_linear":
        s["x"] = _tokens(gen, c["T"], c["K"], dtype)
        shapes = {"w": (c["N"], c["K"])}
    else:
        shapes = {}
    for name, shape in shapes.items():
        if c["op"] == "moe" and not c["w4"]:
            s[name] = _normal(gen, shape, 1 / math.sqrt(shape[-1]), dtype)
        else:
            s[name] = _quantised(gen, shape, c["group"], c["zeros"], dtype)
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        import backward_gate_up_amd as lib

        s["lib"] = lib
        for name in ("w", "wg", "wu", "wd"):  # 4-bit weights are laid out once, when a model is loaded
            if isinstance(s.get(name), tuple):
                s[name] = lib.w4_pack(*s[name])
    return s


# ---- the operators ----------------------------------------------------------


def _route(x, w_router, k, renorm):
    # logits in 64 bits: the choice of experts hangs on their order
    p = torch.softmax(x.double() @ w_router.double().t(), -1)
    # ties go to the lowest index: a stable descending sort keeps it first
    p, ids = torch.sort(p, dim=-1, descending=True, stable=True)
    p, ids = p[:, :k], ids[:, :k]
    if renorm:
        p = p / p.sum(-1, keepdim=True)
    return p.float(), ids.int()


def _float(w):
    """A weight in 32 bits."""
    if not isinstance(w, tuple):
        return w.float()
    codes, scales, zeros = w
    q = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    q = q.view(*scales.shape, -1)
    z = zeros.float()[..., None] if zeros is not None else 8.0
    return ((q - z) * scales.float()[..., None]).flatten(-2)


def _mlp(x, wg, wu, wd):
    g, u = x @ wg.transpose(-1, -2), x @ wu.transpose(-1, -2)
    return (g * torch.sigmoid(g) * u) @ wd.transpose(-1, -2)


def _moe(x, p, ids, wg, wu, wd):
    """[T, D] in 32 bits. With fewer (token, expert) pairs than experts, the pairs' weights are
    gathered; otherwise every expert takes every token and the router's weights are zero elsewhere."""
    E = wg[0].shape[0] if isinstance(wg, tuple) else wg.shape[0]
    T, k = ids.shape
    xf = x.float()
    if T * k <= E:
        at = ids.flatten().long()
        pick = lambda w: _float(tuple(t[at] if t is not None else None for t in w) if isinstance(w, tuple) else w[at])  # noqa: E731
        y = _mlp(xf.repeat_interleave(k, 0)[:, None], pick(wg), pick(wu), pick(wd))
        return (y.view(T, k, -1) * p[..., None]).sum(1)
    dense = torch.zeros((T, E), device=x.device).scatter_(1, ids.long(), p)
    y = _mlp(xf[None], _float(wg), _float(wu), _float(wd))
    return (y * dense.t()[..., None]).sum(0)


def run(state):
    s, c = state, state["case"]
    if own:
        lib = s["lib"]
        if c["op"] == "route":
            return lib.moe_route(s["x"], s["w_router"], c["k"], c["renorm"])
        if c["op"] == "moe":
            return lib.moe_infer(s["x"], s["w_router"], s["wg"], s["wu"], s["wd"], c["k"], c["renorm"])
        if c["op"] == "w4_linear":
            return lib.w4_linear(s["x"], s["w"])
        return lib.infer_w4(s["x"], s["wg"], s["wu"], s["wd"])
    x = s["x"]
    if c["op"] == "route":
        return _route(x, s["w_router"], c["k"], c["renorm"])
    if c["op"] == "moe":
        p, ids = _route(x, s["w_router"], c["k"], c["renorm"])
        return _moe(x, p, ids, s["wg"], s["wu"], s["wd"]).to(x.dtype)
    if c["op"] == "w4_linear":
        return (x.float() @ _float(s["w"]).t()).to(x.dtype)
    return _mlp(x.float(), _float(s["wg"]), _float(s["wu"]), _float(s["wd"])).to(x.dtype)


# ---- the definition in 64 bits ------------------------------------------------


def exact(case, seed):
    c, s = case, _inputs(case, seed)
    x = s["x"].double()

    def weight(w, e=None):
        if not isinstance(w, tuple):
            return (w if e is None else w[e]).double()
        codes, scales, zeros = (t if t is None or e is None else t[e] for t in w)
        n, kk = codes.shape
        full = torch.empty((n, 2 * kk), dtype=torch.float64, device=codes.device)
        full[:, 0::2] = torch.remainder(codes, 16).double()
        full[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
        g = 2 * kk // scales.shape[1]
        full -= 8.0 if zeros is None else zeros.double().repeat_interleave(g, 1)
        return full * scales.double().repeat_interleave(g, 1)

    def block(rows, wg, wu, wd):
        gate = torch.matmul(rows, wg.T)
        return torch.matmul(gate / (1 + torch.exp(-gate)) * torch.matmul(rows, wu.T), wd.T)

    if c["op"] == "w4_linear":
        return torch.matmul(x, weight(s["w"]).T)
    if c["op"] == "mlp_w4":
        return block(x, weight(s["wg"]), weight(s["wu"]), weight(s["wd"]))
    logits = torch.matmul(x, s["w_router"].double().T)
    odds = torch.exp(logits - logits.amax(1, keepdim=True))
    odds = odds / odds.sum(1, keepdim=True)
    left, picks = logits.clone(), []
    rows = torch.arange(c["T"], device=x.device)
    for _ in range(c["k"]):
        best = (left == left.amax(1, keepdim=True)).int().argmax(1)  # the first of equals
        picks.append(best)
        left[rows, best] = -math.inf
    ids = torch.stack(picks, 1)
    p = odds.gather(1, ids)
    if c["renorm"]:
        p = p / p.sum(1, keepdim=True)
    if c["op"] == "route":
        return p, None
    y = torch.zeros_like(x)
    for e in range(c["E"]):
        share = (p * (ids == e)).sum(1)
        at = (ids == e).any(1).nonzero()[:, 0]
        if at.numel():
            y[at] += share[at, None] * block(x[at], weight(s["wg"], e), weight(s["wu"], e), weight(s["wd"], e))
    return y


# ---- what a pass cannot do without ---------------------------------------------


def _weight_bytes(c, n, k):
    """Bytes of one N x K weight of the case."""
    if c.get("w4", True) and c["group"]:
        g = n * k // c["group"]
        return n * k / 2 + 2 * g + (g / 2 if c["zeros"] else 0)
    return n * k * (4 if c["dtype"] == "fp32" else 2)


def work(case):
    c = case
    e = 4 if c["dtype"] == "fp32" else 2
    T = c["T"]
    if c["op"] == "route":
        return {"bytes": (T + c["E"]) * c["D"] * e + T * c["k"] * 8, "flops": 2 * T * c["E"] * c["D"]}
    if c["op"] == "moe":
        E, k, D, H = c["E"], c["k"], c["D"], c["H"]
        hit = E * (1 - (1 - k / E) ** T)  # experts that get a token, expected for an even router
        return {"bytes": 2 * T * D * e + E * D * e + hit * (2 * _weight_bytes(c, H, D) + _weight_bytes(c, D, H)),
                "flops": 2 * T * E * D + 6 * T * k * D * H}
    if c["op"] == "w4_linear":
        return {"bytes": T * (c["N"] + c["K"]) * e + _weight_bytes(c, c["N"], c["K"]), "flops": 2 * T * c["N"] * c["K"]}
    return {"bytes": 2 * T * c["D"] * e + 2 * _weight_bytes(c, c["H"], c["D"]) + _weight_bytes(c, c["D"], c["H"]),
            "flops": 6 * T * c["D"] * c["H"]}
