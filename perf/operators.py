"""The 8-bit linear layer and the expert-grouped products: cases, inputs, plain forms and work.

Kinds of case:
  linear   tokens (binary16 or float32) -> one 8-bit scale per token -> product with int8 rows, one scale per channel
  product  the same product on tokens already held in 8 bits (several layers share one quantized X)
  experts  rows sorted by expert, each expert's rows times its own matrix (binary16, or 8 bits on both sides)
  swiglu   the experts' gate and up products joined as silu(gate) * up
"""
import math

import torch

own = False

F32, F16 = "f32", "f16"
TYPES = {F32: torch.float32, F16: torch.float16}


def listed():
    return [
        # the O projection of a decode step, one token: latency
        dict(name="linear 1x896x896", kind="linear", m=1, n=896, k=896, x=F32, y=F32, bias=False),
        # gate/up of a short prompt
        dict(name="linear 16x4864x896", kind="linear", m=16, n=4864, k=896, x=F16, y=F32, bias=False),
        # c_attn at an odd prompt length, with its bias, binary16 out
        dict(name="linear 513x2304x768", kind="linear", m=513, n=2304, k=768, x=F16, y=F16, bias=True),
        # the down projection of a long prompt: few columns, long rows
        dict(name="linear 4096x896x4864", kind="linear", m=4096, n=896, k=4864, x=F16, y=F32, bias=False),
        # the output head for a batch of sequences: nothing but weights and logits
        dict(name="linear 64x151936x896", kind="linear", m=64, n=151936, k=896, x=F16, y=F32, bias=False),
        # the largest: a long batch through a square layer, X quantized before
        dict(name="product 8192x4096x4096", kind="product", m=8192, n=4096, k=4096, y=F16, bias=False),
        # one token through four of 64 experts, down projections in binary16
        dict(name="experts f16 1 token", kind="experts", form=F16, tokens=1, top=4, e=64, n=896, k=2432, gather=False, y=F32,
             bias=False),
        # a small batch of sequences decoding, 8 bits, about four rows an expert, tokens gathered
        dict(name="experts i8 65 tokens", kind="experts", form="i8", tokens=65, top=4, e=60, n=1408, k=2048, gather=True, y=F16,
             bias=True),
        # a prompt through wide experts in binary16, odd widths
        dict(name="experts f16 1021 tokens", kind="experts", form=F16, tokens=1021, top=2, e=8, n=2429, k=1056, gather=True,
             y=F32, bias=False),
        # a long batch through many experts in 8 bits
        dict(name="experts i8 4096 tokens", kind="experts", form="i8", tokens=4096, top=8, e=64, n=2048, k=1024, gather=False,
             y=F16, bias=False),
        # one decoding token's gate and up projections in 8 bits
        dict(name="swiglu i8 1 token", kind="swiglu", form="i8", tokens=1, top=8, e=64, n=1024, k=2048, gather=True, y=F32),
        # gate and up of a prompt in binary16
        dict(name="swiglu f16 2048 tokens", kind="swiglu", form=F16, tokens=2048, top=4, e=32, n=1408, k=2048, gather=True,
             y=F16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    most = max(work(c)["flops"] for c in listed())
    while True:
        kind = rng.choice(["linear", "product", "experts", "swiglu"])
        k = 32 * _log(rng, 8, 152)
        y = rng.choice([F32, F16])
        if kind in ("linear", "product"):
            n = _log(rng, 64, 151936)
            c = dict(kind=kind, m=_log(rng, 1, 8192), n=n if rng.random() < 0.5 else n + 15 & -16, k=k, y=y,
                     bias=rng.random() < 0.5)
            if kind == "linear":
                c["x"] = rng.choice([F32, F16])
        else:
            e = _log(rng, 2, 128)
            n = _log(rng, 64, 4864)
            c = dict(kind=kind, form=rng.choice([F16, "i8"]), tokens=_log(rng, 1, 4096), top=rng.randint(1, min(8, e)), e=e,
                     n=n if rng.random() < 0.5 else n + 15 & -16, k=k, gather=rng.random() < 0.5, y=y)
            if kind == "experts":
                c["bias"] = rng.random() < 0.5
        # W and Y (and the plain form's float32 copies of them) fit easily; no dearer than the largest listed case
        weights = c["n"] * k * c.get("e", 1)
        rows = c["m"] if "m" in c else c["tokens"] * c["top"]
        if work(c)["flops"] <= most and weights <= 1 << 28 and rows * max(c["n"], k) <= 1 << 28:
            return c


def _shape(case):
    """Rows of Y, and how many matrices of [n][k] one row is multiplied with."""
    if case["kind"] in ("linear", "product"):
        return case["m"], 1
    return case["tokens"] * case["top"], 2 if case["kind"] == "swiglu" else 1


def work(case):
    rows, mats = _shape(case)
    n, k = case["n"], case["k"]
    out = rows * n * (4 if case["y"] == F32 else 2)
    if case["kind"] in ("linear", "product"):
        x = rows * k * {F32: 4, F16: 2}[case["x"]] if case["kind"] == "linear" else rows * (k + 4)
        return {"bytes": x + n * (k + 4) + (4 * n if case["bias"] else 0) + out, "flops": 2 * rows * n * k}
    size, scale = (2, 0) if case["form"] == F16 else (1, 4)
    active = min(case["e"], rows)   # experts that can have rows
    x = (case["tokens"] if case["gather"] else rows) * (k * size + scale) + (4 * rows if case["gather"] else 0)
    w = mats * active * n * (k * size + scale) + (4 * active * n if case.get("bias") else 0)
    return {"bytes": x + w + out + 4 * (case["e"] + 1), "flops": 2 * mats * rows * n * k}


def _tokens(gen, m, k):
    """Activations: normal, with a few channels that are much larger, as hidden states have them."""
    x = torch.randn(m, k, generator=gen, device="cuda")
    loud = torch.randint(0, k, (max(1, k // 128),), generator=gen, device="cuda")
    x[:, loud] *= 8.0
    return x


def _codes(gen, *shape):
    return torch.randint(-127, 128, shape, generator=gen, device="cuda", dtype=torch.int8)


def _scales(gen, *shape):
    return (torch.rand(shape, generator=gen, device="cuda") + 0.5) * (0.08 / 127)


def _rows_of(values):
    """8-bit codes and scales of rows, as a quantizer leaves them (made here without one)."""
    s = (values.abs().amax(-1).double() / 127).float()
    return (values.double() / s.double().unsqueeze(-1)).round().clamp(-127, 127).to(torch.int8), s


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, mats = _shape(case)
    n, k = case["n"], case["k"]
    s = dict(case=case, y=torch.empty(rows, n, dtype=TYPES[case["y"]], device="cuda"))
    if case["kind"] in ("linear", "product"):
        x = _tokens(gen, rows, k)
        s["w"], s["w_scales"] = _codes(gen, n, k), _scales(gen, n)
        s["bias"] = torch.randn(n, generator=gen, device="cuda") if case["bias"] else None
        s["x_codes"], s["x_scales"] = _rows_of(x) if case["kind"] == "product" else (
            torch.empty(rows, k, dtype=torch.int8, device="cuda"), torch.empty(rows, device="cuda"))
        if case["kind"] == "linear":
            s["x"] = x.to(TYPES[case["x"]])
        return s
    e, top, tokens = case["e"], case["top"], case["tokens"]
    # a router's choice: `top` different experts a token, some experts liked much more than others
    liked = torch.randn(e, generator=gen, device="cuda")
    score = liked - torch.log(-torch.log(torch.rand(tokens, e, generator=gen, device="cuda").clamp(1e-7, 1 - 1e-7)))
    ids = score.topk(top, dim=1).indices.reshape(-1)
    order = torch.argsort(ids, stable=True)
    counts = torch.bincount(ids, minlength=e)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
    s["most"] = int(counts.max())   # the fullest expert's rows: what the plain form pads to
    s["x_rows"] = (order // top).to(torch.int32) if case["gather"] else None
    x = _tokens(gen, tokens if case["gather"] else rows, k)
    names = ["w"] if mats == 1 else ["gate", "up"]
    if case["form"] == F16:
        s["x"], s["x_scales"] = x.half(), None
        for name in names:
            s[name], s[name + "_scales"] = (torch.randn(e, n, k, generator=gen, device="cuda") * 0.03).half(), None
    else:
        s["x"], s["x_scales"] = _rows_of(x)
        for name in names:
            s[name], s[name + "_scales"] = _codes(gen, e, n, k), _scales(gen, e, n)
    s["bias"] = torch.randn(e, n, generator=gen, device="cuda") if case.get("bias") else None
    return s


def _own(s):
    import dequantize_mat_vec_amd as dmv
    c = s["case"]
    n, k = c["n"], c["k"]
    if c["kind"] in ("linear", "product"):
        if c["kind"] == "linear":
            dmv.pesti_quant_i8token(c["x"], c["m"], k, s["x"], s["x_codes"], s["x_scales"])
        dmv.pesti_gemm_i8row_i8token(c["m"], n, k, s["w"], s["w_scales"], s["x_codes"], s["x_scales"], s["y"], s["bias"])
        return s["y"]
    form = F16 if c["form"] == F16 else "i8row"
    rows, tokens = c["tokens"] * c["top"], s["x"].shape[0]
    if c["kind"] == "experts":
        dmv.pesti_gemm_experts(form, rows, c["e"], n, k, s["offsets"], s["w"], tokens, s["x"], s["y"], bias=s["bias"],
                               w_scales=s["w_scales"], x_scales=s["x_scales"], x_rows=s["x_rows"])
    else:
        dmv.pesti_gemm_experts_swiglu(form, rows, c["e"], n, k, s["offsets"], s["gate"], s["up"], tokens, s["x"], s["y"],
                                      gate_scales=s["gate_scales"], up_scales=s["up_scales"], x_scales=s["x_scales"],
                                      x_rows=s["x_rows"])
    return s["y"]


def _quantized(x):
    """Codes (as float32) and scales of rows: code = x / scale rounded half away from zero.  The quotient is taken in 64 bits: in
    32 it is rounded onto borders that it does not lie on."""
    scale = (x.float().abs().amax(-1).double() / 127).float()
    q = x.double() / scale.double().unsqueeze(-1)
    q = torch.sign(q) * torch.floor(q.abs() + 0.5)
    return torch.where(scale.unsqueeze(-1) > 0, q, torch.zeros_like(q)).clamp(-127, 127).float(), scale


def _grouped(s, x, x_scales, w, w_scales):
    """Each row times its expert's matrix, in float32: rows laid out as [expert][place], padded to the fullest expert."""
    c = s["case"]
    rows = torch.arange(s["y"].shape[0], device=x.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), rows, right=True)
    place = rows - s["offsets"].long()[expert]
    padded = torch.zeros(c["e"], s["most"], c["k"], device=x.device)
    padded[expert, place] = x
    y = torch.bmm(padded, w.float().transpose(1, 2).contiguous())[expert, place]
    return y if w_scales is None else y * x_scales.unsqueeze(1) * w_scales[expert]


def _plain(s):
    c = s["case"]
    out = TYPES[c["y"]]
    if c["kind"] in ("linear", "product"):
        x, scale = _quantized(s["x"]) if c["kind"] == "linear" else (s["x_codes"].float(), s["x_scales"])
        y = (x @ s["w"].float().t()) * scale.unsqueeze(1) * s["w_scales"]
        return (y if s["bias"] is None else y + s["bias"]).to(out)
    at = slice(None) if s["x_rows"] is None else s["x_rows"].long()
    x, xs = s["x"][at].float(), None if s["x_scales"] is None else s["x_scales"][at]
    if c["kind"] == "swiglu":
        g = _grouped(s, x, xs, s["gate"], s["gate_scales"])
        return (g / (1 + torch.exp(-g)) * _grouped(s, x, xs, s["up"], s["up_scales"])).to(out)
    y = _grouped(s, x, xs, s["w"], s["w_scales"])
    if s["bias"] is not None:
        rows = torch.arange(y.shape[0], device=y.device)
        y = y + s["bias"][torch.searchsorted(s["offsets"][1:].long(), rows, right=True)]
    return y.to(out)


def run(state):
    return _own(state) if own else _plain(state)


def exact(case, seed):
    s = prepare(case, seed)
    n, k = case["n"], case["k"]
    y = torch.empty(s["y"].shape, dtype=torch.float64, device="cuda")
    if case["kind"] in ("linear", "product"):
        if case["kind"] == "linear":
            x = s["x"].double()
            scale = (x.abs().max(dim=1).values / 127).float().double()   # the scale is a float32 number
            safe = torch.where(scale > 0, scale, torch.ones_like(scale))
            ratio = x / safe[:, None]
            whole = ratio.trunc()
            codes = whole + torch.sign(ratio) * ((ratio - whole).abs() >= 0.5)
            x = codes.clamp(-127, 127) * scale[:, None]
        else:
            x = s["x_codes"].double() * s["x_scales"].double()[:, None]
        for n0 in range(0, n, 16384):
            w = s["w"][n0:n0 + 16384].double() * s["w_scales"][n0:n0 + 16384].double()[:, None]
            y[:, n0:n0 + 16384] = torch.mm(x, w.t())
        return y if s["bias"] is None else y + s["bias"].double()
    starts = s["offsets"].tolist()
    for e in range(case["e"]):
        a, b = starts[e], starts[e + 1]
        if a == b:
            continue
        at = torch.arange(a, b, device="cuda") if s["x_rows"] is None else s["x_rows"][a:b].long()
        x = s["x"][at].double()
        if s["x_scales"] is not None:
            x = x * s["x_scales"][at].double()[:, None]

        def times(name):
            w = s[name][e].double()
            return torch.mm(x, (w if s[name + "_scales"] is None else w * s[name + "_scales"][e].double()[:, None]).t())

        if case["kind"] == "swiglu":
            g = times("gate")
            y[a:b] = g * torch.sigmoid(g) * times("up")
        else:
            y[a:b] = times("w") if s["bias"] is None else times("w") + s["bias"][e].double()
    return y
