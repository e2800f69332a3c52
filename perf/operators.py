"""The operators around a 4-bit linear layer, as a decoder's program calls them, with a plain form beside each.

  norm     tb_rms_norm            h = x + residual; n = h w / rms(h), optionally rotated in 1024-blocks,
                                  stored as 16-bit floats or in 8 bits with scales
  linear   tb_q4_linear           y = x' W^T with 4-bit weights, one fp16 scale per 128 of them
  prepare  tb_q4_prepare_weights  a dense W, optionally folded with the rotation, rounded to those 4 bits

`own` chooses between the plain forms (elementary torch operations) and the library's calls.
"""
import torch

own = False

DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8,
      "e4m3": torch.float8_e4m3fn}
SIZE = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1, "e4m3": 1}
EPS = 1e-6


def norm_case(name, m, k, xt, rt, signs, yt, group):
    # rt "": no residual; group 0: floating output, k: one scale a row, 128: one per 128 values
    return {"name": name, "op": "norm", "m": m, "k": k, "xt": xt, "rt": rt, "signs": signs, "yt": yt, "group": group}


def linear_case(name, m, n, k, xt, group, signs, yt):
    # group: of the scales of an 8-bit x (k: one a token, 128: one per 128 values), 0 for a floating x
    return {"name": name, "op": "linear", "m": m, "n": n, "k": k, "xt": xt, "group": group, "signs": signs, "yt": yt}


def prepare_case(name, n, k, wt, signs):
    return {"name": name, "op": "prepare", "n": n, "k": k, "wt": wt, "signs": signs}


def listed():
    return [
        # one token of a 5120-wide decoder, before a layer with 8-bit activations
        norm_case("norm_token_e4m3", 1, 5120, "bf16", "bf16", False, "e4m3", 5120),
        # a small batch, odd width, no residual: another model's fp16 activations in int8, a scale a row
        norm_case("norm_odd_int8", 77, 1027, "fp16", "", False, "int8", 1027),
        # a prompt before a rotated linear layer: norm and rotation in one pass
        norm_case("norm_prompt_rotated_bf16", 2048, 5120, "bf16", "bf16", True, "bf16", 0),
        # a long packed batch with a 32-bit residual stream, 8 bits in groups
        norm_case("norm_batch_e4m3_groups", 16384, 5120, "bf16", "fp32", False, "e4m3", 128),
        # one token through a small projection: latency counts
        linear_case("linear_token_k", 1, 1024, 5120, "bf16", 0, False, "bf16"),
        # one token through a gate/up projection: the matrix-vector product of every decode step
        linear_case("linear_token_gate", 1, 17408, 5120, "bf16", 0, False, "bf16"),
        # sixteen sequences through the down projection, 8-bit activations with a scale a token
        linear_case("linear_16_down_int8", 16, 5120, 17408, "int8", 17408, False, "bf16"),
        # a ragged chunk: odd rows, odd tokens, a width that is no multiple of 1024, scales in groups
        linear_case("linear_33_ragged_e4m3", 33, 1001, 1920, "e4m3", 128, False, "fp16"),
        # an unrotated fp16 input into folded weights: the call rotates it itself
        linear_case("linear_64_rotated_fp16", 64, 6144, 5120, "fp16", 0, True, "fp16"),
        # a prompt through the gate/up projection
        linear_case("linear_prompt_gate", 2048, 17408, 5120, "bf16", 0, False, "bf16"),
        # a small projection's weights, already folded
        prepare_case("prepare_k", 1024, 5120, "fp32", False),
        # a gate/up projection's weights, folded and rounded
        prepare_case("prepare_gate_folded", 17408, 5120, "bf16", True),
    ]


def log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(lo * (hi / lo) ** rng.random()))))


def draw(rng):
    op = rng.choice(["norm", "norm", "linear", "linear", "linear", "prepare"])
    if op == "norm":
        signs = rng.random() < 0.4
        yt = rng.choice(["bf16", "fp16", "int8", "e4m3"])
        group = 0
        k = log_int(rng, 64, 17408)
        if signs:
            k = 1024 * max(1, k // 1024)
        if yt in ("int8", "e4m3"):
            group = rng.choice([0, 128])
            k = k if signs or group == 0 else 128 * max(1, k // 128)
            group = group or k
        m = log_int(rng, 1, min(16384, 16384 * 5120 // k))
        c = norm_case("", m, k, rng.choice(["bf16", "fp16", "fp32"]), rng.choice(["", "bf16", "fp16", "fp32"]), signs, yt,
                      group)
    elif op == "linear":
        signs = rng.random() < 0.3
        k = log_int(rng, 256, 17408)
        k = 1024 * max(1, k // 1024) if signs else 128 * max(2, k // 128)
        n = log_int(rng, 64, min(17408, 17408 * 5120 // k))
        m = log_int(rng, 1, 2048)
        xt = rng.choice(["bf16", "fp16"] if signs else ["bf16", "fp16", "int8", "e4m3"])
        group = 0 if xt in ("bf16", "fp16") else rng.choice([k, 128])
        c = linear_case("", m, n, k, xt, group, signs, rng.choice(["bf16", "fp16"]))
    else:
        signs = rng.random() < 0.5
        k = log_int(rng, 256, 17408)
        k = 1024 * max(1, k // 1024) if signs else 128 * max(2, k // 128)
        c = prepare_case("", log_int(rng, 16, min(17408, 17408 * 5120 // k)), k, rng.choice(["bf16", "fp16", "fp32"]), signs)
    del c["name"]
    return c


# ----------------------------------------------------------------- inputs
def draws(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    def uniform(*shape):
        return torch.rand(*shape, generator=g, device="cuda")

    def signs(k):
        return (torch.randint(0, 2, (k,), generator=g, device="cuda") * 2 - 1).to(torch.int8)

    def whole(lo, hi, shape, dtype):
        return torch.randint(lo, hi, shape, generator=g, device="cuda", dtype=dtype)

    return normal, uniform, signs, whole


def activations(normal, uniform, m, k):
    # what a residual stream looks like: about 1 in 100 values is an outlier, and some rows are larger than others
    x = normal(m, k) * (0.5 + uniform(m, 1))
    return torch.where(uniform(m, k) < 0.01, x * 12.0, x)


def prepare(case, seed):
    normal, uniform, signs, whole = draws(seed)
    c = dict(case)
    s = {"case": c}
    if c["op"] == "norm":
        m, k = c["m"], c["k"]
        s["x"] = activations(normal, uniform, m, k).to(DT[c["xt"]])
        s["residual"] = activations(normal, uniform, m, k).to(DT[c["rt"]]) if c["rt"] else None
        s["residual_out"] = torch.empty_like(s["residual"]) if c["rt"] else None
        s["weight"] = (1.0 + 0.2 * normal(k)).to(torch.bfloat16)
        s["signs"] = signs(k) if c["signs"] else None
        s["y"] = torch.empty(m, k, dtype=DT[c["yt"]], device="cuda")
        s["y_scales"] = torch.empty(m, k // c["group"], device="cuda") if c["group"] else None
        s["values"] = torch.empty(m, k, dtype=torch.bfloat16, device="cuda") if c["yt"] == "int8" else None
    elif c["op"] == "linear":
        m, n, k = c["m"], c["n"], c["k"]
        # byte i of a row holds weights 2i (low nibble) and 2i + 1 (high), each as q + 8
        s["packed"] = whole(0, 256, (n, k // 2), torch.uint8)
        s["scales"] = (normal(n, k // 128).abs() * 0.005).to(torch.float16)
        x = activations(normal, uniform, m, k)
        s["x_scales"] = None
        if c["group"]:
            top = 127.0 if c["xt"] == "int8" else 448.0
            xg = x.view(m, k // c["group"], c["group"])
            s["x_scales"] = xg.abs().amax(-1) / top
            x = (xg / s["x_scales"][..., None]).view(m, k)
            x = x.round() if c["xt"] == "int8" else x.clamp(-448.0, 448.0)
        s["x"] = x.to(DT[c["xt"]])
        s["signs"] = signs(k) if c["signs"] else None
        s["y"] = torch.empty(m, n, dtype=DT[c["yt"]], device="cuda")
    else:
        n, k = c["n"], c["k"]
        s["w"] = (normal(n, k) * 0.02).to(DT[c["wt"]])
        s["signs"] = signs(k) if c["signs"] else None
        s["packed"] = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
        s["scales"] = torch.empty(n, k // 128, dtype=torch.float16, device="cuda")
        s["codes"] = torch.empty(n, k, dtype=torch.int8, device="cuda")
    return s


# ----------------------------------------------------------------- plain forms
def sylvester(dtype):
    """H[i, j] = (-1)^popcount(i & j), 1024 x 1024."""
    i = torch.arange(1024, device="cuda")
    b = i[:, None] & i[None, :]
    b = b ^ (b >> 8)
    b = b ^ (b >> 4)
    b = b ^ (b >> 2)
    b = b ^ (b >> 1)
    return (1 - 2 * (b & 1)).to(dtype)


def rotated(v, signs):
    """H (d * v) / 32 in every 1024-block of the rows of v."""
    u = (v * signs.to(v.dtype)).view(-1, 1024)
    return (u @ sylvester(v.dtype) / 32.0).view(v.shape)


def plain_norm(s):
    c = s["case"]
    h = s["x"].float()
    out = {}
    if s["residual"] is not None:
        r = (h + s["residual"].float()).to(DT[c["rt"]])
        out["residual"] = r
        h = r.float()
    n = h / torch.sqrt((h * h).mean(-1, keepdim=True) + EPS) * s["weight"].float()
    if s["signs"] is not None:
        n = rotated(n, s["signs"])
    if not c["group"]:
        return {"y": n.to(DT[c["yt"]]), **out}
    top = 127.0 if c["yt"] == "int8" else 448.0
    ng = n.view(c["m"], -1, c["group"])
    scale = ng.abs().amax(-1) / top
    q = ng / scale[..., None]
    out["scales"] = scale
    if c["yt"] == "int8":
        out["y"] = (q.round().clamp(-127.0, 127.0) * scale[..., None]).view(n.shape).to(torch.bfloat16)
    else:
        out["y"] = q.clamp(-448.0, 448.0).view(n.shape).to(torch.float8_e4m3fn)
    return out


def plain_linear(s):
    c = s["case"]
    x = s["x"].float()
    if s["x_scales"] is not None:
        x = (x.view(c["m"], -1, c["group"]) * s["x_scales"][..., None]).view(c["m"], c["k"])
    if s["signs"] is not None:
        x = rotated(x, s["signs"])
    p = s["packed"]
    q = torch.stack((p & 15, p >> 4), -1).view(c["n"], -1, 128).float() - 8.0
    w = (q * s["scales"].float()[..., None]).view(c["n"], c["k"])
    return {"y": (x @ w.t()).to(DT[c["yt"]])}


def plain_prepare(s):
    # 64 bits: codes next to a border, and a fold whose sums are exact there
    c = s["case"]
    w = s["w"].double()
    if s["signs"] is not None:
        w = rotated(w, s["signs"])
    wg = w.view(c["n"], -1, 128)
    scale = (wg.abs().amax(-1) / 7.0).float().to(torch.float16)
    d = scale.double()[..., None]
    q = torch.where(d > 0, (wg / d).round().clamp(-8.0, 7.0), torch.zeros_like(wg))
    return {"codes": q.view(c["n"], c["k"]).to(torch.int8), "scales": scale}


# ----------------------------------------------------------------- the library's calls
def code(tb, t):
    return {"bf16": tb.TB_BF16, "fp16": tb.TB_FP16, "fp32": tb.TB_FP32, "int8": tb.TB_INT8, "e4m3": tb.TB_E4M3}[t]


def own_norm(s):
    from ternary_weight_signed_b200 import binding as tb
    c = s["case"]
    tb.tb_rms_norm(s["x"], code(tb, c["xt"]), s["residual"], s["residual_out"], code(tb, c["rt"] or "bf16"), s["weight"],
                   tb.TB_BF16, EPS, s["signs"], c["m"], c["k"], s["y"], code(tb, c["yt"]), s["y_scales"], c["group"])
    out = {"y": s["y"]}
    if s["residual"] is not None:
        out["residual"] = s["residual_out"]
    if c["group"]:
        out["scales"] = s["y_scales"]
    if c["yt"] == "int8":
        # 8 whole bits, as the values that they stand for
        grouped = (c["m"], -1, c["group"])
        torch.mul(s["y"].view(grouped), s["y_scales"][..., None], out=s["values"].view(grouped))
        out["y"] = s["values"]
    return out


def own_linear(s):
    from ternary_weight_signed_b200 import binding as tb
    c = s["case"]
    if "workspace" not in s:
        s["workspace"] = torch.empty(tb.tb_q4_linear_workspace(c["m"], c["n"], c["k"]), dtype=torch.uint8, device="cuda")
    tb.tb_q4_linear(s["x"], code(tb, c["xt"]), s["x_scales"], c["group"], s["packed"], s["scales"], c["m"], c["n"], c["k"],
                    s["signs"], s["y"], code(tb, c["yt"]), s["workspace"], s["workspace"].numel())
    return {"y": s["y"]}


def own_prepare(s):
    from ternary_weight_signed_b200 import binding as tb
    c = s["case"]
    tb.tb_q4_prepare_weights(s["w"], code(tb, c["wt"]), s["signs"], c["n"], c["k"], s["packed"], s["scales"])
    tb.tb_q4_unpack(s["packed"], c["n"], c["k"], s["codes"])
    return {"codes": s["codes"], "scales": s["scales"]}


def run(state):
    op = state["case"]["op"]
    if own:
        return {"norm": own_norm, "linear": own_linear, "prepare": own_prepare}[op](state)
    return {"norm": plain_norm, "linear": plain_linear, "prepare": plain_prepare}[op](state)


def work(case):
    c = case
    if c["op"] == "norm":
        mk = c["m"] * c["k"]
        b = mk * (SIZE[c["xt"]] + SIZE[c["yt"]] + (2 * SIZE[c["rt"]] if c["rt"] else 0)) + 2 * c["k"]
        b += 4 * mk // c["group"] if c["group"] else 0
        return {"bytes": b + (c["k"] if c["signs"] else 0), "flops": mk * (16 if c["signs"] else 5)}
    nk = c["n"] * c["k"]
    if c["op"] == "linear":
        b = nk // 2 + nk // 64 + c["m"] * (c["k"] * SIZE[c["xt"]] + c["n"] * SIZE[c["yt"]])
        b += 4 * c["m"] * c["k"] // c["group"] if c["group"] else 0
        return {"bytes": b + (c["k"] if c["signs"] else 0), "flops": 2 * c["m"] * nk + (11 * c["m"] * c["k"] if c["signs"] else 0)}
    # the dense weights in, the packed ones and (as the values they stand for) the codes out
    return {"bytes": nk * SIZE[c["wt"]] + nk // 2 + nk + nk // 64 + (c["k"] if c["signs"] else 0),
            "flops": nk * (14 if c["signs"] else 3)}


# ----------------------------------------------------------------- the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    c = s["case"]

    def rotate(v):
        # the transform as ten sums and differences: H_1024 is H_2 (x) ... (x) H_2
        u = (v.double() * s["signs"].double()).view(-1, 1024)
        for p in range(10):
            u = u.view(-1, 1024 >> (p + 1), 2, 1 << p)
            u = torch.stack((u[:, :, 0] + u[:, :, 1], u[:, :, 0] - u[:, :, 1]), 2)
        return u.reshape(v.shape) / 32.0

    if c["op"] == "norm":
        h = s["x"].double()
        out = {}
        if c["rt"]:
            h = (h + s["residual"].double()).to(DT[c["rt"]]).double()
            out["residual"] = h
        n = h * s["weight"].double() * torch.rsqrt(h.square().sum(-1, keepdim=True) / c["k"] + EPS)
        if c["signs"]:
            n = rotate(n)
        if not c["group"]:
            return {"y": n, **out}
        ng = n.reshape(c["m"], c["k"] // c["group"], c["group"])
        if c["yt"] == "int8":
            scale = ng.abs().amax(-1) / 127.0
            y = torch.round(ng / scale[..., None]) * scale[..., None]
        else:
            scale = ng.abs().amax(-1) / 448.0
            v = ng / scale[..., None]
            unit = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3.0)  # 4 significant bits
            y = torch.round(v / unit) * unit
        return {"y": y.reshape(n.shape), "scales": scale, **out}
    if c["op"] == "linear":
        if 2 * c["m"] * c["n"] * c["k"] > 4e12:
            return None
        x = s["x"].double()
        if c["group"]:
            x = x * s["x_scales"].double().repeat_interleave(c["group"], 1)
        if c["signs"]:
            x = rotate(x)
        w = torch.empty(c["n"], c["k"], dtype=torch.float64, device="cuda")
        w[:, 0::2] = (s["packed"] % 16).double() - 8.0
        w[:, 1::2] = (s["packed"] // 16).double() - 8.0
        w *= s["scales"].double().repeat_interleave(128, 1)
        return {"y": torch.einsum("mk,nk->mn", x, w)}
    w = rotate(s["w"]) if c["signs"] else s["w"].double()
    wg = w.reshape(c["n"], c["k"] // 128, 128)
    # the scale's definition rounds twice, to 32 and then to 16 bits
    scale = (torch.maximum(wg.amax(-1), -wg.amin(-1)) / 7.0).float().to(torch.float16)
    q = torch.round(wg / scale.double()[..., None]).clamp(-8.0, 7.0)
    q = torch.nan_to_num(q, nan=0.0) * (scale != 0)[..., None]
    return {"codes": q.reshape(c["n"], c["k"]).to(torch.int8), "scales": scale}
