"""Measured cases of two groups of serving operators, with their plain forms.

* the 8-bit integer product with a scale per token and per output channel, from float rows
  (quantised in the call) or from codes that are already there;
* the whole latent mixture-of-experts layer for a few tokens.

own = False computes the plain form with elementary torch operations; own = True calls the
package. exact() computes the definition in float64.
"""
import math

import torch

own = False

INT8_SCALE_MIN = 2.0 ** -126  # smallest normal float32: the scale of an all-zero row
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
NORM_EPS, PRE_NORM_EPS = 1e-6, 1e-5
LOGIT_SCALE, ROUTED_SCALING = 0.17677669529663687, 2.5  # released router: 1 / sqrt(32) before the sigmoid


# ------------------------------------------------------------------------------- the cases
def listed():
    def linear(name, T, N, K, x="bf16", out="bf16", codes=False, pad=0):
        return {"name": name, "op": "int8", "T": T, "N": N, "K": K, "x": x, "out": out, "codes": codes, "pad": pad}

    def layer(name, T, D, L, I, E, k, kind="bf16", released=False):
        return {"name": name, "op": "layer", "T": T, "D": D, "L": L, "I": I, "E": E, "k": k, "kind": kind,
                "released": released}

    return [
        # one decoded token through the full-size pooler: the latency of the smallest call
        linear("int8 pooler 1 token", 1, 4096, 8192),
        # odd sizes, float32 in and out, rows cut from a wider buffer
        linear("int8 odd f32 padded", 5, 1000, 2064, x="f32", out="f32", pad=48),
        # a decode batch through the full-size unpooler
        linear("int8 unpooler 64 tokens", 64, 8192, 4096),
        # a ragged prompt chunk whose rows are quantised already (one quantisation, several products)
        linear("int8 codes 777 tokens", 777, 4096, 4096, codes=True),
        # a full prefill batch through the pooler
        linear("int8 pooler prefill", 8192, 4096, 8192),
        # the smallest layer, in float32
        layer("layer tiny f32 3 tokens", 3, 256, 128, 128, 8, 2, kind="f32"),
        # one token through the mid-sized layer: launch latency decides
        layer("layer mid 1 token", 1, 2048, 1024, 1024, 64, 4),
        # uneven widths, the released router and norms (sigmoid, bias, pre-expert norm, shared gain)
        layer("layer released 4 tokens", 4, 1536, 640, 896, 40, 6, released=True),
        # one token through the full-size layer
        layer("layer full 1 token", 1, 8192, 4096, 4096, 256, 8),
        # the same with NVFP4 experts
        layer("layer full nvfp4 1 token", 1, 8192, 4096, 4096, 256, 8, kind="nvfp4"),
        # eight sequences decoding together: about 57 of 256 experts are touched
        layer("layer full nvfp4 8 tokens", 8, 8192, 4096, 4096, 256, 8, kind="nvfp4"),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.5:
        T = _spread(rng, 1, 4096)
        K = 16 * _spread(rng, 4, 640)
        N = _spread(rng, 50, 9000)
        codes = rng.random() < 0.3
        T = max(1, min(T, 2 ** 38 // (N * K)))  # no more work than a prefill batch through the pooler
        return {"op": "int8", "T": T, "N": N, "K": K, "x": "bf16" if codes else rng.choice(("bf16", "f32")),
                "out": rng.choice(("bf16", "f32")), "codes": codes,
                "pad": 0 if codes else rng.choice((0, 0, 16, 80))}
    kind = rng.choice(("bf16", "bf16", "nvfp4", "f32"))
    step = 256 if kind == "nvfp4" else 128
    D, L, I = (unit * _spread(rng, 1, top // unit) for unit, top in ((128, 8192), (step, 4096), (step, 4096)))
    E = _spread(rng, 4, 128)
    case = {"op": "layer", "T": rng.randint(1, 8), "D": D, "L": L, "I": I, "E": E, "k": rng.randint(1, min(8, E)),
            "kind": kind, "released": rng.random() < 0.3}
    while work(case)["bytes"] > 1.5e9:  # no more than eight tokens through the full-size NVFP4 layer
        case["T"], case["k"] = max(1, case["T"] - 1), max(1, case["k"] - 1)
    return case


def work(case):
    c = case
    T = c["T"]
    if c["op"] == "int8":
        N, K = c["N"], c["K"]
        xb = 1 if c["codes"] else 4 if c["x"] == "f32" else 2
        ob = 4 if c["out"] == "f32" else 2
        return {"bytes": T * K * xb + (4 * T if c["codes"] else 0) + N * K + 4 * N + T * N * ob, "flops": 2 * T * N * K}
    D, L, I, E, k = (c[n] for n in ("D", "L", "I", "E", "k"))
    a = 4 if c["kind"] == "f32" else 2
    w = 0.5625 if c["kind"] == "nvfp4" else a
    touched = E * (1.0 - (1.0 - k / E) ** T)  # distinct experts of T tokens, routed evenly
    return {"bytes": int(a * (E * D + 2 * L * D + 2 * T * D) + touched * (3 * I * L * w + L * a)),
            "flops": 2 * T * (E * D + 2 * L * D + 3 * k * I * L)}


# ------------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(gen, shape, std, dtype):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _nvfp4_pool(w):
    """Codes, E4M3 block scales and matrix scale of normal weights [rows, cols]."""
    mscale = w.abs().amax() / (6.0 * 448.0)
    blocks = w.view(w.shape[0], -1, 16)
    scales = (blocks.abs().amax(-1) / (6.0 * mscale)).clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn)
    q = blocks / (scales.float() * mscale)[..., None]
    borders = torch.tensor([(a + b) / 2 for a, b in zip(E2M1, E2M1[1:])], device=w.device)
    code = torch.bucketize(q.abs(), borders).to(torch.uint8) | ((q < 0).to(torch.uint8) << 3)
    code = code.view(w.shape[0], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), scales.view(torch.uint8), mscale


def _nvfp4_experts(gen, E, rows, cols):
    """E expert matrices: the quantised magnitudes of two normal matrices in turn, with signs of their own."""
    pool = [_nvfp4_pool(_normal(gen, (rows, cols), cols ** -0.5, torch.float32)) for _ in range(2)]
    pick = torch.arange(E, device="cuda") % 2
    codes = torch.stack([p[0] for p in pool])[pick]
    codes ^= torch.randint(0, 256, codes.shape, dtype=torch.uint8, device="cuda", generator=gen) & 0x88
    return codes, torch.stack([p[1] for p in pool])[pick], torch.stack([p[2] for p in pool])[pick].contiguous()


def _int8_state(case, seed):
    gen = _gen(seed)
    T, N, K = case["T"], case["N"], case["K"]
    dt = torch.float32 if case["x"] == "f32" else torch.bfloat16
    # activations with a few wide channels, as a residual stream has them
    x = _normal(gen, (T, K + case["pad"]), 1.0, dt)[:, :K]
    x[:, :: max(1, K // 8)] *= 6.0
    w = _normal(gen, (N, K), K ** -0.5, torch.float32)
    codes, scales = _plain_quantise(w)
    s = {"x": x, "w_codes": codes.to(torch.int8), "w_scales": scales[:, 0].contiguous(),
         "out": torch.float32 if case["out"] == "f32" else torch.bfloat16}
    if case["codes"]:
        q, sx = _plain_quantise(x.float())
        s["x_codes"], s["x_scales"] = q.to(torch.int8), sx[:, 0].contiguous()
    if own:
        import latent_mixture_experts_moe_b200 as moe
        s["linear"] = moe.Int8Linear(s["w_codes"], s["w_scales"], T_max=T, scale_rule=moe.INT8_SCALE_RECIPROCAL)
    return s


def _layer_state(case, seed):
    gen = _gen(seed)
    T, D, L, I, E = (case[n] for n in ("T", "D", "L", "I", "E"))
    dt = torch.float32 if case["kind"] == "f32" else torch.bfloat16
    released = case["released"]
    w = {"W_router": _normal(gen, (E, D), D ** -0.5, dt), "W_pool": _normal(gen, (L, D), D ** -0.5, dt),
         "W_unpool": _normal(gen, (D, L), L ** -0.5, dt),
         "gamma": _normal(gen, (L,) if released else (E, L), 0.1 ** 0.5, dt)}
    for name, shape in (("W_gate", (I, L)), ("W_up", (I, L)), ("W_down", (L, I))):
        if case["kind"] == "nvfp4":
            w[name + "_codes"], w[name + "_scales"], w[name + "_mscale"] = _nvfp4_experts(gen, E, *shape)
        else:
            w[name] = _normal(gen, (E,) + shape, shape[1] ** -0.5, dt)
    if released:
        w["router_bias"] = _normal(gen, (E,), 0.05, torch.float32)
        w["pre_norm_gain"] = _normal(gen, (L,), 0.3, dt)
    s = {"x": _normal(gen, (T, D), 1.0, dt), "w": w, "k": case["k"], "released": released}
    if own:
        import latent_mixture_experts_moe_b200 as moe
        modes = dict(router_mode=moe.ROUTER_SIGMOID, router_logit_scale=LOGIT_SCALE, routed_scaling=ROUTED_SCALING,
                     norm_mode=moe.NORM_INPUT_SCALED, gamma_shared=True, pre_norm_eps=PRE_NORM_EPS) if released else {}
        s["layer"] = moe.LatentMoE(w, T_max=T, k=case["k"], eps=NORM_EPS, **modes)
    return s


def prepare(case, seed):
    return _int8_state(case, seed) if case["op"] == "int8" else _layer_state(case, seed)


# ------------------------------------------------------------------------------- plain forms
def _plain_quantise(x):
    """Codes (whole numbers in float32) and the scale of every row."""
    amax = x.abs().amax(1, keepdim=True)
    scale = (amax / 127.0).clamp_min(INT8_SCALE_MIN)
    return torch.round(x / scale).clamp(-127.0, 127.0), scale


def _plain_int8(s):
    if "x_codes" in s:
        q, sx = s["x_codes"].float(), s["x_scales"][:, None]
    else:
        q, sx = _plain_quantise(s["x"].float())
    return ((q @ s["w_codes"].float().T) * (sx * s["w_scales"])).to(s["out"])


def _plain_expert_weights(w, name, idx):
    """The matrices of experts idx, in float32."""
    if name in w:
        return w[name][idx].float()
    codes = w[name + "_codes"][idx]
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    v = table[torch.stack((codes & 15, codes >> 4), -1).int()].flatten(-2)
    sc = w[name + "_scales"][idx].view(torch.float8_e4m3fn).float() * w[name + "_mscale"][idx][..., None, None]
    return (v.unflatten(-1, (-1, 16)) * sc[..., None]).flatten(-2)


def _plain_layer(s):
    w, k, released = s["w"], s["k"], s["released"]
    x = s["x"].float()
    logits = x @ w["W_router"].float().T
    if released:
        p = torch.sigmoid(LOGIT_SCALE * logits)
        idx = torch.sort(p + w["router_bias"], dim=1, descending=True, stable=True).indices[:, :k]
        g = p.gather(1, idx)
        g = ROUTED_SCALING * g / (g.sum(1, keepdim=True) + 1e-15)
    else:
        idx = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :k]
        g = logits.gather(1, idx)
        g = torch.exp(g - g.amax(1, keepdim=True))
        g = g / g.sum(1, keepdim=True)
    z = x @ w["W_pool"].float().T
    if released:
        z = z * torch.rsqrt((z * z).mean(1, keepdim=True) + PRE_NORM_EPS) * (1.0 + w["pre_norm_gain"].float())
    zs = z[:, None, :, None]
    a = _plain_expert_weights(w, "W_gate", idx) @ zs
    h = a * torch.sigmoid(a) * (_plain_expert_weights(w, "W_up", idx) @ zs)
    y = (_plain_expert_weights(w, "W_down", idx) @ h)[..., 0]
    gain = 1.0 + (w["gamma"] if released else w["gamma"][idx]).float()
    u = y * gain
    n = (u if released else y).square().mean(2, keepdim=True)
    c = (g[..., None] * u * torch.rsqrt(n + NORM_EPS)).sum(1)
    return (c @ w["W_unpool"].float().T).to(s["x"].dtype)


def run(state):
    if "x" in state and "w" in state:
        return state["layer"].few_tokens(state["x"]) if own else _plain_layer(state)
    if own:
        if "x_codes" in state:
            return state["linear"].matmul(state["x_codes"], state["x_scales"], out_dtype=state["out"])
        return state["linear"](state["x"], out_dtype=state["out"])
    return _plain_int8(state)


# ------------------------------------------------------------------------------- float64
def _exact_int8(s):
    if "x_codes" in s:
        q, sx = s["x_codes"].double(), s["x_scales"].double()
    else:
        x = s["x"].double()
        sx = torch.clamp(x.abs().max(dim=1).values / 127.0, min=INT8_SCALE_MIN).float().double()
        q = torch.clamp(torch.round(x / sx.unsqueeze(1)), -127, 127)
    return torch.einsum("tk,nk->tn", q, s["w_codes"].double()) * sx.unsqueeze(1) * s["w_scales"].double().unsqueeze(0)


def _exact_matrix(w, name, e):
    if name in w:
        return w[name][e].double()
    codes = w[name + "_codes"][e].long()
    out = torch.empty(codes.shape[0], 2 * codes.shape[1], dtype=torch.float64, device=codes.device)
    for half, nibble in enumerate((codes & 15, codes >> 4)):
        sign = 1.0 - 2.0 * (nibble >> 3).double()
        exponent, mantissa = (nibble >> 1) & 3, (nibble & 1).double()
        low = (exponent == 0).double()
        out[:, half::2] = sign * (low * 0.5 * mantissa + (1 - low) * (1 + 0.5 * mantissa) * torch.exp2(exponent.double() - 1))
    scale = w[name + "_scales"][e].view(torch.float8_e4m3fn).double() * w[name + "_mscale"][e].double()
    return out * scale.repeat_interleave(16, dim=1)


def _exact_layer(s):
    w, k, released = s["w"], s["k"], s["released"]
    rows = []
    for x in s["x"].double():
        logits = torch.mv(w["W_router"].double(), x)
        score = 1.0 / (1.0 + torch.exp(-LOGIT_SCALE * logits)) if released else logits
        key = (score + w["router_bias"].double() if released else score).tolist()
        chosen = sorted(range(len(key)), key=lambda e: (-key[e], e))[:k]
        g = score[chosen] if released else torch.softmax(score[chosen], 0)
        if released:
            g = ROUTED_SCALING * g / (g.sum() + 1e-15)
        z = torch.mv(w["W_pool"].double(), x)
        if released:
            z = z / torch.sqrt(z.pow(2).mean() + PRE_NORM_EPS) * (1 + w["pre_norm_gain"].double())
        c = torch.zeros_like(z)
        for weight, e in zip(g, chosen):
            a, b = torch.mv(_exact_matrix(w, "W_gate", e), z), torch.mv(_exact_matrix(w, "W_up", e), z)
            y = torch.mv(_exact_matrix(w, "W_down", e), a / (1 + torch.exp(-a)) * b)
            gain = 1 + (w["gamma"] if released else w["gamma"][e]).double()
            rms = torch.sqrt((y * gain if released else y).pow(2).mean() + NORM_EPS)
            c += weight * y * gain / rms
        rows.append(torch.mv(w["W_unpool"].double(), c))
    return torch.stack(rows)


def exact(case, seed):
    s = prepare(case, seed)
    return _exact_int8(s) if case["op"] == "int8" else _exact_layer(s)
