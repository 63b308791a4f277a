"""The decoder block's operators around the rotated W4 linear layer, as timed
cases: the layer with a bias, an activation and a residual in its epilogue,
the gated up-projection (gate and up weights, activation and product in one
call), and the root-mean-square norm with the residual's addition, with its
output in fp16 or in 8 bits with scales.

With `own` false, run() computes each operator from its formula in elementary
torch operations in 32 bits, rounded once at the end; with `own` true it makes
the calls a user of rotated_w4_linear_b200.binding makes. exact() evaluates the
same definitions in 64 bits.

    linear   Y = act((X T^-1) w_hat^T + b) + R
    gated    H = act((X T^-1) w_gate^T + b_gate) * ((X T^-1) w_up^T + b_up)
    norm     v = x + b + r,  H = v,  Y = v / sqrt(mean(v^2) + eps) * weight,
             Y in fp16, or as 8-bit e4m3 codes Y / s with s = max|Y| / 448 over
             128 channels or over the row

T is the scaled pairwise rotation of include/paro.h (K layers of Givens
rotations inside every quantisation group, after a division by alpha), and
w_hat = fp16((q - z) s) the W4 weight as that header defines it.

Shapes are the layer shapes of bench.py (Llama-3-8B, Qwen3-4B and Qwen3-14B
like), and odd ones inside the same ranges.
"""
import math

import numpy as np
import torch

own = False

K_LAYERS = 8
EPS = 1e-5
E4M3_MAX = 448.0


# --------------------------------------------------------------------- cases
def listed():
    return [
        # decode, one token: the down projection that adds to the residual stream
        {"name": "down_residual_t1", "op": "linear", "tokens": 1, "in": 14336, "out": 4096, "group": 128,
         "rotated": True, "act": "none", "bias": False, "residual": True},
        # decode, a full decode batch: the attention output projection with its residual
        {"name": "o_residual_t16", "op": "linear", "tokens": 16, "in": 4096, "out": 4096, "group": 128,
         "rotated": True, "act": "none", "bias": False, "residual": True},
        # a short ragged prompt through a biased GELU layer, groups of 64, no rotation
        {"name": "gelu_bias_t77_g64", "op": "linear", "tokens": 77, "in": 2560, "out": 9744, "group": 64,
         "rotated": False, "act": "gelu", "bias": True, "residual": False},
        # prefill: the down projection with its residual
        {"name": "down_residual_t2048", "op": "linear", "tokens": 2048, "in": 14336, "out": 4096, "group": 128,
         "rotated": True, "act": "none", "bias": False, "residual": True},
        # decode, one token: gate and up with SiLU (the smallest call of the block's largest weights)
        {"name": "gated_t1", "op": "gated", "tokens": 1, "in": 4096, "inter": 14336, "group": 128,
         "rotated": True, "act": "silu", "bias": False},
        # decode, an odd batch on the small model's shapes
        {"name": "gated_t11_small", "op": "gated", "tokens": 11, "in": 2560, "inter": 9728, "group": 128,
         "rotated": True, "act": "silu", "bias": False},
        # a ragged prompt, tanh-GELU gate with biases, groups of 256
        {"name": "gated_t333_g256", "op": "gated", "tokens": 333, "in": 5120, "inter": 17416, "group": 256,
         "rotated": True, "act": "gelu_tanh", "bias": True},
        # prefill of a long prompt: the largest call
        {"name": "gated_t8192", "op": "gated", "tokens": 8192, "in": 4096, "inter": 14336, "group": 128,
         "rotated": True, "act": "silu", "bias": False},
        # decode, one token: residual and norm before the next projection
        {"name": "norm_t1", "op": "norm", "tokens": 1, "features": 4096, "add": "fp16", "residual": True,
         "bias": False, "out": "fp16"},
        # prefill: residual and norm at HBM speed
        {"name": "norm_t8192", "op": "norm", "tokens": 8192, "features": 4096, "add": "fp16", "residual": True,
         "bias": False, "out": "fp16"},
        # a ragged batch after a row-parallel layer: fp32 sums, bias and residual in, 8-bit codes per 128 channels out
        {"name": "norm_q8_t1023_fp32", "op": "norm", "tokens": 1023, "features": 2576, "add": "fp32",
         "residual": True, "bias": True, "out": "q8_128"},
        # long prompt, 8-bit codes with one scale per token
        {"name": "norm_q8_row_t4096", "op": "norm", "tokens": 4096, "features": 5120, "add": "fp16",
         "residual": True, "bias": False, "out": "q8_row"},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], even over the logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["linear", "gated", "norm"])
    if op == "norm":
        features = 16 * _spread(rng, 16, 1088)
        tokens = _spread(rng, 1, max(1, min(16384, 8192 * 5120 // features)))
        return {"op": op, "tokens": tokens, "features": features, "add": rng.choice(["fp16", "fp32"]),
                "residual": rng.random() < 0.8, "bias": rng.random() < 0.3,
                "out": rng.choice(["fp16", "q8_128", "q8_row"])}
    group = rng.choice([64, 128, 128, 256])
    n_in = 256 * _spread(rng, 2, 64) if group == 256 else 128 * _spread(rng, 4, 136)
    acts = ["none", "relu", "silu", "gelu", "gelu_tanh"]
    n_out = 8 * _spread(rng, 32, 2176) if op == "gated" else 16 * _spread(rng, 16, 1088)
    width = 2 * n_out if op == "gated" else n_out
    tokens = _spread(rng, 1, max(1, min(8192, 8192 * 4096 * 28672 // (n_in * width))))
    case = {"op": op, "tokens": tokens, "in": n_in, "group": group, "rotated": rng.random() < 0.8,
            "act": rng.choice(acts[1:] if op == "gated" else acts), "bias": rng.random() < 0.4}
    if op == "gated":
        case["inter"] = n_out
    else:
        case["out"] = n_out
        case["residual"] = rng.random() < 0.6
    return case


# -------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _normal(g, *shape):
    return torch.randn(*shape, device="cuda", generator=g)


def _activations(g, tokens, features):
    """N(0, 1) with four channels twenty times larger, as hidden states have."""
    x = _normal(g, tokens, features)
    at = torch.randperm(features, device="cuda", generator=g)[:4]
    x[:, at] *= 20.0
    return x


def _codes(g, n_out, n_in, group):
    """W4 codes of N(0, 0.02) weights: round to nearest between a group's least and greatest weight."""
    w = (_normal(g, n_out, n_in) * 0.02).view(n_out, n_in // group, group)
    lo, hi = w.amin(2), w.amax(2)
    s = ((hi - lo) / 15).half()
    z = torch.clamp(torch.round(-lo / s.float()), 0, 15)
    q = torch.clamp(torch.round(w / s.float()[:, :, None]) + z[:, :, None], 0, 15)
    return q.view(n_out, n_in).to(torch.uint8), s, z.to(torch.uint8)


def _rotation(g, n_in, group):
    """K layers of random perfect matchings inside the groups, angles and channel scales."""
    G = n_in // group
    order = torch.rand(K_LAYERS, G, group, device="cuda", generator=g).argsort(2)
    pairs = order.view(K_LAYERS, G, group // 2, 2)
    theta = (torch.rand(K_LAYERS, G, group // 2, device="cuda", generator=g) * 2 - 1) * math.pi
    alpha = torch.exp(0.3 * _normal(g, n_in))
    return pairs, theta, alpha


def _apply_layers(v, pairs, theta):
    """Layers 1..K on the last axis of v [..., G, group], in v's type: (i, j) -> (c i - s j, s i + c j)."""
    for t in range(pairs.shape[0]):
        i, j = pairs[t, :, :, 0], pairs[t, :, :, 1]
        c, s = torch.cos(theta[t].double()).to(v.dtype), torch.sin(theta[t].double()).to(v.dtype)
        i, j = i.expand(*v.shape[:-2], *i.shape), j.expand(*v.shape[:-2], *j.shape)
        a, b = v.gather(-1, i), v.gather(-1, j)
        v = v.scatter(-1, i, c * a - s * b).scatter(-1, j, s * a + c * b)
    return v


def _group_matrices(pairs, theta, alpha, group):
    """Each group's diag(1/alpha) R_1^T ... R_K^T, fp32 [G][group][group]: the layers applied to the rows of diag(1/alpha)."""
    G = alpha.numel() // group
    rows = torch.diag_embed(1.0 / alpha.double().view(G, group)).transpose(0, 1).contiguous()   # [group][G][group]
    return _apply_layers(rows, pairs, theta).transpose(0, 1).contiguous().float()


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        T, F = case["tokens"], case["features"]
        x = _activations(g, T, F)
        st = {"case": case, "x": x if case["add"] == "fp32" else x.half(),
              "residual": (2 * _normal(g, T, F)).half() if case["residual"] else None,
              "bias": (0.1 * _normal(g, F)).half() if case["bias"] else None,
              "weight": (1 + 0.2 * _normal(g, F)).half()}
        if own:
            st["H"] = torch.empty(T, F, dtype=torch.float16, device="cuda")
            if case["out"] == "fp16":
                st["Y"] = torch.empty(T, F, dtype=torch.float16, device="cuda")
            else:
                n = -(-F // 128) if case["out"] == "q8_128" else 1
                st["Y"] = torch.empty(T, F, dtype=torch.float8_e4m3fn, device="cuda")
                st["S"] = torch.empty(T, n, dtype=torch.float32, device="cuda")
        return st
    T, n_in, group = case["tokens"], case["in"], case["group"]
    n_out = 2 * case["inter"] if case["op"] == "gated" else case["out"]
    width = case["inter"] if case["op"] == "gated" else n_out
    x = _activations(g, T, n_in).half()
    q, s, z = _codes(g, n_out, n_in, group)                 # gated: the gate's rows, then the up projection's
    rot = _rotation(g, n_in, group) if case["rotated"] else None
    st = {"case": case, "x": x,
          "bias": (0.1 * _normal(g, n_out)).half() if case["bias"] else None,
          "residual": (2 * _normal(g, T, width)).half() if case.get("residual") else None}
    if own:
        from rotated_w4_linear_b200 import binding as B
        handle = None
        if rot is not None:
            pairs, theta, alpha = (v.cpu().numpy() for v in rot)
            handle = B.paro_rot_create(pairs.astype(np.int16), theta, alpha, group=group)
        st["Y"] = torch.empty(T, width, dtype=torch.float16, device="cuda")
        if case["op"] == "gated":
            st["layer"] = B.ParoGated(handle, *B.paro_pack_gated(q, s, z, group=group), n_in, case["inter"],
                                      group=group, bias=st["bias"], act=case["act"])
        else:
            st["layer"] = B.ParoLinear(handle, *B.paro_pack_weights(q, s, z, group=group), n_in, n_out,
                                       group=group, bias=st["bias"], act=case["act"])
    else:
        st.update(q=q, s=s, z=z)
        st["M"] = _group_matrices(*rot, group) if rot is not None else None
    return st


# ---------------------------------------------------------------- plain forms
def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "silu":
        return v / (1 + torch.exp(-v))
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _plain_sums(st):
    """(X T^-1) w_hat^T + b in 32 bits."""
    case, x = st["case"], st["x"].float()
    group, n_in = case["group"], case["in"]
    if st["M"] is not None:
        x = torch.matmul(x.view(-1, n_in // group, group).transpose(0, 1), st["M"]).transpose(0, 1).reshape(-1, n_in)
    q = st["q"].view(-1, n_in // group, group).float()
    w = ((q - st["z"].float()[:, :, None]) * st["s"].float()[:, :, None]).half().float().view(-1, n_in)
    y = torch.matmul(x, w.t())
    return y if st["bias"] is None else y + st["bias"].float()


def _plain_norm(st):
    case = st["case"]
    v = st["x"].float()
    if st["bias"] is not None:
        v = v + st["bias"].float()
    if st["residual"] is not None:
        v = v + st["residual"].float()
    h = v.half()
    y = v * torch.rsqrt((v * v).mean(1, keepdim=True) + EPS) * st["weight"].float()
    if case["out"] == "fp16":
        return {"H": h, "Y": y.half()}
    T, F = y.shape
    c = 128 if case["out"] == "q8_128" else F
    n = -(-F // c)
    y = torch.nn.functional.pad(y, (0, n * c - F)).view(T, n, c)
    s = y.abs().amax(2) / E4M3_MAX
    codes = (y / s[:, :, None]).view(T, n * c)[:, :F]
    return {"H": h, "Y": torch.nan_to_num(codes, nan=0.0).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn), "S": s}


def run(st):
    case = st["case"]
    if own:
        if case["op"] == "norm":
            from rotated_w4_linear_b200 import binding as B
            if case["out"] == "fp16":
                y, h = B.paro_rmsnorm(st["x"], st["weight"], EPS, residual=st["residual"], bias=st["bias"],
                                      H=st["H"], Y=st["Y"])
                return {"H": h, "Y": y}
            y, s, h = B.paro_rmsnorm_q8(st["x"], st["weight"], EPS, residual=st["residual"], bias=st["bias"],
                                        scale_group=128 if case["out"] == "q8_128" else 0,
                                        H=st["H"], Y=st["Y"], S=st["S"])
            return {"H": h, "Y": y, "S": s}
        if case["op"] == "gated":
            return {"Y": st["layer"](st["x"], st["Y"])}
        return {"Y": st["layer"](st["x"], st["Y"], residual=st["residual"])}
    if case["op"] == "norm":
        return _plain_norm(st)
    z = _plain_sums(st)
    if case["op"] == "gated":
        gate, up = z[:, :case["inter"]], z[:, case["inter"]:]
        return {"Y": (_act(gate, case["act"]) * up).half()}
    y = _act(z, case["act"])
    return {"Y": (y if st["residual"] is None else y + st["residual"].float()).half()}


# ------------------------------------------------------------- what it takes
def work(case):
    T = case["tokens"]
    if case["op"] == "norm":
        F = case["features"]
        n = {"fp16": 0, "q8_128": -(-F // 128), "q8_row": 1}[case["out"]]
        per = (4 if case["add"] == "fp32" else 2) + (2 if case["residual"] else 0) + 2 \
            + (2 if case["out"] == "fp16" else 1)                       # x, r in; H, Y out
        return {"bytes": T * F * per + 4 * T * n + 2 * F * (2 if case["bias"] else 1),
                "flops": T * F * 6}
    n_in, group = case["in"], case["group"]
    n_out = 2 * case["inter"] if case["op"] == "gated" else case["out"]
    width = case["inter"] if case["op"] == "gated" else n_out
    G = n_in // group
    nbytes = n_in * n_out // 2 + n_out * G * 2 + n_out * G // 2 + 2 * T * n_in + 2 * T * width
    flops = 2 * T * n_in * n_out
    if case["bias"]:
        nbytes += 2 * n_out
    if case.get("residual"):
        nbytes += 2 * T * width
    if case["rotated"]:
        nbytes += K_LAYERS * (n_in // 2) * (8 + 2) + 4 * n_in           # angles' cos and sin, pair bytes, alpha
        flops += 3 * K_LAYERS * T * n_in
    return {"bytes": nbytes, "flops": flops}


# ------------------------------------------------------------ in 64 bits
def _rotated_exactly(x, pairs, theta, alpha, group):
    """X T^-1 layer by layer: channel c becomes cos(th) x_c -/+ sin(th) x_partner, minus for a pair's first channel."""
    G = alpha.numel() // group
    base = torch.arange(G, device=x.device)[:, None] * group
    x = x / alpha.double()
    for layer, angle in zip(pairs, theta.double()):
        first, second = (layer[:, :, 0] + base).flatten(), (layer[:, :, 1] + base).flatten()
        partner = torch.empty(alpha.numel(), dtype=torch.long, device=x.device)
        partner[first], partner[second] = second, first
        own_part, other_part = torch.empty(2, alpha.numel(), dtype=torch.float64, device=x.device)
        own_part[first] = own_part[second] = torch.cos(angle).flatten()
        other_part[first], other_part[second] = -torch.sin(angle).flatten(), torch.sin(angle).flatten()
        x = x * own_part + x[:, partner] * other_part
    return x


def exact(case, seed):
    g = _gen(seed)
    if case["op"] == "norm":
        T, F = case["tokens"], case["features"]
        x = _activations(g, T, F)
        v = (x if case["add"] == "fp32" else x.half()).double()
        r = (2 * _normal(g, T, F)).half().double() if case["residual"] else 0.0
        b = (0.1 * _normal(g, F)).half().double() if case["bias"] else 0.0
        weight = (1 + 0.2 * _normal(g, F)).half().double()
        v = v + r + b
        y = v / torch.sqrt(torch.sum(v ** 2, 1, keepdim=True) / F + EPS) * weight
        if case["out"] == "fp16":
            return {"H": v, "Y": y}
        # the codes before they are rounded to 8 bits, and the scales
        parts = torch.split(y, 128 if case["out"] == "q8_128" else F, 1)
        scales = [p.abs().max(1, keepdim=True).values / E4M3_MAX for p in parts]
        return {"H": v, "Y": torch.cat([p / s for p, s in zip(parts, scales)], 1), "S": torch.cat(scales, 1)}
    T, n_in, group = case["tokens"], case["in"], case["group"]
    n_out = 2 * case["inter"] if case["op"] == "gated" else case["out"]
    width = case["inter"] if case["op"] == "gated" else n_out
    x = _activations(g, T, n_in).half().double()
    q, s, z = _codes(g, n_out, n_in, group)
    if case["rotated"]:
        x = _rotated_exactly(x, *_rotation(g, n_in, group), group)
    bias = (0.1 * _normal(g, n_out)).half().double() if case["bias"] else 0.0
    residual = (2 * _normal(g, T, width)).half().double() if case.get("residual") else 0.0
    each = torch.repeat_interleave
    w = ((q.double() - each(z, group, 1).double()) * each(s, group, 1).double()).half().double()
    sums = x @ w.T + bias
    a = sums[:, :width]
    a = {"none": lambda: a, "relu": lambda: torch.where(a > 0, a, 0.0), "silu": lambda: a * torch.sigmoid(a),
         "gelu": lambda: a * 0.5 * torch.erfc(-a / math.sqrt(2)),
         "gelu_tanh": lambda: a * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (a + 0.044715 * a ** 3))}[case["act"]]()
    return {"Y": a * sums[:, width:] if case["op"] == "gated" else a + residual}
