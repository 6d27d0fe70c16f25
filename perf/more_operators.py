"""Training through 8-bit activation checkpoints, measured: layer norms with their
backward pass, linear layers with bias, activation and residual in the product's
epilogue, and the gradients that read the saved activations as INT8 payloads.

Each case is one step of one operator as a training program (or, for single tokens,
a server) makes it. `own` chooses between the framework's kernels and their plain
form, elementary torch operations in 32 bits.

Operators (`op` of a case):
  ln       fc_layer_norm; with a group, the forward pass that also writes the INT8
           checkpoint of x, then fc_layer_norm_backward from that checkpoint
  lnback   fc_layer_norm_backward of a 16-bit x or of its checkpoint
  linear   fc_linear_act: a w^T + bias, activation, product with a second tensor, residual
  linback  fc_linear_input_grad, fc_linear_weight_grad from the checkpoint of the
           layer's input, and the bias gradient
  actback  fc_activation_backward from the checkpoint of the pre-activations
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
ACTS = ["none", "relu", "silu", "gelu", "gelu_tanh"]


def listed():
    return [
        # one decoded token's layer norm (LLaMA-3-70B hidden size), no statistics kept
        dict(name="ln_token_70b", op="ln", T=1, H=8192, dt="bf16", rms=False, bias=True, group=0),
        # a training batch at the 8B hidden size: forward with the checkpoint of x, and the backward pass from it
        dict(name="ln_step_8b", op="ln", T=8192, H=4096, dt="f16", rms=False, bias=True, group=128),
        # an odd hidden size and a ragged token count, from the saved 16-bit x
        dict(name="lnback_odd", op="lnback", T=1777, H=5003, dt="bf16", rms=False, bias=True, group=0, skip=False),
        # the RMS norm of the 70B block, from the checkpoint, added to the gradient of the skip connection
        dict(name="lnback_70b", op="lnback", T=8192, H=8192, dt="bf16", rms=True, bias=False, group=128, skip=True),
        # one token through a rank's gate projection (70B, TP = 4), times the up projection's output
        dict(name="linear_token_70b", op="linear", R=1, T=1, K=8192, H=7168, dt="bf16", bias=False, act="silu", mul=True, skip=False, keep=False),
        # a ragged decode batch through the four ranks' d_proj slices (8B, TP = 4), with bias and residual
        dict(name="linear_decode_8b", op="linear", R=4, T=77, K=3584, H=4096, dt="f16", bias=True, act="none", mul=False, skip=True, keep=False),
        # odd in every dimension
        dict(name="linear_odd", op="linear", R=1, T=333, K=1001, H=2047, dt="bf16", bias=True, act="relu", mul=False, skip=False, keep=False),
        # a rank's up projection of a training batch (70B, TP = 4), the pre-activations kept
        dict(name="linear_train_70b", op="linear", R=1, T=8192, K=8192, H=7168, dt="bf16", bias=True, act="gelu", mul=False, skip=False, keep=True),
        # the gradients of that layer
        dict(name="linback_70b", op="linback", R=1, T=8192, K=8192, H=7168, dt="bf16", bias=True, group=128),
        # few channels and many, ragged tokens: sums over a long axis
        dict(name="linback_long", op="linback", R=1, T=32773, K=512, H=320, dt="f16", bias=True, group=64),
        # a small batch's activation, with the bias gradient
        dict(name="actback_small", op="actback", R=1, T=100, H=3584, dt="f16", act="gelu", mul=False, bias=True, group=32),
        # the gated activation of a training batch (70B, TP = 4): both factors from checkpoints
        dict(name="actback_70b", op="actback", R=1, T=8192, H=7168, dt="bf16", act="silu", mul=True, bias=False, group=128),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _grouped(rng, lo, hi):
    """A group length and a row length that it divides."""
    g = rng.choice([8, 16, 24, 32, 64, 96, 128, 256, 512])
    return g, g * max(1, _log(rng, lo, hi) // g)


def draw(rng):
    op = rng.choice(["ln", "lnback", "linear", "linback", "actback"])
    c = dict(op=op, dt=rng.choice(["bf16", "f16"]))
    if op in ("ln", "lnback"):
        c.update(T=_log(rng, 1, 8192), rms=rng.random() < 0.4, bias=rng.random() < 0.7, group=0, H=_log(rng, 64, 8192))
        if rng.random() < 0.5:
            c["group"], c["H"] = _grouped(rng, 64, 8192)
        if op == "lnback":
            c["skip"] = rng.random() < 0.5
        return c
    c["R"] = rng.choice([1, 1, 2, 4])
    if op == "actback":
        c.update(T=_log(rng, 1, 8192 // c["R"]), act=rng.choice(ACTS[1:]), mul=rng.random() < 0.4, bias=rng.random() < 0.6)
        c["group"], c["H"] = _grouped(rng, 64, 7168)
        return c
    c.update(T=_log(rng, 1, 8192 // c["R"]), bias=rng.random() < 0.7, H=_log(rng, 16, 7168))
    if op == "linear":
        c.update(K=_log(rng, 32, 8192), act=rng.choice(ACTS), mul=rng.random() < 0.3, skip=rng.random() < 0.4,
                 keep=rng.random() < 0.3)
        if rng.random() < 0.5:   # most models' sizes are multiples of 64
            c["K"], c["H"] = [-(-n // 64) * 64 for n in (c["K"], c["H"])]
    else:
        c["group"], c["K"] = _grouped(rng, 32, 8192)
        if rng.random() < 0.5:
            c["H"] = min(7168, -(-c["H"] // 64) * 64)
    return c


def _activations(gen, shape, dt):
    """Normal activations with a few hidden channels scaled up, as in LLM blocks."""
    x = torch.randn(shape, generator=gen, device=DEV)
    hot = torch.randint(0, shape[-1], (max(1, shape[-1] // 200),), generator=gen, device=DEV)
    x[..., hot] *= 20.0
    return (x * 0.5).to(dt)


def _payload(x, group):
    """INT8 codes of each group with an fp16 scale and zero: what fc_quantize_groups writes."""
    g = x.float().unflatten(-1, (-1, group))
    mn, mx = g.amin(-1), g.amax(-1)
    s, z = ((mx - mn) / 255.0).half(), mn.half()
    sf = s.float()[..., None]
    inv = torch.where(sf > 0, 1.0 / sf.clamp_min(1e-30), 0.0)
    q = ((g - z.float()[..., None]) * inv).round().clamp(0, 255)
    return q.flatten(-2).to(torch.uint8), s.view(torch.uint16), z.view(torch.uint16)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DTYPES[c["dt"]]

    def normal(*shape, scale=1.0):
        return (torch.randn(shape, generator=gen, device=DEV) * scale).to(dt)

    op, T, H = c["op"], c["T"], c["H"]
    if op in ("ln", "lnback"):
        x = _activations(gen, (T, H), dt) + normal(T, 1)
        c["w"] = (1 + 0.2 * torch.randn(H, generator=gen, device=DEV)).to(dt)
        c["b"] = normal(H, scale=0.1) if c["bias"] else None
        if op == "lnback" or c["group"]:
            c["dy"] = normal(T, H, scale=0.1)
        if op == "ln":
            c["x"] = x
            return c
        xf = x.float()
        c["mean"] = None if c["rms"] else xf.mean(-1)
        centred = xf if c["rms"] else xf - c["mean"][:, None]
        c["rstd"] = torch.rsqrt(centred.square().mean(-1) + EPS)
        c["dres"] = normal(T, H, scale=0.1) if c["skip"] else None
        if c["group"]:
            c["payload"] = _payload(x, c["group"])
        else:
            c["x"] = x
        return c
    R = c["R"]
    if op == "linear":
        K = c["K"]
        c["a"] = _activations(gen, (R, T, K), dt)
        c["w"] = normal(R, H, K, scale=K ** -0.5)
        c["b"] = normal(R, H, scale=0.5) if c["bias"] else None
        c["m"] = normal(R, T, H) if c["mul"] else None
        c["res"] = normal(R, T, H, scale=2.0) if c["skip"] else None
    elif op == "linback":
        K = c["K"]
        c["dy"] = normal(R, T, H, scale=0.1)
        c["w"] = normal(R, H, K, scale=K ** -0.5)
        c["payload"] = _payload(_activations(gen, (R, T, K), dt), c["group"])
    else:
        c["dy"] = normal(R, T, H, scale=0.1)
        c["payload"] = _payload(normal(R, T, H, scale=1.5), c["group"])
        c["m"] = _payload(normal(R, T, H), c["group"]) if c["mul"] else None
    return c


# --- the plain forms ---------------------------------------------------------

def _values(payload, group):
    codes, s, z = payload
    q = codes.float().unflatten(-1, (-1, group))
    return (q * s.view(torch.float16).float()[..., None] + z.view(torch.float16).float()[..., None]).flatten(-2)


def _act(z, act):
    if act == "relu":
        return torch.where(z > 0, z, 0.0)
    if act == "silu":
        return z / (1 + torch.exp(-z))
    if act == "gelu":
        return 0.5 * z * torch.special.erfc(z * -math.sqrt(0.5))
    if act == "gelu_tanh":
        return z / (1 + torch.exp(-2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    return z


def _act_slope(z, act):
    if act == "relu":
        return (z > 0).to(z.dtype)
    if act == "silu":
        p = 1 / (1 + torch.exp(-z))
        return p * (1 + z * (1 - p))
    if act == "gelu":
        return 0.5 * torch.special.erfc(z * -math.sqrt(0.5)) + z * torch.exp(-0.5 * z * z) * (1 / math.sqrt(2 * math.pi))
    if act == "gelu_tanh":
        c = 2 * math.sqrt(2 / math.pi)
        p = 1 / (1 + torch.exp(-c * (z + 0.044715 * z * z * z)))
        return p + z * p * (1 - p) * c * (1 + 3 * 0.044715 * z * z)
    return torch.ones_like(z)


def _ln_backward(s, x, mean, rstd, dres):
    dy, w = s["dy"].float(), s["w"].float()
    n = (x if mean is None else x - mean[:, None]) * rstd[:, None]
    g = dy * w
    dx = g - n * (g * n).mean(-1, keepdim=True)
    if mean is not None:
        dx = dx - g.mean(-1, keepdim=True)
    dx = dx * rstd[:, None]
    if dres is not None:
        dx = dx + dres.float()
    out = [dx.to(s["dy"].dtype), (dy * n).sum(0)]
    return out + [dy.sum(0)] if s["bias"] else out


def _plain(s):
    op = s["op"]
    if op == "ln":
        x = s["x"].float()
        mean = None if s["rms"] else x.mean(-1)
        centred = x if s["rms"] else x - mean[:, None]
        rstd = torch.rsqrt(centred.square().mean(-1) + EPS)
        y = centred * rstd[:, None] * s["w"].float()
        if s["b"] is not None:
            y = y + s["b"].float()
        y = y.to(s["x"].dtype)
        if not s["group"]:
            return [y]
        return [y] + _ln_backward(s, _values(_payload(s["x"], s["group"]), s["group"]), mean, rstd, None)
    if op == "lnback":
        x = _values(s["payload"], s["group"]) if s["group"] else s["x"].float()
        return _ln_backward(s, x, s["mean"], s["rstd"], s["dres"])
    if op == "linear":
        dt = s["a"].dtype
        z = torch.matmul(s["a"].float(), s["w"].float().transpose(-1, -2).contiguous())
        if s["b"] is not None:
            z = z + s["b"].float()[:, None]
        y = _act(z, s["act"])
        if s["m"] is not None:
            y = y * s["m"].float()
        if s["res"] is not None:
            y = y + s["res"].float()
        return [y.to(dt), z.to(dt)] if s["keep"] else [y.to(dt)]
    dy = s["dy"].float()
    dt = s["dy"].dtype
    if op == "linback":
        # the checkpoint stands for activations of the layer's type
        x = _values(s["payload"], s["group"]).to(dt).float()
        out = [torch.matmul(dy, s["w"].float()).to(dt), torch.matmul(dy.transpose(-1, -2).contiguous(), x)]
        return out + [dy.sum(1)] if s["bias"] else out
    z = _values(s["payload"], s["group"])
    if s["m"] is None:
        dz = dy * _act_slope(z, s["act"])
        out = [dz.to(dt)]
    else:
        m = _values(s["m"], s["group"])
        dz = dy * m * _act_slope(z, s["act"])
        out = [dz.to(dt), (dy * _act(z, s["act"])).to(dt)]
    return out + [dz.sum(1)] if s["bias"] else out


# --- the framework's calls ---------------------------------------------------

def _call(s):
    import bit_activation_compression_amd as fc
    op = s["op"]
    if op == "ln":
        if not s["group"]:
            return [fc.fc_layer_norm(s["x"], s["w"], s["b"], EPS, rms=s["rms"])[0]]
        y, mean, rstd, payload = fc.fc_layer_norm(s["x"], s["w"], s["b"], EPS, rms=s["rms"], stats=True, group=s["group"])
        grads = fc.fc_layer_norm_backward(s["dy"], payload, mean, rstd, s["w"], rms=s["rms"], bias=s["bias"])
        return [y] + [g for g in grads if g is not None]
    if op == "lnback":
        x = s["payload"] if s["group"] else s["x"]
        grads = fc.fc_layer_norm_backward(s["dy"], x, s["mean"], s["rstd"], s["w"], rms=s["rms"], bias=s["bias"], dres=s["dres"])
        return [g for g in grads if g is not None]
    if op == "linear":
        y, z = fc.fc_linear_act(s["a"], s["w"], s["b"], s["act"], mul=s["m"], residual=s["res"], z=s["keep"])
        return [y, z] if s["keep"] else [y]
    if op == "linback":
        out = [fc.fc_linear_input_grad(s["dy"], s["w"]), fc.fc_linear_weight_grad(s["dy"], s["payload"])]
        if s["bias"]:
            out.append(fc.fc_activation_backward(s["dy"], "none", bias=True)[2])
        return out
    out = fc.fc_activation_backward(s["dy"], s["act"], s["payload"], mul=s["m"], bias=s["bias"])
    return [t for t in out if t is not None]


def run(state):
    return _call(state) if own else _plain(state)


def work(case):
    c = case
    op, T, H = c["op"], c["T"], c["H"]

    def saved(n, group):   # a payload, or 16-bit values
        return n * (1 + 4 / group) if group else 2 * n

    if op in ("ln", "lnback"):
        n = T * H
        back = 2 * n + 2 * n + 4 * T * (1 if c["rms"] else 2) + 2 * H + 4 * H * (2 if c["bias"] else 1)
        if op == "lnback":
            return {"bytes": back + saved(n, c["group"]) + (2 * n if c["skip"] else 0), "flops": 12.0 * n}
        b = 4 * n + 2 * H * (2 if c["bias"] else 1)
        if not c["group"]:
            return {"bytes": b, "flops": 8.0 * n}
        stats = 4 * T * (1 if c["rms"] else 2)
        return {"bytes": b + stats + saved(n, c["group"]) + back + saved(n, c["group"]), "flops": 24.0 * n}
    R = c["R"]
    n = R * T * H
    if op == "linear":
        K = c["K"]
        b = 2 * (R * T * K + R * H * K + n * (1 + c["mul"] + c["skip"] + c["keep"]) + R * H * c["bias"])
        return {"bytes": b, "flops": 2.0 * n * K}
    if op == "linback":
        K = c["K"]
        b = 2 * n + 2 * R * H * K + saved(R * T * K, c["group"]) + 2 * R * T * K + 4 * R * H * K + 4 * R * H * c["bias"]
        return {"bytes": b, "flops": 4.0 * n * K}
    b = (2 + 2 + 2 * c["mul"]) * n + saved(n, c["group"]) * (1 + c["mul"]) + 4 * R * H * c["bias"]
    return {"bytes": b, "flops": 12.0 * n}


# --- the definitions in 64 bits ----------------------------------------------

def _held(payload, group):
    codes, s, z = payload
    wide = [t.view(torch.float16).double().repeat_interleave(group, -1) for t in (s, z)]
    return codes.double() * wide[0] + wide[1]


def _bell(z):
    return torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)


def _exact_act(z, act):
    """(value, slope) of the activation."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        return z.clamp_min(0), (z > 0).double()
    if act == "gelu":
        cdf = torch.special.ndtr(z)
        return z * cdf, cdf + z * _bell(z)
    u = z if act == "silu" else math.sqrt(8 / math.pi) * (z + 0.044715 * z ** 3)
    du = 1.0 if act == "silu" else math.sqrt(8 / math.pi) * (1 + 0.134145 * z ** 2)
    p = torch.sigmoid(u)
    return z * p, p + z * p * torch.sigmoid(-u) * du


def _exact_ln_backward(s, x, mean, rstd, dres):
    dy, w, H = s["dy"].double(), s["w"].double(), s["H"]
    n = x * rstd
    if mean is not None:
        n = n - mean * rstd
    g = dy * w
    dx = rstd * (H * g - n * (g * n).sum(-1, keepdim=True)) / H
    if mean is not None:
        dx = dx - rstd * g.sum(-1, keepdim=True) / H
    if dres is not None:
        dx = dx + dres.double()
    out = [dx, (dy * n).sum(0)]
    return out + [dy.sum(0)] if s["bias"] else out


def exact(case, seed):
    s = prepare(case, seed)
    op, H = s["op"], s["H"]
    if op == "ln":
        x = s["x"].double()
        mean = None if s["rms"] else x.sum(-1, keepdim=True) / H
        c = x if mean is None else x - mean
        rstd = 1 / torch.sqrt((c * c).sum(-1, keepdim=True) / H + EPS)
        y = c * rstd * s["w"].double()
        if s["b"] is not None:
            y = y + s["b"].double()
        if not s["group"]:
            return [y]
        # codes are defined by their binary32 steps
        held = _held(_payload(s["x"], s["group"]), s["group"])
        return [y] + _exact_ln_backward(s, held, mean, rstd, None)
    if op == "lnback":
        x = _held(s["payload"], s["group"]) if s["group"] else s["x"].double()
        mean = None if s["mean"] is None else s["mean"].double()[:, None]
        return _exact_ln_backward(s, x, mean, s["rstd"].double()[:, None], s["dres"])
    out = [[], [], []]
    for r in range(s["R"]):
        if op == "linear":
            z = s["a"][r].double() @ s["w"][r].double().t().contiguous()
            if s["b"] is not None:
                z = z + s["b"][r].double()
            y = _exact_act(z, s["act"])[0]
            if s["m"] is not None:
                y = y * s["m"][r].double()
            if s["res"] is not None:
                y = y + s["res"][r].double()
            one = [y, z if s["keep"] else None, None]
        elif op == "linback":
            dy = s["dy"][r].double()
            # rounded to the layer's type from the binary32 value, as fc_dequantize does
            x = _held([t[r] for t in s["payload"]], s["group"]).float().to(s["dy"].dtype).double()
            one = [dy @ s["w"][r].double(), dy.t().contiguous() @ x, dy.sum(0) if s["bias"] else None]
        else:
            dy = s["dy"][r].double()
            a, slope = _exact_act(_held([t[r] for t in s["payload"]], s["group"]), s["act"])
            m = 1.0 if s["m"] is None else _held([t[r] for t in s["m"]], s["group"])
            dz = dy * m * slope
            one = [dz, None if s["m"] is None else dy * a, dz.sum(0) if s["bias"] else None]
        for i in range(3):
            out[i].append(one[i])
    return [torch.stack(o) for o in out if o[0] is not None]
