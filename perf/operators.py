"""The operators around the low-bit all-reduce, measured: the block norms fused with
the residual update, and the products in microscaled 4-bit floating point (MXFP4).

Each case is one call of one operator as a tensor-parallel LLM server makes it.
`own` chooses between the framework's kernels and their plain form, elementary
torch operations in 32 bits.

Operators (`op` of a case):
  norm     fc_residual_norm: a 16-bit block output, post-normed, gated and added
           to the scaled residual stream; the next block's pre-norm of the sum
  wire     fc_dequantize_residual_norm: the same on the all-gathered payload of
           the all-reduce (codes, fp16 scales and zeros)
  code     fc_quantize_mxfp4, then fc_dequantize_mxfp4: the values the codes hold
  linear   fc_linear_mxfp4: 16-bit activations, quantized in the call, times
           MXFP4 weights
  matmul   fc_matmul_mxfp4: both operands already MXFP4
"""
import math

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16}
EPS = 1e-5
BLOCK = 32        # values that share one scale
STEP = 128        # rows of codes are padded to a multiple of this many values


def listed():
    return [
        # one decoded token's block output (LLaMA-3-70B hidden size), per-channel gate
        dict(name="norm_token_70b", op="norm", T=1, H=8192, dt="bf16", post=True, gate="channel", pre=True),
        # a prefill batch of LLaMA-3-8B, post-norm and pre-norm, no gate
        dict(name="norm_prefill_8b", op="norm", T=8192, H=4096, dt="f16", post=True, gate="none", pre=True),
        # an odd hidden size and a ragged token count, one gate row per token
        dict(name="norm_odd_rows", op="norm", T=1777, H=5003, dt="bf16", post=True, gate="token", pre=True),
        # the decode batch after its all-reduce (70B, INT4 payload)
        dict(name="wire_decode_70b", op="wire", T=64, H=8192, dt="bf16", bits=4, group=128, post=True, gate="channel", pre=True),
        # the prefill batch after its all-reduce (70B, INT4 payload), pre-norm only as in LLaMA
        dict(name="wire_prefill_70b", op="wire", T=8192, H=8192, dt="bf16", bits=4, group=128, post=False, gate="none", pre=True),
        # groups that are not a power of two, INT8 payload, ragged tokens
        dict(name="wire_g96_int8", op="wire", T=1111, H=4608, dt="f16", bits=8, group=96, post=True, gate="channel", pre=True),
        # activations of a small decode batch, odd row length
        dict(name="code_decode_odd", op="code", T=5, K=4100, dt="bf16"),
        # a whole weight matrix of the 70B o_proj
        dict(name="code_weight_70b", op="code", T=8192, K=8192, dt="bf16"),
        # one token through the four ranks' o_proj slices (70B, TP = 4)
        dict(name="linear_token_70b", op="linear", R=4, T=1, K=2048, H=8192, dt="bf16"),
        # a ragged decode batch through the four ranks' d_proj slices (8B, TP = 4)
        dict(name="linear_decode_8b", op="linear", R=4, T=77, K=3584, H=4096, dt="f16"),
        # the o_proj of a prefill batch (70B, TP = 4), activations quantized in the call
        dict(name="linear_prefill_70b", op="linear", R=4, T=8192, K=2048, H=8192, dt="bf16"),
        # the d_proj of a prefill batch (70B, TP = 4), both operands coded
        dict(name="matmul_prefill_70b", op="matmul", R=4, T=8192, K=7168, H=8192, dt="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "wire", "code", "linear", "matmul"])
    c = dict(op=op, dt=rng.choice(["bf16", "f16"]))
    if op in ("norm", "wire"):
        c.update(T=_log(rng, 1, 8192), post=rng.random() < 0.6, gate=rng.choice(["none", "channel", "token", "sequence"]),
                 pre=rng.random() < 0.9)
        if op == "norm":
            c["H"] = _log(rng, 64, 8192)
        else:
            c["bits"] = rng.choice([4, 8])
            c["group"] = rng.choice([8, 24, 32, 64, 96, 128, 160, 256, 512])
            c["H"] = c["group"] * max(1, _log(rng, 64, 8192) // c["group"])
    elif op == "code":
        c.update(T=_log(rng, 1, 8192), K=_log(rng, 32, 8192))
    else:
        c.update(R=rng.choice([1, 2, 3, 4, 8]), T=_log(rng, 1, 8192), K=_log(rng, 32, 8192), H=_log(rng, 16, 8192))
        if op == "linear" and c["T"] > 512:
            c["T"] = _log(rng, 1, 512) if rng.random() < 0.5 else c["T"]
        c["R"] = max(1, min(c["R"], int(3.8e12 / (2.0 * c["T"] * c["K"] * c["H"]))))
    return c


def _gate_rows(c):
    """Rows of the gate, and the tokens that share one."""
    T = c["T"]
    per = {"channel": T, "token": 1, "sequence": max(1, (T + 2) // 3)}[c["gate"]]
    return (T + per - 1) // per, per


def _activations(gen, shape, dt):
    """Normal activations with a few hidden channels scaled up, as in LLM blocks."""
    x = torch.randn(shape, generator=gen, device=DEV)
    hot = torch.randint(0, shape[-1], (max(1, shape[-1] // 200),), generator=gen, device=DEV)
    x[..., hot] *= 20.0
    return (x * 0.5).to(dt)


def prepare(case, seed):
    c = dict(case)
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    dt = DTYPES[c["dt"]]
    op = c["op"]
    if op in ("norm", "wire"):
        T, H = c["T"], c["H"]
        c["residual"] = _activations(gen, (T, H), dt) * 4
        c["w_post"] = (1 + 0.2 * torch.randn(H, generator=gen, device=DEV)).to(dt) if c["post"] else None
        c["w_pre"] = (1 + 0.2 * torch.randn(H, generator=gen, device=DEV)).to(dt) if c["pre"] else None
        c["gate_t"], c["gate_tokens"] = None, 1
        if c["gate"] != "none":
            rows, c["gate_tokens"] = _gate_rows(c)
            c["gate_t"] = torch.randn((rows, H), generator=gen, device=DEV).to(dt)
        c["res_scale"], c["out_scale"] = (1.25, 0.22) if c["post"] else (1.0, 1.0)
        x = _activations(gen, (T, H), dt)
        if op == "norm":
            c["x"] = x
        else:
            c["codes"], c["s"], c["z"] = _payload(x.float(), c["bits"], c["group"])
    elif op == "code":
        c["x"] = _activations(gen, (c["T"], c["K"]), dt)
    else:
        R, T, K, H = c["R"], c["T"], c["K"], c["H"]
        w = torch.randn((R, H, K), generator=gen, device=DEV).mul_(K ** -0.5)
        c["w_codes"], c["w_scales"] = _pack(*_encode(w))
        del w
        a = _activations(gen, (R, T, K), dt)
        if op == "linear":
            c["a"] = a
        else:
            c["a_codes"], c["a_scales"] = _pack(*_encode(a.float()))
    return c


def _payload(x, bits, group):
    """Min/max codes of each group with an fp16 scale and zero: what the all-gather delivers."""
    T, H = x.shape
    g = x.view(T, H // group, group)
    mn, mx = g.amin(-1), g.amax(-1)
    top = float((1 << bits) - 1)
    s, z = ((mx - mn) / top).half(), mn.half()
    q = ((g - z.float()[..., None]) / s.float()[..., None].clamp_min(1e-30)).round().clamp(0, top)
    q = q.view(T, H).to(torch.uint8)
    if bits == 4:
        q = q[:, 0::2] | (q[:, 1::2] << 4)
    return q.contiguous(), s.view(torch.uint16), z.view(torch.uint16)


# --- the plain forms ---------------------------------------------------------

def _pow2(e):
    """2^e, exactly, for whole e in [-149, 127]: two factors whose exponents are normal."""
    e = e.to(torch.int32)
    half = e >> 1
    return ((half + 127) << 23).view(torch.float32) * ((e - half + 127) << 23).view(torch.float32)


def _encode(x):
    """MXFP4 of [..., K] float32: (codes as whole numbers [..., Kp], scale bytes [..., Kp / 32]).
    A block's scale is 2^(floor(log2(max|x|)) - 2); values are rounded half to even to
    {0, 0.5, 1, 1.5, 2, 3, 4, 6} and saturate."""
    K = x.shape[-1]
    x = torch.nn.functional.pad(x, (0, -K % STEP))
    b = x.view(*x.shape[:-1], -1, BLOCK)
    top = b.abs().amax(-1)
    e = torch.where(top > 0, torch.frexp(top)[1] - 3, -127).clamp(-127, 127)
    v = b * _pow2(-e)[..., None]
    m = v.abs()
    step = torch.where(m < 2, 0.5, torch.where(m < 4, 1.0, 2.0))
    q = ((m / step).round() * step).clamp(max=6.0)
    code = torch.where(q < 2, q * 2, torch.where(q < 4, q + 2, q / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(v).to(torch.uint8) << 3)
    return code.view(x.shape), (e + 127).to(torch.uint8)


def _pack(code, scale):
    return (code[..., 0::2] | (code[..., 1::2] << 4)).contiguous(), scale.contiguous()


def _decode(codes, scales):
    """Packed codes and scale bytes -> float32 values [..., Kp]."""
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                        device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).view(*codes.shape[:-1], -1, BLOCK)
    return (grid[c.int()] * _pow2(scales.int() - 127)[..., None]).view(*codes.shape[:-1], -1)


def _norms(s, x):
    residual = s["residual"].float()
    n = x
    if s["w_post"] is not None:
        n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["w_post"].float()
    if s["gate_t"] is not None:
        rows = torch.arange(s["T"], device=x.device) // s["gate_tokens"]
        n = n * s["gate_t"].float()[rows]
    h = s["res_scale"] * residual + s["out_scale"] * n
    dt = s["residual"].dtype
    if s["w_pre"] is None:
        return [h.to(dt)]
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + EPS) * s["w_pre"].float()
    return [h.to(dt), y.to(dt)]


def _unwire(s):
    q = s["codes"]
    if s["bits"] == 4:
        q = torch.stack((q & 15, q >> 4), -1)
    q = q.reshape(s["T"], -1, s["group"]).float()
    x = q * s["s"].view(torch.float16).float()[..., None] + s["z"].view(torch.float16).float()[..., None]
    return x.view(s["T"], s["H"])


def _product(a, w, dt):
    return torch.matmul(a, w.transpose(-1, -2).contiguous()).to(dt)


def _plain(s):
    op = s["op"]
    if op == "norm":
        return _norms(s, s["x"].float())
    if op == "wire":
        return _norms(s, _unwire(s))
    if op == "code":
        x = s["x"]
        return _decode(*_pack(*_encode(x.float())))[..., :s["K"]].to(x.dtype)
    w = _decode(s["w_codes"], s["w_scales"])
    if op == "linear":
        return _product(_decode(*_pack(*_encode(s["a"].float()))), w, s["a"].dtype)
    return _product(_decode(s["a_codes"], s["a_scales"]), w, DTYPES[s["dt"]])


# --- the framework's calls ---------------------------------------------------

def _call(s):
    import bit_activation_compression_amd as fc
    op = s["op"]
    if op in ("norm", "wire"):
        kw = dict(w_post=s["w_post"], w_pre=s["w_pre"], gate=s["gate_t"], gate_tokens=s["gate_tokens"], eps=EPS,
                  res_scale=s["res_scale"], out_scale=s["out_scale"])
        if op == "norm":
            h, y = fc.fc_residual_norm(s["x"], s["residual"], **kw)
        else:
            h, y = fc.fc_dequantize_residual_norm(s["codes"], s["s"], s["z"], s["T"], s["H"], s["bits"], s["group"],
                                                  s["residual"], **kw)
        return [h] if y is None else [h, y]
    if op == "code":
        codes, scales = fc.fc_quantize_mxfp4(s["x"])
        return fc.fc_dequantize_mxfp4(codes, scales, s["K"], s["x"].dtype)
    if op == "linear":
        return fc.fc_linear_mxfp4(s["a"], s["w_codes"], s["w_scales"])
    return fc.fc_matmul_mxfp4(s["a_codes"], s["a_scales"], s["w_codes"], s["w_scales"], DTYPES[s["dt"]])


def run(state):
    return _call(state) if own else _plain(state)


def work(case):
    c = case
    op = c["op"]
    if op in ("norm", "wire"):
        T, H = c["T"], c["H"]
        n = T * H
        b = 2 * n if op == "norm" else n * c["bits"] / 8 + 4 * n / c["group"]
        b += 2 * n + 2 * n + (2 * n + 2 * H if c["pre"] else 0) + (2 * H if c["post"] else 0)
        if c["gate"] != "none":
            b += 2 * H * _gate_rows(c)[0]
        return {"bytes": b, "flops": 12.0 * n}
    if op == "code":
        # the values in, the codes and scales out; those in, the values out
        n = c["T"] * c["K"]
        coded = n * (0.5 + 1 / BLOCK)
        return {"bytes": 2 * (2 * n + coded), "flops": 4.0 * n}
    R, T, K, H = c["R"], c["T"], c["K"], c["H"]
    coded = 0.5 + 1 / BLOCK
    b = R * (H * K * coded + T * K * (2 if op == "linear" else coded) + 2 * T * H)
    return {"bytes": b, "flops": 2.0 * R * T * K * H}


# --- the definitions in 64 bits ----------------------------------------------

_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _exact_quantized(x):
    """The MXFP4 values of [..., K] in float64, by counting the rounding borders below each value:
    borders lie halfway between neighbours, and a value on one goes to the even code."""
    K = x.shape[-1]
    out = torch.zeros(*x.shape[:-1], K, dtype=torch.float64, device=x.device)
    whole = torch.zeros(*x.shape[:-1], (K + BLOCK - 1) // BLOCK * BLOCK, dtype=torch.float64, device=x.device)
    whole[..., :K] = x
    blocks = whole.unflatten(-1, (-1, BLOCK))
    top = blocks.abs().amax(-1, keepdim=True)
    e = torch.floor(torch.log2(top.clamp_min(2.0 ** -140))).clamp_min(-125.0) - 2.0
    unit = ((e.long() + 1023) << 52).view(torch.float64)   # 2^e
    m = blocks.abs() / unit
    q = torch.zeros_like(m)
    for i in range(7):
        mid = (_VALUES[i] + _VALUES[i + 1]) / 2
        up = (m >= mid) if i % 2 else (m > mid)
        q += up * (_VALUES[i + 1] - _VALUES[i])
    out.copy_((q * unit * torch.sign(blocks)).flatten(-2)[..., :K])
    return out


def _exact_coded(codes, scales, K):
    value = torch.tensor(_VALUES, dtype=torch.float64, device=codes.device)
    out = torch.empty(*codes.shape[:-1], codes.shape[-1] * 2, dtype=torch.float64, device=codes.device)
    for i in range(2):
        nib = (codes >> (4 * i)) & 15
        out[..., i::2] = value[(nib & 7).long()] * (1.0 - 2.0 * (nib >> 3).double())
    unit = ((scales.long() + (1023 - 127)) << 52).view(torch.float64)   # 2^(byte - 127)
    return (out * unit.repeat_interleave(BLOCK, -1))[..., :K]


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op in ("norm", "wire"):
        T, H = s["T"], s["H"]
        if op == "norm":
            x = s["x"].double()
        else:
            q = s["codes"]
            if s["bits"] == 4:
                pair = torch.empty(T, H, dtype=torch.uint8, device=q.device)
                pair[:, 0::2], pair[:, 1::2] = q % 16, q // 16
                q = pair
            wide = [t.view(torch.float16).double().repeat_interleave(s["group"], -1) for t in (s["s"], s["z"])]
            x = q.double() * wide[0] + wide[1]
        if s["w_post"] is not None:
            x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / H + EPS) * s["w_post"].double()
        if s["gate_t"] is not None:
            x = x * s["gate_t"].double().repeat_interleave(s["gate_tokens"], 0)[:T]
        h = s["residual"].double() * s["res_scale"] + x * s["out_scale"]
        if s["w_pre"] is None:
            return [h]
        return [h, h / torch.sqrt((h * h).sum(-1, keepdim=True) / H + EPS) * s["w_pre"].double()]
    if op == "code":
        return _exact_quantized(s["x"].double())
    R, T, K, H = s["R"], s["T"], s["K"], s["H"]
    y = torch.empty(R, T, H, dtype=torch.float64, device=s["w_codes"].device)
    for r in range(R):
        if op == "linear":
            a = _exact_quantized(s["a"][r].double())
        else:
            a = _exact_coded(s["a_codes"][r], s["a_scales"][r], K)
        w = _exact_coded(s["w_codes"][r], s["w_scales"][r], K)
        y[r] = a @ w.t().contiguous()
    return y
