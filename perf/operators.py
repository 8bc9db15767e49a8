"""The operators of BitLinear's training side, in their plain form and through the package.

One pass of each: layer norm forward (bf16 out, or the 8-bit codes that a BitLinear reads), the backward pass of
layer norm and RMSNorm, the 8-bit checkpoint of a squared-ReLU gated FFN and the backward pass that reads it, and
the two matrix products of BitLinear's straight-through gradient.  ``run`` computes them with elementary torch
operations, or, where ``own`` is true, by the package's calls.

Shapes are those of the package's own layers (2560, 6912, 640, and the 2048 <-> 11008 MLP) and odd ones.  Inputs are
drawn like the package's: activations N(0, 1) with one entry in a hundred ten times larger, ternary weights with 42%
zeros, gradients of a batch whose last tokens are padding (their rows are zero).
"""
import math

import torch

own = False

EPS = 1e-5


# ---------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # a micro-batch of 16 tokens: the launch is what counts
        {"name": "layernorm_16x2560", "op": "layernorm", "M": 16, "K": 2560, "out": "bf16", "bias": True},
        # the norm before the FFN of one training batch, straight to the codes that gate and up read
        {"name": "layernorm_codes_4096x2560", "op": "layernorm", "M": 4096, "K": 2560, "out": "codes", "bias": True},
        # its backward pass
        {"name": "layernorm_bwd_4096x2560", "op": "norm_backward", "M": 4096, "K": 2560, "kind": "layer"},
        # a ragged batch through the sub-norm before a wide down projection
        {"name": "rmsnorm_bwd_999x11008", "op": "norm_backward", "M": 999, "K": 11008, "kind": "rms"},
        # the FFN's gate saved in 8 bits and its backward pass: a small batch, and a full one of the widest layer
        {"name": "glu_ckpt_256x6912", "op": "glu_checkpoint", "M": 256, "N": 6912},
        {"name": "glu_ckpt_4096x11008", "op": "glu_checkpoint", "M": 4096, "N": 11008},
        # weight gradients: a key projection on a ragged batch, the gate of one batch, the widest MLP on a long one
        {"name": "dweight_777x640x2560", "op": "backward_weight", "M": 777, "N": 640, "K": 2560},
        {"name": "dweight_2048x6912x2560", "op": "backward_weight", "M": 2048, "N": 6912, "K": 2560},
        {"name": "dweight_8192x11008x2048", "op": "backward_weight", "M": 8192, "N": 11008, "K": 2048},
        # input gradients: a few tokens, the gate's joined to the up projection's, and 2:4 weights
        {"name": "dinput_16x2560x6912", "op": "backward_input", "M": 16, "N": 2560, "K": 6912, "add": False,
         "pattern": "dense"},
        {"name": "dinput_add_2048x6912x2560", "op": "backward_input", "M": 2048, "N": 6912, "K": 2560, "add": True,
         "pattern": "dense"},
        {"name": "dinput_24_4096x11008x2048", "op": "backward_input", "M": 4096, "N": 11008, "K": 2048, "add": False,
         "pattern": "2:4"},
    ]


WIDTHS = (256, 512, 640, 2048, 2560, 6912, 11008)


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    return rng.choice(WIDTHS) if rng.random() < 0.5 else _log_int(rng, 64, 11008)


def draw(rng):
    op = rng.choice(["layernorm", "norm_backward", "glu_checkpoint", "backward_weight", "backward_input"])
    case = {"op": op, "M": _log_int(rng, 1, 8192)}
    if op == "layernorm":
        case.update(K=_width(rng), out=rng.choice(["bf16", "codes"]), bias=rng.random() < 0.7)
    elif op == "norm_backward":
        case.update(K=_width(rng), kind=rng.choice(["layer", "rms"]))
    elif op == "glu_checkpoint":
        case.update(N=_width(rng), M=min(case["M"], 4096))
    else:
        case.update(N=_width(rng), K=_width(rng))
        case["M"] = max(1, min(case["M"], int(8192 * 11008 * 2048 / (case["N"] * case["K"]))))
        if op == "backward_input":
            case.update(add=rng.random() < 0.5, pattern=rng.choice(["dense", "dense", "2:4"]))
            if case["pattern"] == "2:4":
                case["K"] = (case["K"] + 3) // 4 * 4
    return case


def work(case):
    M, N, K = case["M"], case.get("N", 0), case.get("K", 0)
    op = case["op"]
    if op == "layernorm":  # x in; y (two bytes) or codes (one) out
        return {"bytes": M * K * (4 if case["out"] == "bf16" else 3) + 8 * K + 8 * M, "flops": 8 * M * K}
    if op == "norm_backward":  # x and dy in, dx out; the weight in, its gradients out
        return {"bytes": 6 * M * K + 12 * K + 8 * M, "flops": 14 * M * K}
    if op == "glu_checkpoint":  # g, u in, three codes out; dh and two codes in, dg and du out
        return {"bytes": 15 * M * N + 24 * M, "flops": 24 * M * N}
    if op == "backward_weight":
        return {"bytes": 2 * M * N + M * K + 4 * M + 4 * N * K, "flops": 2 * M * N * K}
    packed = N * K // 4 if case["pattern"] == "dense" else N * K // 4  # 2:4: an eighth of values, an eighth of positions
    return {"bytes": 2 * M * N + packed + 2 * M * K * (2 if case["add"] else 1), "flops": 2 * M * N * K}


# ---------------------------------------------------------------------------------------------- inputs
def _activations(M, K, gen):
    x = torch.randn(M, K, device="cuda", generator=gen)
    return torch.where(torch.rand(M, K, device="cuda", generator=gen) < 0.01, 10.0 * x, x).to(torch.bfloat16)


def _gradient(M, N, gen):
    dy = 1e-3 * torch.randn(M, N, device="cuda", generator=gen)
    if M >= 8:
        dy[M - M // 8:] = 0.0  # padding at the end of the batch
    return dy.to(torch.bfloat16)


def _codes(x):
    """Per-token absmax codes and their scale: q = clamp(rne(127 x / (gamma + 1e-5)), -128, 127)."""
    x = x.float()
    gamma = x.abs().amax(1)
    q = torch.round(x * 127.0 / (gamma + 1e-5)[:, None]).clamp(-128, 127)
    return q.to(torch.int8), gamma


def _pad_to(t, cols, value):
    return torch.nn.functional.pad(t, (0, cols - t.shape[1]), value=value).contiguous()


def _pack_bits(v, width):
    """Whole numbers below 2 ** width, 8 / width to a byte, the first in the lowest bits."""
    v = v.reshape(v.shape[0], -1, 8 // width).int()
    shift = torch.arange(0, 8, width, device=v.device, dtype=torch.int32)
    return (v << shift).sum(2).to(torch.uint8)


def _packed_weights(N, K, pattern, gen):
    """Ternary weights in the package's packed layout (codes and 2:4 positions, rows a multiple of 16 bytes)."""
    u = torch.rand(N, K, device="cuda", generator=gen)
    code = (u >= 0.29).int() + (u >= 0.71).int()  # 0, 1, 2 for -1, 0, +1
    meta = None
    if pattern == "2:4":
        keep = torch.rand(N, K // 4, 4, device="cuda", generator=gen).argsort(2)[:, :, :2].sort(2).values
        code = code.reshape(N, K // 4, 4).gather(2, keep).reshape(N, K // 2)
        meta = _pack_bits(_pad_to((keep[:, :, 0] | (keep[:, :, 1] << 2)).int(), 32 * ((K + 127) // 128), 0), 4)
    codes = _pack_bits(_pad_to(code, 64 * ((code.shape[1] + 63) // 64), 1), 2)
    alpha = 0.01 + 0.04 * torch.rand(1, device="cuda", generator=gen)
    return codes, meta, alpha


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    M, N, K, op = case["M"], case.get("N"), case.get("K"), case["op"]
    s = {"case": case}
    if op in ("layernorm", "norm_backward"):
        s["x"] = _activations(M, K, gen)
        s["weight"] = 1.0 + 0.1 * torch.randn(K, device="cuda", generator=gen)
        s["bias"] = 0.1 * torch.randn(K, device="cuda", generator=gen) if case.get("bias") else None
    if op == "norm_backward":
        s["dy"] = _gradient(M, K, gen)
        if case["kind"] == "layer":  # what the forward pass saved
            s["mean"], s["rstd"] = _moments(s["x"])
    elif op == "glu_checkpoint":
        s["g"], s["u"] = (torch.randn(M, N, device="cuda", generator=gen).to(torch.bfloat16) for _ in "gu")
        s["dh"] = _gradient(M, N, gen)
    elif op == "backward_weight":
        s["dy"] = _gradient(M, N, gen)
        s["q"], s["gamma"] = _codes(_activations(M, K, gen))
    elif op == "backward_input":
        s["dy"] = _gradient(M, N, gen)
        s["codes"], s["meta"], s["alpha"] = _packed_weights(N, K, case["pattern"], gen)
        s["add"] = _gradient(M, K, gen) if case["add"] else None
    return s


# ---------------------------------------------------------------------------------------------- the plain forms
def _moments(x):
    """Mean and 1 / sqrt(variance + eps) of each row; sums in 64 bits, since codes hang on the last bit."""
    x = x.double()
    mean = x.mean(1)
    var = (x - mean[:, None]).square().mean(1).float()
    return mean.float(), (1.0 / torch.sqrt(var.double() + _f32(EPS))).float()


def _f32(v):
    return float(torch.tensor(v, dtype=torch.float32))


def _restore(q, gamma):
    return q.float() * (gamma / 127.0)[:, None]


def _bf16(x):
    return x.to(torch.bfloat16)


def _layernorm(s):
    mean, rstd = _moments(s["x"])
    y = (s["x"].float() - mean[:, None]) * rstd[:, None] * s["weight"]
    if s["bias"] is not None:
        y = y + s["bias"]
    return _bf16(y) if s["case"]["out"] == "bf16" else _bf16(_restore(*_codes(y))), mean, rstd


def _norm_backward(s):
    x, dy = s["x"].float(), s["dy"].float()
    layer = s["case"]["kind"] == "layer"
    if layer:
        mean, rstd = s["mean"], s["rstd"]
        xh = (x - mean[:, None]) * rstd[:, None]
    else:
        rstd = (1.0 / torch.sqrt(s["x"].double().square().mean(1).float().double() + _f32(EPS))).float()
        xh = x * rstd[:, None]
    a = dy * s["weight"]
    t = a - xh * (a * xh).mean(1, keepdim=True)
    if layer:
        t = t - a.mean(1, keepdim=True)
    dx, dw = _bf16(t * rstd[:, None]), (dy * xh).sum(0)
    return (dx, dw, dy.sum(0)) if layer else (dx, dw)


def _glu_checkpoint(s):
    g, u, dh = s["g"].float(), s["u"].float(), s["dh"].float()
    h = _bf16(_bf16(torch.relu(g).square()).float() * u)
    r = torch.relu(_restore(*_codes(g)))
    return _bf16(2.0 * dh * r * _restore(*_codes(u))), _bf16(dh * r.square()), _bf16(_restore(*_codes(h)))


def _backward_weight(s):
    return s["dy"].float().t() @ _bf16(_restore(s["q"], s["gamma"])).float()


def _unpack_bits(b, width):
    shift = torch.arange(0, 8, width, device=b.device, dtype=torch.int32)
    return ((b.int()[:, :, None] >> shift) & ((1 << width) - 1)).reshape(b.shape[0], -1)


def _ternary(s):
    N, K = s["case"]["N"], s["case"]["K"]
    code = _unpack_bits(s["codes"], 2)
    if s["meta"] is None:
        return code[:, :K].float() - 1.0
    nib = _unpack_bits(s["meta"], 4)[:, :K // 4]
    at = torch.stack([nib & 3, nib >> 2], 2).long()
    kept = code[:, :K // 2].reshape(N, K // 4, 2).float() - 1.0
    return torch.zeros(N, K // 4, 4, device=kept.device).scatter_(2, at, kept).reshape(N, K)


def _backward_input(s):
    dx = (s["dy"].float() @ _ternary(s)) * s["alpha"]
    return _bf16(dx if s["add"] is None else dx + s["add"].float())


# ---------------------------------------------------------------------------------------------- one pass
def _run_own(s):
    import ternary_weight_linear_fwd_b200 as bl
    case, op = s["case"], s["case"]["op"]
    if op == "layernorm":
        if case["out"] == "bf16":
            return bl.layernorm(s["x"], s["weight"], s["bias"], EPS, want_stats=True)
        q, gamma, _, mean, rstd = bl.layernorm_quant_act(s["x"], s["weight"], s["bias"], EPS, want_stats=True)
        return bl.dequant_act(q, gamma), mean, rstd
    if op == "norm_backward":
        if case["kind"] == "layer":
            return bl.layernorm_backward(s["dy"], s["x"], s["weight"], s["mean"], s["rstd"])
        return bl.rmsnorm_backward(s["dy"], s["x"], s["weight"], EPS)
    if op == "glu_checkpoint":
        c = bl.relu2_glu_quant_act(s["g"], s["u"])
        dg, du = bl.relu2_glu_backward(s["dh"], c.q_g, c.gamma_g, c.q_u, c.gamma_u)
        return dg, du, bl.dequant_act(c.q_h, c.gamma_h)
    if op == "backward_weight":
        return bl.backward_weight(s["dy"], s["q"], s["gamma"])
    n, m = (2, 4) if case["pattern"] == "2:4" else (0, 0)
    w = bl.PackedWeights(case["N"], case["K"], n, m, s["codes"], s["meta"], s["alpha"])
    return bl.backward_input(w, s["dy"], add=s["add"])


def run(state):
    if own:
        return _run_own(state)
    return {"layernorm": _layernorm, "norm_backward": _norm_backward, "glu_checkpoint": _glu_checkpoint,
            "backward_weight": _backward_weight, "backward_input": _backward_input}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------------------------- in 64 bits
def _exact_codes(x):
    """The value that each entry's 8-bit code stands for, x in 64 bits."""
    gamma = x.abs().max(1, keepdim=True).values
    return torch.clamp(torch.round(127.0 * x / (gamma + 1e-5)), -128, 127) * gamma / 127.0


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    d = {k: v.double() for k, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if op == "layernorm":
        mean = d["x"].sum(1, keepdim=True) / case["K"]
        c = d["x"] - mean
        rstd = ((c * c).sum(1, keepdim=True) / case["K"] + EPS).rsqrt()
        y = c * rstd * d["weight"] + (d["bias"] if "bias" in d else 0.0)
        return y if case["out"] == "bf16" else _exact_codes(y), mean[:, 0], rstd[:, 0]
    if op == "norm_backward":
        x, dy, w, K = d["x"], d["dy"], d["weight"], case["K"]
        if case["kind"] == "layer":
            r, c = d["rstd"][:, None], x - d["mean"][:, None]
            p = torch.einsum("mk,k,mk->m", dy, w, c)[:, None] * r * r / K
            dx = r * (dy * w - torch.einsum("mk,k->m", dy, w)[:, None] / K - c * p)
            return dx, torch.einsum("mk,mk->k", dy, c * r), torch.einsum("mk->k", dy)
        r = (torch.einsum("mk,mk->m", x, x)[:, None] / K + EPS).rsqrt()
        p = torch.einsum("mk,k,mk->m", dy, w, x)[:, None] * r * r / K
        return r * (dy * w - x * p), torch.einsum("mk,mk->k", dy, x * r)
    if op == "glu_checkpoint":
        zero = torch.zeros((), dtype=torch.float64, device="cuda")
        h = (torch.maximum(d["g"], zero) ** 2).to(torch.bfloat16).double() * d["u"]
        g, u = torch.maximum(_exact_codes(d["g"]), zero), _exact_codes(d["u"])
        return d["dh"] * g * u * 2, g * d["dh"] * g, _exact_codes(h.to(torch.bfloat16).double())
    if op == "backward_weight":  # the checkpoint restores the activation in its own type, bf16
        scale = (d["gamma"] / 127.0).float().double()  # one rounding each: the scale, the product, the bf16 value
        x = (s["q"].double() * scale[:, None]).float().to(torch.bfloat16).double()
        return torch.einsum("mn,mk->nk", d["dy"], x)
    N, K = case["N"], case["K"]
    c = s["codes"].long()
    t = torch.stack([c % 4, c // 4 % 4, c // 16 % 4, c // 64], 2).reshape(N, -1).double() - 1
    if case["pattern"] == "2:4":
        b = s["meta"].long()
        at = torch.stack([b % 4, b // 4 % 4, b // 16 % 4, b // 64], 2).reshape(N, -1)[:, :K // 2]
        at = at + torch.arange(K // 4, device="cuda").repeat_interleave(2) * 4
        t = torch.zeros(N, K, dtype=torch.float64, device="cuda").scatter_(1, at, t[:, :K // 2])
    dx = torch.einsum("mn,nk->mk", d["dy"], t[:, :K]) * d["alpha"]
    return dx + d["add"] if case["add"] else dx
