"""The 8-bit integer layer (SmoothQuant W8A8) and the channels-last group norm, as measured workloads.

Four operators, each in two forms: the plain one in elementary torch operations, and the library's.

  linear_i8    Y[m, n] = sx[m] sw[n] sum_k Xq[m, k] Wq[n, k] + bias[n]                  (int8 codes, exact sum)
  forward_i8   the layer from its 16-bit input: X_hat = f32(X inv_s), quantized row by row
               (sx = f32(a / 127), a the row's largest magnitude; q = rint(f32(X_hat f32(127 / a)))), then linear_i8
  group_norm   Y = act(gamma (X - mean) / sqrt(var + eps) + beta), statistics over the rows and the channels of a
               group, X of shape [batch, rows, channels]
  norm_i8      group_norm in float32, quantized as forward_i8 quantizes, then linear_i8: the norm in front of a
               projection
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5
TINY = 2.0 ** -100          # a row whose largest magnitude is below this is all zeros in 8 bits


def listed():
    return [
        # generating one token: the weight is read once, 50 MB, and hardly any arithmetic
        dict(name="linear one token", op="linear_i8", M=1, K=4096, N=12288, type="bf16", bias=True),
        # the text tokens of a prompt, a width that is no multiple of the tiles
        dict(name="linear prompt 77", op="linear_i8", M=77, K=2048, N=1288, type="fp16", bias=False),
        # the square layer of the rank sweep
        dict(name="linear 4096 cubed", op="linear_i8", M=4096, K=4096, N=4096, type="bf16", bias=True),
        # four images of 4608 tokens in one batch
        dict(name="linear four images", op="linear_i8", M=18432, K=4096, N=4096, type="bf16", bias=False),
        # a conditioning vector through a layer: the smallest call, where latency counts
        dict(name="layer one row", op="forward_i8", M=1, K=1280, N=5120, type="fp16", bias=True),
        # odd sizes and a float32 result
        dict(name="layer ragged", op="forward_i8", M=333, K=1040, N=1001, type="bf16", out="fp32", bias=True),
        # one image's tokens into a fused query, key and value projection
        dict(name="layer one image", op="forward_i8", M=4608, K=4096, N=12288, type="bf16", bias=True),
        # a residual block of a U-Net at its middle resolution, two prompts
        dict(name="norm block", op="group_norm", B=2, S=4096, C=640, G=32, type="bf16", act="silu"),
        # float32 activations, an odd picture, no activation
        dict(name="norm odd fp32", op="group_norm", B=3, S=1961, C=320, G=32, type="fp32", act="none"),
        # the last block of an image decoder: a megapixel of 128 channels
        dict(name="norm megapixel", op="group_norm", B=1, S=1048576, C=128, G=32, type="bf16", act="silu"),
        # the norm in front of a transformer block's first projection, low resolution
        dict(name="norm and projection 1280", op="norm_i8", B=2, S=1024, C=1280, G=32, N=1280, type="fp16",
             act="none", bias=True),
        # the same where the picture is large and the channels few
        dict(name="norm and projection 320", op="norm_i8", B=1, S=16384, C=320, G=32, N=320, type="bf16",
             act="none", bias=True),
    ]


def draw(rng):
    def spread(lo, hi):
        return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))

    op = rng.choice(["linear_i8", "forward_i8", "group_norm", "norm_i8"])
    kind = rng.choice(["bf16", "fp16"])
    if op in ("linear_i8", "forward_i8"):
        M, K, N = spread(1, 18432), 16 * spread(4, 768), spread(16, 12288)
        while M * K * N > 18432 * 4096 * 4096:
            M = max(1, M // 2)
        c = dict(op=op, M=M, K=K, N=N, type=kind, bias=rng.random() < 0.5)
        if rng.random() < 0.25:
            c["out"] = "fp32"
        return c
    act = rng.choice(["none", "silu", "gelu"])
    G = rng.choice([1, 4, 8, 16, 32])
    if op == "group_norm":
        C = G * spread(1, 1280 // G)
        B = spread(1, 4)
        S = spread(1, max(1, min(1 << 20, (1 << 27) // (B * C))))
        return dict(op=op, B=B, S=S, C=C, G=G, type=rng.choice(["bf16", "fp16", "fp32"]), act=act)
    C = 64 * spread(1, 20)
    B = spread(1, 4)
    return dict(op=op, B=B, S=spread(1, 16384 // B), C=C, G=G, N=spread(16, 2560), type=kind, act=act,
                bias=rng.random() < 0.5)


def _out(case):
    return TYPES[case.get("out", case["type"])]


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev).manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=dev, dtype=torch.float32)

    def uniform(lo, hi, *shape):
        return lo + (hi - lo) * torch.rand(*shape, generator=g, device=dev, dtype=torch.float32)

    s = {"case": dict(case)}
    op, kind = case["op"], TYPES[case["type"]]
    if op != "group_norm":
        K, N = case.get("K", case.get("C")), case["N"]
        # codes of a per-channel quantized weight: normal, the largest of each channel at 127
        w = normal(N, K)
        a = w.abs().amax(dim=1, keepdim=True)
        s["Wq"] = torch.round(w * (127.0 / a)).to(torch.int8)
        s["sw"] = (0.02 * a / 127.0).reshape(-1).contiguous()
        s["bias"] = 0.3 * normal(N) if case["bias"] else None
    if op == "linear_i8":
        M, K = case["M"], case["K"]
        x = normal(M, K)
        a = x.abs().amax(dim=1, keepdim=True)
        s["Xq"] = torch.round(x * (127.0 / a)).to(torch.int8)
        s["sx"] = (a * uniform(0.5, 2.0, M, 1) / 127.0).reshape(-1).contiguous()
    elif op == "forward_i8":
        M, K = case["M"], case["K"]
        # one channel in a hundred is an outlier, which the smoothing halves in the exponent
        amp = torch.where(uniform(0, 1, K) < 0.01, uniform(20, 60, K), torch.ones(K, device=dev))
        s["X"] = (normal(M, K) * amp).to(kind)
        s["inv_s"] = (uniform(0.8, 1.25, K) / amp.sqrt()).contiguous()
    else:
        B, S, C = case["B"], case["S"], case["C"]
        # channels with means and spreads of their own
        s["X"] = (normal(B, S, C) * uniform(0.3, 2.0, C) + uniform(-1.0, 1.0, C)).to(kind)
        s["gamma"], s["beta"] = uniform(0.5, 1.5, C), 0.2 * normal(C)
        if op == "norm_i8":
            s["inv_s"] = uniform(0.5, 2.0, C)
    return s


# ------------------------------------------------------------------ the plain forms --
def _plain_linear(xq, sx, s, out):
    y = torch.matmul(xq.to(torch.float32), s["Wq"].to(torch.float32).t()) * sx[:, None] * s["sw"][None, :]
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(out)


def _plain_quantize(xh):
    a = xh.abs().amax(dim=1, keepdim=True)
    steps = torch.full_like(a, 127.0)
    zero = a < TINY
    q = torch.round(xh * (steps / torch.where(zero, steps, a)))
    return torch.where(zero, torch.zeros_like(q), q), torch.where(zero, torch.zeros_like(a), a / steps).reshape(-1)


def _plain_norm(s, case):
    B, S, C, G = case["B"], case["S"], case["C"], case["G"]
    x = s["X"].to(torch.float32).reshape(B, S, G, C // G)
    mean = x.mean(dim=(1, 3), keepdim=True)
    d = x - mean
    var = (d * d).mean(dim=(1, 3), keepdim=True)
    y = (d / torch.sqrt(var + EPS)).reshape(B, S, C) * s["gamma"] + s["beta"]
    if case["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif case["act"] == "gelu":
        y = y / (1.0 + torch.exp(-2.0 * math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    return y


def _plain(s):
    case = s["case"]
    op, out = case["op"], _out(case)
    if op == "linear_i8":
        return _plain_linear(s["Xq"], s["sx"], s, out)
    if op == "forward_i8":
        q, sx = _plain_quantize(s["X"].to(torch.float32) * s["inv_s"])
        return _plain_linear(q, sx, s, out)
    y = _plain_norm(s, case)
    if op == "group_norm":
        return y.to(out)
    q, sx = _plain_quantize(y.reshape(-1, case["C"]) * s["inv_s"])
    return _plain_linear(q, sx, s, out)


# ------------------------------------------------------------- the library's operators --
def _buffers(s):
    """Output, quantized activations and workspace, kept from call to call as a program keeps them."""
    b = s.get("buffers")
    if b is None:
        from w4a4_rank_absorbed_b200 import svdq as L
        case, dev = s["case"], s["X"].device if "X" in s else s["Xq"].device
        b = s["buffers"] = {"L": L}
        if case["op"] == "group_norm":
            b["Y"] = torch.empty_like(s["X"])
        else:
            M = case["M"] if "M" in case else case["B"] * case["S"]
            b["Y"] = torch.empty((M, case["N"]), dtype=_out(case), device=dev)
        if case["op"] == "forward_i8":
            b["work"] = torch.empty(L.svdq_forward_i8_workspace_bytes(case["M"], case["K"]), dtype=torch.uint8,
                                    device=dev)
        if case["op"] in ("group_norm", "norm_i8"):
            b["work"] = L.new_group_norm_workspace(case["B"], case["S"], case["C"], case["G"], dev)
            b["act"] = {"none": L.SVDQ_ACT_NONE, "silu": L.SVDQ_ACT_SILU, "gelu": L.SVDQ_ACT_GELU}[case["act"]]
        if case["op"] == "norm_i8":
            b["Xq"] = torch.empty((M, case["C"]), dtype=torch.int8, device=dev)
            b["sx"] = torch.empty(M, dtype=torch.float32, device=dev)
    return b


def _library(s):
    case, b = s["case"], _buffers(s)
    op, L = case["op"], b["L"]
    if op == "linear_i8":
        L.svdq_linear_i8(s["Xq"], s["sx"], s["Wq"], s["sw"], s["bias"], b["Y"], case["M"], case["N"], case["K"])
    elif op == "forward_i8":
        L.svdq_forward_i8(s["X"], case["M"], case["K"], s["inv_s"], s["Wq"], s["sw"], s["bias"], b["Y"], case["N"],
                          b["work"])
    elif op == "group_norm":
        L.svdq_group_norm(s["X"], case["B"], case["S"], case["C"], case["G"], s["gamma"], s["beta"], EPS, b["act"],
                          b["Y"], b["work"])
    else:
        L.svdq_group_norm_quantize_i8(s["X"], case["B"], case["S"], case["C"], case["G"], s["gamma"], s["beta"], EPS,
                                      b["act"], s["inv_s"], b["Xq"], b["sx"], b["work"])
        L.svdq_linear_i8(b["Xq"], b["sx"], s["Wq"], s["sw"], s["bias"], b["Y"], case["B"] * case["S"], case["N"],
                         case["C"])
    return b["Y"]


def run(state):
    return _library(state) if own else _plain(state)


# ------------------------------------------------------------------------- the floor --
def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    si, so = size[case["type"]], size[case.get("out", case["type"])]
    if op == "group_norm":
        n = case["B"] * case["S"] * case["C"]
        return {"bytes": n * (si + so) + 8 * case["C"], "flops": 8 * n}
    M = case["M"] if "M" in case else case["B"] * case["S"]
    K, N = case.get("K", case.get("C")), case["N"]
    weight = N * K + 4 * N * (2 if case["bias"] else 1)
    if op == "linear_i8":
        return {"bytes": M * K + 4 * M + weight + M * N * so, "flops": 2 * M * N * K}
    return {"bytes": M * K * si + 4 * K * (1 if op == "forward_i8" else 3) + weight + M * N * so,
            "flops": 2 * M * N * K}


# ---------------------------------------------------------------- values in 64 bits --
def _exact_layer(q, sx, s):
    """q, sx: whole numbers and scales in 64 bits."""
    y = torch.mm(q, s["Wq"].double().T)
    y.mul_(sx.unsqueeze(1)).mul_(s["sw"].double())
    return y if s["bias"] is None else y.add_(s["bias"].double())


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear_i8":
        return _exact_layer(s["Xq"].double(), s["sx"].double(), s)
    if op == "forward_i8":
        # the quantizer is defined by its binary32 steps: the codes are those, the rest is in 64 bits
        import numpy as np
        xh = np.multiply(s["X"].float().cpu().numpy(), s["inv_s"].cpu().numpy(), dtype=np.float32)
        top = np.max(np.abs(xh), axis=1)
        live = top >= np.float32(TINY)
        up = np.divide(np.float32(127), top, dtype=np.float32, where=live, out=np.zeros_like(top))
        q = np.rint(np.multiply(xh, up[:, None], dtype=np.float32))
        sx = np.where(live, np.divide(top, np.float32(127), dtype=np.float32), np.float32(0))
        dev = s["X"].device
        return _exact_layer(torch.from_numpy(q).to(dev).double(), torch.from_numpy(sx).to(dev).double(), s)
    B, S, C, G = case["B"], case["S"], case["C"], case["G"]
    x = s["X"].double().view(B, S, G, C // G)
    var, mean = torch.var_mean(x, dim=(1, 3), keepdim=True, unbiased=False)
    y = x.sub(mean).mul_(torch.rsqrt(var + EPS)).view(B, S, C)
    y.mul_(s["gamma"].double()).add_(s["beta"].double())
    if case["act"] == "silu":
        y = y * torch.sigmoid(y)
    elif case["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y ** 3)))
    if op == "group_norm":
        return y
    xh = y.view(B * S, C).mul_(s["inv_s"].double())
    top = xh.abs().amax(1)
    live = top >= TINY
    q = torch.round(xh * torch.where(live, 127.0 / top.clamp_min(TINY), torch.zeros_like(top)).unsqueeze(1))
    return _exact_layer(q, torch.where(live, top / 127.0, torch.zeros_like(top)), s)
