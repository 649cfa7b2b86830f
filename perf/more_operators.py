"""Cases and plain forms of the operators between the decoder stack's linears, and of linears on 8-bit operands.

Three operators, as a training step of the decoder stack (or its scoring and decoding) meets them:

norm    Root-mean-square norm of x (+ residual), s = x + residual being the new residual stream: y = s r w with
        r = 1 / sqrt(mean(s^2) + eps), in the stream's type or in FP8 (E4M3 under amax / 448 per 128 of a row); with
        the gradients of s (one more may come in for s itself) and of w.
fp8     A linear layer Y = X W^T on FP8 operands: X under a scale per 128 of a row, W under one per 128 x 128; from
        stored codes (serving) or fp32 masters (training, with dX = Q(dY) W^ and dW = Q(dY^T) Q(X^), W^ and X^ the
        forward's quantised tensors, X^ grouped anew along the tokens).
ffn     The gated feed-forward block Y = (act(X Wg^T) * (X Wu^T)) Wd^T in bf16 and the gradients of X and the weights.
"""
import math

import torch

own = False
DEV = "cuda"
VOCAB, D, F, TOKENS = 50304, 1024, 4096, 16384  # the 370M-style decoder stack
EPS = 1e-6


def listed():
    return [
        # the stream of one sequence that decodes a token, into the operand of an FP8 projection
        dict(name="norm one token", op="norm", rows=1, cols=D, dtype="bf16", residual=True, fp8=True, grad=False),
        # a training batch before the FP8 projections of a block
        dict(name="norm fp8 370M", op="norm", rows=TOKENS, cols=D, dtype="bf16", residual=True, fp8=True, grad=False),
        # the same stream in training, both passes
        dict(name="norm train 370M", op="norm", rows=TOKENS, cols=D, dtype="bf16", residual=True, fp8=False, grad=True),
        # an fp32 stream of odd width, its first norm (nothing to add yet)
        dict(name="norm train f32 ragged", op="norm", rows=1555, cols=1003, dtype="f32", residual=False, fp8=False, grad=True),
        # one token through a gate projection while decoding
        dict(name="fp8 one token", op="fp8", M=1, K=D, N=F, train=False),
        # the head for a batch of sequences that each decode one token
        dict(name="fp8 head 24 tokens", op="fp8", M=24, K=D, N=VOCAB, train=False),
        # a fine-tuning batch of uneven length through a small projection
        dict(name="fp8 train ragged", op="fp8", M=777, K=656, N=1552, train=True),
        # a gate projection of the 370M-style stack in training
        dict(name="fp8 train 370M", op="fp8", M=TOKENS, K=D, N=F, train=True),
        # one token through the 370M-style stack's feed-forward block
        dict(name="ffn one token", op="ffn", T=1, D=D, F=F, act="silu", grad=False),
        # scoring a prompt
        dict(name="ffn prompt", op="ffn", T=300, D=D, F=F, act="silu", grad=False),
        # a small model's step with another activation and uneven sizes
        dict(name="ffn train ragged", op="ffn", T=1235, D=528, F=1552, act="gelu", grad=True),
        # the feed-forward block of the 370M-style stack in training
        dict(name="ffn train 370M", op="ffn", T=TOKENS, D=D, F=F, act="silu", grad=True),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def log16(lo, hi):
        return max(16, log(lo, hi) // 16 * 16)

    op = rng.choice(["norm", "norm", "fp8", "fp8", "ffn", "ffn"])
    if op == "norm":
        fp8 = rng.random() < 0.5
        cols = log16(64, F) if fp8 else log(33, F)
        return dict(op=op, rows=log(1, TOKENS * D // max(D, cols)), cols=cols, dtype=rng.choice(["bf16", "bf16", "f32"]),
                    residual=rng.random() < 0.7, fp8=fp8, grad=not fp8 and rng.random() < 0.7)
    if op == "fp8":
        if rng.random() < 0.5:
            return dict(op=op, M=log(1, 512), K=log16(128, F), N=log16(128, VOCAB), train=False)
        return dict(op=op, M=log(16, TOKENS), K=log16(128, D), N=log16(128, F), train=True)
    grad = rng.random() < 0.6
    return dict(op=op, T=log(1, TOKENS), D=log16(96, D), F=log16(128, F), act=rng.choice(["silu", "silu", "gelu", "gelu_tanh"]),
                grad=grad)


# ---- inputs ------------------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, rows, cols, std, outliers=0.0):
    """Normal values; a share of the columns several times as large, as activations and gradients have them."""
    x = torch.randn(rows, cols, generator=g, device=DEV).mul_(std)
    if outliers:
        x.mul_(torch.where(torch.rand(cols, generator=g, device=DEV) < outliers, 8.0, 1.0))
    return x


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "norm":
        dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
        n, k = case["rows"], case["cols"]
        s = dict(case=case, x=_normal(g, n, k, 0.5, 0.03).to(dt), w=1.0 + _normal(g, 1, k, 0.1)[0])
        if case["residual"]:
            s["residual"] = _normal(g, n, k, 1.5, 0.03).to(dt)
        if case["grad"]:
            s["dy"] = _normal(g, n, k, 1e-3, 0.03).to(dt)
            s["dsum"] = _normal(g, n, k, 1e-3).to(dt) if case["residual"] else None
        return s
    if op == "fp8":
        M, K, N = case["M"], case["K"], case["N"]
        s = dict(case=case, X=_normal(g, M, K, 1.0, 0.03).to(torch.bfloat16))
        s["X"][M // 2, :] *= 0.0 if M > 4 else 1.0  # a padding position
        W = _normal(g, N, K, 0.02)
        if case["train"]:
            return dict(s, W=W, dY=_normal(g, M, N, 1e-3, 0.03).to(torch.bfloat16))
        q, scale = _fp8_block(W)
        codes = torch.zeros(N, -(-K // 128) * 128, dtype=torch.uint8, device=DEV)
        codes[:, :K] = q.to(torch.float8_e4m3fn).view(torch.uint8)
        return dict(s, codes=codes, scales=scale)
    T, d, f = case["T"], case["D"], case["F"]
    s = dict(case=case, X=_normal(g, T, d, 1.0, 0.03).to(torch.bfloat16))
    for name, rows, cols in (("Wg", f, d), ("Wu", f, d), ("Wd", d, f)):
        s[name] = _normal(g, rows, cols, 0.6 / math.sqrt(cols)).to(torch.bfloat16)
    if case["grad"]:
        s["dY"] = _normal(g, T, d, 1e-3, 0.03).to(torch.bfloat16)
    return s


# ---- plain forms: elementary operations in 32 bits -----------------------------------------------------------------
def _scale(amax):
    """The stored scale amax / 448 (a tensor divides: a number would be multiplied by its rounded reciprocal), and
    what elements are multiplied by; a group below 2^-100 counts as empty."""
    s = torch.where(amax < 2.0 ** -100, torch.zeros_like(amax), amax / torch.full_like(amax, 448.0))
    return s, torch.where(s > 0, 1.0 / s, torch.zeros_like(s))


def _e4m3(v):
    """v to the nearest value of E4M3 (4 exponent bits, 3 of mantissa, up to 448), ties to even."""
    v = v.clamp(-448.0, 448.0)
    e = torch.frexp(v)[1].clamp(min=-5) - 4  # of a step of v's binade, 2^-9 at least
    step = ((e + 127) << 23).view(torch.float32)
    up = ((127 - e) << 23).view(torch.float32)
    return torch.round(v * up) * step


def _fp8_row(x):
    """Elements and scales of fp32 x [rows, len] in groups of 128 along a row."""
    rows, n = x.shape
    p = torch.zeros(rows, -(-n // 128) * 128, dtype=torch.float32, device=x.device)
    p[:, :n] = x
    p = p.view(rows, -1, 128)
    s, inv = _scale(p.abs().amax(2, keepdim=True))
    return _e4m3(p * inv).reshape(rows, -1)[:, :n], s.squeeze(2)


def _fp8_block(x):
    """Elements and scales of fp32 x [rows, len] in blocks of 128 x 128."""
    rows, n = x.shape
    nr, nc = -(-rows // 128), -(-n // 128)
    p = torch.zeros(nr * 128, nc * 128, dtype=torch.float32, device=x.device)
    p[:rows, :n] = x
    p = p.view(nr, 128, nc, 128)
    s, inv = _scale(p.abs().amax((1, 3), keepdim=True))
    return _e4m3(p * inv).reshape(nr * 128, nc * 128)[:rows, :n], s.view(nr, nc)


def _row_values(q, s):
    return q * s.repeat_interleave(128, 1)[:, : q.shape[1]]


def _block_values(q, s):
    return q * s.repeat_interleave(128, 0).repeat_interleave(128, 1)[: q.shape[0], : q.shape[1]]


def _plain_norm(st):
    c, x, w = st["case"], st["x"], st["w"]
    s = (x.float() + st["residual"].float()).to(x.dtype) if c["residual"] else x
    v = s.float()
    r = torch.rsqrt(v.pow(2).mean(1, keepdim=True) + EPS)
    xh = v * r
    y = xh * w
    out = [s] if c["residual"] else []
    if c["fp8"]:
        return out + [_row_values(*_fp8_row(y)).to(torch.bfloat16)]
    out.append(y.to(x.dtype))
    if c["grad"]:
        g = st["dy"].float()
        gw = g * w
        ds = r * (gw - xh * (gw * xh).mean(1, keepdim=True))
        if st["dsum"] is not None:
            ds = ds + st["dsum"].float()
        out += [ds.to(x.dtype), (g * xh).sum(0)]
    return out


def _plain_fp8(st):
    c = st["case"]
    X = _row_values(*_fp8_row(st["X"].float()))
    if not c["train"]:
        q = st["codes"].view(torch.float8_e4m3fn)[:, : c["K"]].float()
        return (X @ _block_values(q, st["scales"]).t()).to(torch.bfloat16)
    W = _block_values(*_fp8_block(st["W"]))
    dY = st["dY"].float()
    dX = _row_values(*_fp8_row(dY)) @ W
    dW = _row_values(*_fp8_row(dY.t().contiguous())) @ _row_values(*_fp8_row(X.t().contiguous())).t()
    return (X @ W.t()).to(torch.bfloat16), dX.to(torch.bfloat16), dW


def _activation(name, g):
    """act(g) and its derivative."""
    if name == "silu":
        p = 1.0 / (1.0 + torch.exp(-g))
        return g * p, p * (1.0 + g * (1.0 - p))
    if name == "gelu":
        p = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * p, p + g * torch.exp(-0.5 * g * g) * (1.0 / math.sqrt(2.0 * math.pi))
    a = math.sqrt(2.0 / math.pi)
    t = torch.tanh(a * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * a * (1.0 + 3 * 0.044715 * g * g)


def _plain_ffn(st):
    X, Wg, Wu, Wd = (st[n].float() for n in ("X", "Wg", "Wu", "Wd"))
    G, U = X @ Wg.t(), X @ Wu.t()
    a, da = _activation(st["case"]["act"], G)
    H = a * U
    Y = (H @ Wd.t()).to(torch.bfloat16)
    if not st["case"]["grad"]:
        return Y
    dY = st["dY"].float()
    dH = dY @ Wd
    dG, dU = dH * U * da, dH * a
    grads = dG @ Wg + dU @ Wu, dG.t() @ X, dU.t() @ X, dY.t() @ H
    return [Y] + [t.to(torch.bfloat16) for t in grads]


# ---- one pass ------------------------------------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return dict(norm=_plain_norm, fp8=_plain_fp8, ffn=_plain_ffn)[s["case"]["op"]](s)


def _own(s):
    import bit_fully_quantized_amd as tj2

    c = s["case"]
    if c["op"] == "norm":
        y, total, rstd = tj2.rms_norm_fwd(s["x"], s["w"], residual=s.get("residual"), eps=EPS, fp8=c["fp8"])
        out = [total] if c["residual"] else []
        if c["fp8"]:
            return out + [tj2.fp8_dequantize(y)]
        out.append(y)
        if c["grad"]:
            out += tj2.rms_norm_bwd(s["dy"], total, s["w"], rstd, dsum=s["dsum"])
        return out
    if c["op"] == "fp8":
        if not c["train"]:
            Wq = tj2.QTensor.wrap(tj2.FP8_BLOCK, c["N"], c["K"], s["codes"], None, s["scales"])
            return tj2.fp8_linear_fwd(s["X"], None, c["N"], Wq=Wq)[0]
        Y, saved = tj2.fp8_linear_fwd(s["X"], s["W"], c["N"])
        dX, dW = tj2.fp8_linear_bwd(s["dY"], saved, c["K"])
        return Y, dX, dW
    Y, saved = tj2.gated_ffn_fwd(s["X"], s["Wg"], s["Wu"], s["Wd"], activation=c["act"], save=c["grad"])
    if not c["grad"]:
        return Y
    return [Y] + list(tj2.gated_ffn_bwd(s["dY"], s["X"], s["Wg"], s["Wu"], s["Wd"], saved, activation=c["act"]))


def work(case):
    op = case["op"]
    if op == "norm":
        n, b = case["rows"] * case["cols"], 2 if case["dtype"] == "bf16" else 4
        r = 1 if case["residual"] else 0
        total = n * b * (1 + 2 * r) + n * (2 if case["fp8"] else b) + 4 * case["cols"]
        if case["grad"]:  # dy (and what comes in for s), ds, dw; s is read again
            total += n * b * (3 + r) + 4 * case["cols"] - n * b * (1 - r)
        return dict(bytes=total, flops=n * (20 if case["grad"] else 8))
    if op == "fp8":
        M, K, N = case["M"], case["K"], case["N"]
        if not case["train"]:
            return dict(bytes=2 * M * K + N * K + 2 * M * N, flops=2 * M * N * K)
        return dict(bytes=2 * M * K + 4 * N * K + 2 * M * N + 2 * M * N + 2 * M * K + 4 * N * K, flops=6 * M * N * K)
    T, d, f = case["T"], case["D"], case["F"]
    if not case["grad"]:
        return dict(bytes=4 * T * d + 6 * d * f, flops=6 * T * d * f)
    return dict(bytes=8 * T * d + 12 * d * f, flops=18 * T * d * f)


# ---- the definitions in 64 bits, written apart ---------------------------------------------------------------------
def _exact_fp8(x, rows, cols):
    """The values that x (64 bits) has on E4M3 under a scale per tile of rows x cols. The scale, its reciprocal, the
    scaled element and the value are fp32 by definition (bf16 inputs often lie on a border between two elements)."""
    m, n = x.shape
    p = torch.nn.functional.pad(x, (0, -n % cols, 0, -m % rows))
    t = p.reshape(p.shape[0] // rows, rows, p.shape[1] // cols, cols).transpose(1, 2)
    top = t.abs().flatten(2).max(2).values[:, :, None, None]
    scale = torch.where(top < 2.0 ** -100, 0.0, top / 448.0).float().double()
    inverse = torch.where(scale > 0, 1.0 / scale, 0.0).float().double()
    v = (t * inverse).float().double().clamp(-448, 448)
    quantum = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    q = v / quantum
    whole = torch.floor(q)
    part = q - whole
    up = (part > 0.5) | ((part == 0.5) & (whole % 2 != 0))
    out = ((whole + up) * quantum * scale).float().double()
    return out.transpose(1, 2).reshape(p.shape)[:m, :n]


def _exact_norm(st):
    c, w = st["case"], st["w"].double()
    s = st["x"].double()
    if c["residual"]:
        s = (s + st["residual"].double()).to(st["x"].dtype).double()
    n = s.shape[1]
    r = 1.0 / torch.sqrt((s * s).sum(1, keepdim=True) / n + EPS)
    y = s * r * w
    out = [s] if c["residual"] else []
    out.append(_exact_fp8(y, 1, 128) if c["fp8"] else y)
    if c["grad"]:
        g = st["dy"].double()
        ds = r * g * w - s * r ** 3 * (g * w * s).sum(1, keepdim=True) / n
        out += [ds if st["dsum"] is None else ds + st["dsum"].double(), (g * s * r).sum(0)]
    return out


def _exact_linear(st):
    c = st["case"]
    X = _exact_fp8(st["X"].double(), 1, 128)
    if not c["train"]:
        b = st["codes"][:, : c["K"]].long()
        e, m = (b >> 3) & 15, (b & 7).double()
        mag = torch.where(e > 0, torch.exp2(e.double() - 7) * (1 + m / 8), m * 2.0 ** -9)
        W = torch.where(b > 127, -mag, mag)
        i = torch.arange(c["N"], device=DEV) // 128
        j = torch.arange(c["K"], device=DEV) // 128
        return X @ (W * st["scales"].double()[i][:, j]).T
    W = _exact_fp8(st["W"].double(), 128, 128)
    dY = st["dY"].double()
    return [X @ W.T, _exact_fp8(dY, 1, 128) @ W, _exact_fp8(dY, 128, 1).T @ _exact_fp8(X, 128, 1)]


def _exact_ffn(st):
    X, Wg, Wu, Wd = (st[n].double() for n in ("X", "Wg", "Wu", "Wd"))
    G, U = X @ Wg.T, X @ Wu.T
    act = st["case"]["act"]
    if act == "silu":
        sig = torch.sigmoid(G)
        a, slope = G * sig, sig + G * sig * (1 - sig)
    elif act == "gelu":
        cdf = 0.5 * torch.special.erfc(-G / math.sqrt(2))
        a, slope = G * cdf, cdf + G * torch.exp(-G * G / 2) / math.sqrt(2 * math.pi)
    else:
        k = math.sqrt(2 / math.pi)
        sig = torch.sigmoid(2 * k * (G + 0.044715 * G ** 3))  # (1 + tanh z) / 2
        a, slope = G * sig, sig + G * sig * (1 - sig) * 2 * k * (1 + 3 * 0.044715 * G ** 2)
    H = a * U
    if not st["case"]["grad"]:
        return H @ Wd.T
    dY = st["dY"].double()
    dH = dY @ Wd
    dG, dU = dH * U * slope, dH * a
    return [H @ Wd.T, dG @ Wg + dU @ Wu, dG.T @ X, dU.T @ X, dY.T @ H]


def exact(case, seed):
    s = prepare(case, seed)
    return dict(norm=_exact_norm, fp8=_exact_linear, ffn=_exact_ffn)[case["op"]](s)
