"""Cases and plain forms of the microscaled 4-bit linear layer and of the losses taken at the language-model head.

Three operators and the quantiser that one of them stands on, as a training step of the decoder stack (or its
scoring and decoding) meets them:

quantize  MXFP4: E2M1 elements under one power-of-two scale per 32 of them, along rows or (transposed) along
          columns, with or without the 16-wide Hadamard transform; the values that codes and scales stand for.
linear    Y = Q(X) Q(W)^T on MXFP4 operands; from packed weights (serving) or fp32 masters (training, with
          dX = Q(dY) Q(W^)  and  dW = Q(dY^T) Q(X^),  W^ and X^ the forward's quantised tensors, grouped anew).
ce        Per-token cross entropy of logits X W^T over a large vocabulary, and the gradients of X and W, without
          the logits being returned.
distill   Per-token loss of student logits against a teacher's top logits (temperature, optional hard target),
          and the gradient of the logits.
"""
import math

import torch

own = False
DEV = "cuda"
VOCAB, D, F, TOKENS = 50304, 1024, 4096, 16384  # the 370M-style decoder stack


def listed():
    return [
        # activations of a training batch, grouped along the features for the forward product
        dict(name="quantize rows train", op="quantize", rows=TOKENS, cols=D, dtype="bf16", by="row", rht=False),
        # an output gradient grouped along the tokens for the weight gradient, Hadamard-transformed
        dict(name="quantize cols rht train", op="quantize", rows=TOKENS, cols=F, dtype="bf16", by="col", rht=True),
        # fp32 masters of an odd-sized projection, grouped along the output features
        dict(name="quantize cols f32 ragged", op="quantize", rows=1555, cols=1104, dtype="f32", by="col", rht=False),
        # one token through a gate projection while decoding
        dict(name="linear one token", op="linear", M=1, K=D, N=F, train=False),
        # the head for a batch of sequences that each decode one token
        dict(name="linear head 24 tokens", op="linear", M=24, K=D, N=VOCAB, train=False),
        # a fine-tuning batch of uneven length through a small projection
        dict(name="linear train ragged", op="linear", M=777, K=656, N=1552, train=True),
        # a gate projection of the 370M-style stack in training
        dict(name="linear train 370M", op="linear", M=TOKENS, K=D, N=F, train=True),
        # scoring a short continuation
        dict(name="ce score 5 tokens", op="ce", T=5, K=D, V=VOCAB, grad=False),
        # a small model's step with an odd vocabulary
        dict(name="ce train ragged", op="ce", T=1235, K=528, V=32003, grad=True),
        # the head of the 370M-style stack in training
        dict(name="ce train 370M", op="ce", T=TOKENS, K=D, V=VOCAB, grad=True),
        # fp32 logits of a few positions, odd vocabulary, part hard target
        dict(name="distill f32 ragged", op="distill", T=37, V=32003, k=50, dtype="f32", tau=2.0, alpha=0.5),
        # a distilled training batch of the 370M-style stack
        dict(name="distill train 370M", op="distill", T=TOKENS, V=VOCAB, k=64, dtype="bf16", tau=2.0, alpha=1.0),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def log16(lo, hi):
        return max(16, log(lo, hi) // 16 * 16)

    op = rng.choice(["quantize", "linear", "linear", "ce", "ce", "distill"])
    if op == "quantize":
        return dict(op=op, rows=log(16, TOKENS), cols=log16(64, F), dtype=rng.choice(["bf16", "f32"]),
                    by=rng.choice(["row", "col"]), rht=rng.random() < 0.5)
    if op == "linear":
        if rng.random() < 0.5:
            return dict(op=op, M=log(1, 512), K=log16(128, F), N=log16(128, VOCAB), train=False)
        return dict(op=op, M=log(16, TOKENS), K=log16(128, D), N=log16(128, F), train=True)
    if op == "ce":
        return dict(op=op, T=log(1, TOKENS), K=log16(64, D), V=log(1000, VOCAB), grad=rng.random() < 0.7)
    return dict(op=op, T=log(1, TOKENS), V=log(1000, VOCAB), k=log(1, 128), dtype=rng.choice(["bf16", "bf16", "f32"]),
                tau=rng.choice([1.0, 1.5, 2.0, 4.0]), alpha=rng.choice([0.3, 0.5, 1.0]))


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


def _pack(values, scale):
    """Codes and scale bytes of MXFP4 values [rows, len] under exponents [rows, len/32] in the stored layout: rows
    padded to whole 128 elements, two codes a byte with the first in the low half, one byte 2^(b - 127) per 32."""
    rows, n = values.shape
    nb = -(-n // 128)
    half = scale >> 1
    up = (_pow2(-half) * _pow2(half - scale)).repeat_interleave(32, 1)[:, :n]
    mag = values.abs() * up
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=values.device)
    code = (torch.bucketize(mag, grid) | (torch.signbit(values).long() << 3)).to(torch.uint8)
    full = torch.zeros(rows, nb * 128, dtype=torch.uint8, device=values.device)
    full[:, :n] = code
    sb = torch.zeros(rows, nb * 4, dtype=torch.uint8, device=values.device)
    sb[:, : scale.shape[1]] = (scale + 127).to(torch.uint8)
    return full[:, 0::2] | (full[:, 1::2] << 4), sb


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "quantize":
        x = _normal(g, case["rows"], case["cols"], 0.02 if case["dtype"] == "f32" else 1.0, 0.03)
        x[case["rows"] // 2] = 0.0  # a padding position
        mask = int(torch.randint(0, 1 << 16, (1,), generator=torch.Generator().manual_seed(seed)))
        return dict(case=case, x=x.to(torch.bfloat16) if case["dtype"] == "bf16" else x, mask=mask)
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        s = dict(case=case, X=_normal(g, M, K, 1.0, 0.03).to(torch.bfloat16))
        W = _normal(g, N, K, 0.02)
        if case["train"]:
            return dict(s, W=W, dY=_normal(g, M, N, 1e-3, 0.03).to(torch.bfloat16))
        codes, scales = _pack(*_mx(W, parts=True))
        return dict(s, codes=codes, scales=scales)
    if op == "ce":
        T, K, V = case["T"], case["K"], case["V"]
        W = _normal(g, V, K, 0.02).to(torch.bfloat16)
        y = torch.randint(0, V, (T,), generator=g, device=DEV)
        X = _normal(g, T, K, 1.0)
        Wy = W[y].float()
        X += Wy / Wy.norm(dim=1, keepdim=True) * torch.rand(T, 1, generator=g, device=DEV) * 24.0  # half-learned targets
        y[torch.rand(T, generator=g, device=DEV) < 0.02] = -100  # padding
        dloss = torch.where(y >= 0, 1.0 / max(1, T), 0.0)
        return dict(case=case, X=X.to(torch.bfloat16), W=W, y=y, dloss=dloss)
    T, V, k = case["T"], case["V"], case["k"]
    z = _normal(g, T, V, 2.0)
    start = torch.randint(0, V, (T, 1), generator=g, device=DEV)
    step = torch.randint(1, max(2, V // k), (T, 1), generator=g, device=DEV)
    ids = (start + step * torch.arange(k, device=DEV)) % V
    teacher = 14.0 - torch.rand(T, k, generator=g, device=DEV).cumsum(1) * (16.0 / k)
    z.scatter_(1, ids, teacher + torch.randn(T, k, generator=g, device=DEV))
    kept = torch.randint(1, k + 1, (T, 1), generator=g, device=DEV)  # a top-p teacher keeps fewer of some rows
    drop = (torch.rand(T, 1, generator=g, device=DEV) < 0.25) & (torch.arange(k, device=DEV) >= kept)
    drop |= torch.rand(T, 1, generator=g, device=DEV) < 0.01        # and of some none
    y = ids[:, 0].clone()
    ids = torch.where(drop, torch.full_like(ids, -1), ids)
    y[torch.rand(T, generator=g, device=DEV) < 0.02] = -100
    weight = torch.full((T,), 1.0 / T, device=DEV)
    dt = torch.bfloat16 if case["dtype"] == "bf16" else torch.float32
    return dict(case=case, z=z.to(dt), ids=ids.to(torch.int32), teacher=teacher.to(dt), y=y, weight=weight)


# ---- plain forms: elementary operations in 32 bits -----------------------------------------------------------------
def _pow2(e):
    """2^e as fp32 for whole e in [-126, 127], put together from its bits (exp2 is not exact on every device)."""
    return ((e.to(torch.int32) + 127) << 23).view(torch.float32)


def _round_e2m1(a):
    """|a| <= 6 to the nearest of 0, .5, 1, 1.5, 2, 3, 4, 6, ties to the even code."""
    return torch.where(a <= 2.0, torch.round(a * 2.0) * 0.5, torch.where(a <= 4.0, torch.round(a), torch.round(a * 0.5) * 2.0))


def _mx(x, parts=False):
    """The MXFP4 values of fp32 x [rows, len] in groups of 32 along len: scale 2^(floor(log2(max|group|)) - 2)."""
    rows, n = x.shape
    padded = torch.zeros(rows, -(-n // 32) * 32, dtype=torch.float32, device=x.device)
    padded[:, :n] = x
    gr = padded.view(rows, -1, 32)
    amax = gr.abs().amax(2, keepdim=True)
    e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
    e = torch.where(amax == 0, torch.full_like(e, -127), e)
    half = e >> 1  # in two exact steps: 2^-e alone may leave the range
    q = _round_e2m1((gr.abs() * _pow2(-half) * _pow2(half - e)).clamp(max=6.0))
    v = torch.copysign(q * _pow2(half) * _pow2(e - half), gr).reshape(rows, -1)[:, :n]
    return (v, e.squeeze(2)) if parts else v


def _butterfly(v, h):
    a = v.view(*v.shape[:-1], 16 // (2 * h), 2, h)
    return torch.stack((a[..., 0, :] + a[..., 1, :], a[..., 0, :] - a[..., 1, :]), dim=-2).view(v.shape)


def _rht(x, mask):
    """The 16-wide Hadamard transform along the last axis, positions in `mask` negated first; a last piece of fewer
    than 16 positions stays as it is."""
    n = x.shape[1] // 16 * 16
    sign = 1.0 - 2.0 * ((mask >> torch.arange(16, device=x.device)) & 1).to(torch.float32)
    v = x[:, :n].reshape(x.shape[0], -1, 16) * sign
    v = _butterfly(_butterfly(_butterfly(_butterfly(v, 1), 2), 4), 8) * 0.25
    return torch.cat((v.reshape(x.shape[0], n), x[:, n:]), dim=1)


def _unpack(codes, scales, n):
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), dim=2).reshape(codes.shape[0], -1)[:, :n].long()
    e = scales.to(torch.int32) - 127
    s = (_pow2(e >> 1) * _pow2(e - (e >> 1))).repeat_interleave(32, 1)[:, :n]
    return grid[c] * s


def _plain_quantize(s):
    x = s["x"].float()
    x = x.t().contiguous() if s["case"]["by"] == "col" else x
    x = _rht(x, s["mask"]) if s["case"]["rht"] else x
    return _mx(x).to(torch.bfloat16)


def _plain_linear(s):
    c = s["case"]
    X = _mx(s["X"].float())
    if not c["train"]:
        return (X @ _unpack(s["codes"], s["scales"], c["K"]).t()).to(torch.bfloat16)
    W = _mx(s["W"])
    dY = s["dY"].float()
    dX = _mx(dY) @ _mx(W.t().contiguous()).t()
    dW = _mx(dY.t().contiguous()) @ _mx(X.t().contiguous()).t()
    return (X @ W.t()).to(torch.bfloat16), dX.to(torch.bfloat16), dW


def _plain_ce(s):
    X, W, y = s["X"].float(), s["W"].float(), s["y"]
    z = X @ W.t()
    m = z.amax(1, keepdim=True)
    e = torch.exp(z - m)
    total = e.sum(1, keepdim=True)
    kept = y >= 0
    at = y.clamp(min=0).unsqueeze(1)
    loss = torch.where(kept, (m + torch.log(total) - z.gather(1, at)).squeeze(1), torch.zeros_like(s["dloss"]))
    if not s["case"]["grad"]:
        return loss
    w = torch.where(kept, s["dloss"], torch.zeros_like(s["dloss"])).unsqueeze(1)
    dz = e / total
    dz.scatter_add_(1, at, torch.full_like(m, -1.0))
    dz *= w
    return loss, (dz @ W).to(torch.bfloat16), (dz.t() @ X).to(torch.bfloat16)


def _plain_distill(s):
    tau, alpha = s["case"]["tau"], s["case"]["alpha"]
    z, y = s["z"].float(), s["y"]
    kept = (y >= 0).unsqueeze(1)
    m = z.amax(1, keepdim=True)
    et = torch.exp((z - m) / tau)
    st = et.sum(1, keepdim=True)
    valid = s["ids"] >= 0
    some = valid.any(1, keepdim=True)
    u = torch.where(valid, s["teacher"].float() / tau, torch.full_like(s["teacher"], -math.inf, dtype=torch.float32))
    mu = torch.where(some, u.amax(1, keepdim=True), torch.zeros_like(m))
    eu = torch.exp(u - mu)
    su = torch.where(some, eu.sum(1, keepdim=True), torch.ones_like(m))
    p = eu / su
    at = s["ids"].clamp(min=0).long()
    logp = torch.where(valid, u - mu - torch.log(su), torch.zeros_like(u))
    logq = (z.gather(1, at) - m) / tau - torch.log(st)
    kl = (p * (logp - logq)).sum(1, keepdim=True)
    hard = y.clamp(min=0).unsqueeze(1)
    e1 = torch.exp(z - m)
    s1 = e1.sum(1, keepdim=True)
    ce = m + torch.log(s1) - z.gather(1, hard)
    loss = torch.where(kept, alpha * tau * tau * kl + (1.0 - alpha) * ce, torch.zeros_like(m))
    w = torch.where(kept, s["weight"].unsqueeze(1), torch.zeros_like(m))
    dz = et * (torch.where(some, alpha * tau * w, torch.zeros_like(w)) / st)
    dz.scatter_add_(1, at, -alpha * tau * w * p)
    if alpha != 1.0:
        dz += e1 * ((1.0 - alpha) * w / s1)
        dz.scatter_add_(1, hard, -(1.0 - alpha) * w)
    return loss.squeeze(1), dz.to(s["z"].dtype)


# ---- one pass ------------------------------------------------------------------------------------------------------
def run(s):
    if own:
        return _own(s)
    return dict(quantize=_plain_quantize, linear=_plain_linear, ce=_plain_ce, distill=_plain_distill)[s["case"]["op"]](s)


def _own(s):
    import bit_fully_quantized_amd as tj2

    c = s["case"]
    if c["op"] == "quantize":
        q = tj2.mx_quantize(s["x"], grouping=tj2.GROUP_COL if c["by"] == "col" else tj2.GROUP_ROW, rht=c["rht"],
                            signs=s["mask"] if c["rht"] else 0)
        return tj2.mx_dequantize(q)
    if c["op"] == "linear":
        if not c["train"]:
            Wq = tj2.QTensor.wrap(tj2.MXFP4, c["N"], c["K"], s["codes"], s["scales"])
            return tj2.mx_linear_fwd(s["X"], None, c["N"], Wq=Wq)[0]
        Y, saved = tj2.mx_linear_fwd(s["X"], s["W"], c["N"])
        dX, dW = tj2.mx_linear_bwd(s["dY"], saved, c["K"], seed=0, offset=0, rht=False, rounding=tj2.RTN)
        return Y, dX, dW
    if c["op"] == "ce":
        loss, lse = tj2.linear_ce_fwd(s["X"], s["W"], s["y"])
        if not c["grad"]:
            return loss
        dX, dW = tj2.linear_ce_bwd(s["X"], s["W"], s["y"], lse, s["dloss"])
        return loss, dX, dW
    return tj2.distill_topk(s["z"], s["ids"], s["teacher"], temperature=c["tau"], alpha=c["alpha"], targets=s["y"],
                            weight=s["weight"], grad=True)


def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        return dict(bytes=n * ((2 if case["dtype"] == "bf16" else 4) + 2), flops=4 * n)
    if op == "linear":
        M, K, N = case["M"], case["K"], case["N"]
        if not case["train"]:
            return dict(bytes=2 * M * K + N * K * 17 / 32 + 2 * M * N, flops=2 * M * N * K)
        return dict(bytes=2 * M * K + 4 * N * K + 2 * M * N + 2 * M * N + 2 * M * K + 4 * N * K, flops=6 * M * N * K)
    if op == "ce":
        T, K, V = case["T"], case["K"], case["V"]
        if not case["grad"]:
            return dict(bytes=2 * T * K + 2 * V * K + 12 * T, flops=2 * T * V * K)
        return dict(bytes=4 * T * K + 4 * V * K + 16 * T, flops=6 * T * V * K)
    T, V, k, b = case["T"], case["V"], case["k"], 2 if case["dtype"] == "bf16" else 4
    return dict(bytes=2 * T * V * b + T * k * (4 + b) + 16 * T, flops=8 * T * V)


# ---- the definitions in 64 bits, written apart ---------------------------------------------------------------------
def _exact_mx(x, axis):
    """MXFP4 values of x (64 bits) in groups of 32 along `axis`, by the distance to each grid value."""
    x = x.movedim(axis, -1)
    lead, n = x.shape[:-1], x.shape[-1]
    grid = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=x.device)
    mid = (grid[1:] + grid[:-1]) / 2
    pad = (-n) % 32
    g = torch.nn.functional.pad(x, (0, pad)).reshape(*lead, -1, 32)
    top = g.abs().max(-1, keepdim=True).values
    exponent = torch.where(top > 0, torch.frexp(top).exponent.long() - 3, -127).clamp(min=-127)
    scale = ((exponent + 1023) << 52).view(torch.float64)
    a = (g.abs() / scale).contiguous()
    low, high = torch.bucketize(a, mid, right=False), torch.bucketize(a, mid, right=True)
    index = torch.where(low % 2 == 0, low, high)  # on a border both neighbours are as near: the even code
    v = torch.where(g < 0, -grid[index], grid[index]) * scale
    return v.reshape(*lead, n + pad)[..., :n].movedim(-1, axis)


def _exact_linear(s):
    c = s["case"]
    X = _exact_mx(s["X"].double(), 1)
    if c["train"]:
        W = _exact_mx(s["W"].double(), 1)
        dY = s["dY"].double()
        return [X @ W.T, _exact_mx(dY, 1) @ _exact_mx(W, 0), _exact_mx(dY, 0).T @ _exact_mx(X, 0)]
    e2m1 = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device=DEV)
    b = s["codes"].long()
    nib = torch.empty(b.shape[0], b.shape[1] * 2, dtype=torch.long, device=DEV)
    nib[:, ::2], nib[:, 1::2] = b % 16, b // 16
    W = e2m1[nib % 8] * (1 - 2 * (nib // 8)).double()
    scale = ((s["scales"].long() - 127 + 1023) << 52).view(torch.float64)
    W = (W.view(W.shape[0], -1, 32) * scale.unsqueeze(2)).view(W.shape)
    return X @ W[:, : c["K"]].T


def _exact_hadamard(x, mask):
    h = torch.ones(1, 1, dtype=torch.float64, device=DEV)
    for _ in range(4):
        h = torch.cat((torch.cat((h, h), 1), torch.cat((h, -h), 1)), 0)
    sign = torch.tensor([-1.0 if mask >> j & 1 else 1.0 for j in range(16)], dtype=torch.float64, device=DEV)
    n = x.shape[1] // 16 * 16
    out = x.clone()
    out[:, :n] = ((x[:, :n].reshape(-1, 16) * sign) @ h / 4).reshape(x.shape[0], n)
    return out


def _exact_ce(s):
    X, W, y = s["X"].double(), s["W"].double(), s["y"]
    T, loss, dX, dW = X.shape[0], [], [], torch.zeros_like(W)
    for a in range(0, T, 4096):
        rows, yy = X[a:a + 4096], y[a:a + 4096]
        logp = torch.log_softmax(rows @ W.T, dim=1)
        keep = yy != -100
        pick = torch.where(keep, yy, 0)
        loss.append(torch.where(keep, -logp[torch.arange(len(yy), device=DEV), pick], 0.0))
        if s["case"]["grad"]:
            d = logp.exp_()
            d[torch.arange(len(yy), device=DEV), pick] -= 1
            d *= (s["dloss"][a:a + 4096].double() * keep)[:, None]
            dX.append(d @ W)
            dW += d.T @ rows
    return [torch.cat(loss), torch.cat(dX), dW] if s["case"]["grad"] else torch.cat(loss)


def _exact_distill(s):
    tau, alpha = s["case"]["tau"], s["case"]["alpha"]
    losses, grads = [], []
    for a in range(0, s["z"].shape[0], 4096):
        z, ids, u, y, w = (s[n][a:a + 4096] for n in ("z", "ids", "teacher", "y", "weight"))
        z, u, w, ids = z.double(), u.double(), w.double(), ids.long()
        row = torch.arange(len(y), device=DEV)
        on = y != -100
        has = (ids >= 0).sum(1) > 0
        p = torch.softmax(torch.where(ids >= 0, u / tau, -torch.inf), dim=1)
        p = torch.where((ids >= 0) & has[:, None], p, 0.0)
        logq = torch.log_softmax(z / tau, dim=1)
        kl = (torch.xlogy(p, p) - p * torch.gather(logq, 1, ids.clamp(min=0))).sum(1)
        logs = torch.log_softmax(z, dim=1)
        pick = torch.where(on, y, 0)
        loss = alpha * tau ** 2 * kl - (1 - alpha) * logs[row, pick]
        losses.append(torch.where(on, loss, 0.0))
        d = alpha * tau * (logq.exp_() * has[:, None].double())
        d = d.scatter_add(1, ids.clamp(min=0), -alpha * tau * p)
        h = logs.exp_()
        h[row, pick] -= 1
        grads.append((d + (1 - alpha) * h) * (w * on)[:, None])
    return [torch.cat(losses), torch.cat(grads)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        x = s["x"].double()
        x = x.T if case["by"] == "col" else x
        return _exact_mx(_exact_hadamard(x, s["mask"]) if case["rht"] else x, 1)
    return dict(linear=_exact_linear, ce=_exact_ce, distill=_exact_distill)[case["op"]](s)
