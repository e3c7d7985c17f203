"""The training operators around the MoE layer -- layer norm, the head's cross entropy over a large
vocabulary, the head's distillation from a teacher's top logits -- as measurable cases.

`run` computes them in plain torch (32 bits, rounded once at the end) or, with `own` set, through the
package's entry points.  `exact` states the definitions once more in 64 bits.
"""
import math

import torch

own = False

BF16, F32 = "bf16", "f32"
_TORCH = {BF16: torch.bfloat16, F32: torch.float32}
_BYTES = {BF16: 2, F32: 4}
EPS = 1e-5
EXACT_FLOPS = 1.2e13      # 64-bit matrix products past this take too long to state the exact result


def _ln(direction, rows, d, x=BF16, w=BF16, **kw):
    return dict(op="layer_norm", direction=direction, rows=rows, d=d, x=x, w=w, **kw)


def _ce(direction, T, d, V, ignored=0.0, **kw):
    return dict(op="cross_entropy", direction=direction, T=T, d=d, V=V, ignored=ignored, **kw)


def _kd(direction, T, d, V, K, temperature=1.0, ragged=0.0, **kw):
    return dict(op="distill", direction=direction, T=T, d=d, V=V, K=K, temperature=temperature, ragged=ragged, **kw)


def listed():
    return [
        # one token through the norm in front of a layer of width 7168: a launch's latency
        _ln("fwd", 1, 7168, name="ln_fwd_1x7168"),
        # a long batch of tokens in front of the layer, 32-bit weights beside 16-bit activations
        _ln("fwd", 16384, 7168, w=F32, name="ln_fwd_16384x7168"),
        # its backward pass at the layer's headline batch
        _ln("bwd", 4096, 7168, w=F32, name="ln_bwd_4096x7168"),
        # 32-bit activations of an odd width, ragged row count
        _ln("bwd", 1531, 1001, x=F32, w=F32, name="ln_bwd_1531x1001_f32"),
        # scoring one token against a vocabulary: the head's weight is read once
        _ce("fwd", 1, 2048, 32768, name="ce_fwd_1_d2048_V32768"),
        # the loss of a training batch, width 7168, large vocabulary
        _ce("fwd", 4096, 7168, 65536, name="ce_fwd_4096_d7168_V65536"),
        # the gradients of that batch at half the vocabulary, some prompt tokens without a loss
        _ce("bwd", 4096, 7168, 32768, ignored=0.1, name="ce_bwd_4096_d7168_V32768"),
        # a small model's step: ragged batch, odd vocabulary, a third of the tokens ignored
        _ce("bwd", 777, 1000, 50001, ignored=0.33, name="ce_bwd_777_d1000_V50001"),
        # a fine-tuning step with few tokens: the weight's gradient is what is written
        _ce("bwd", 64, 2048, 32768, name="ce_bwd_64_d2048_V32768"),
        # a student's loss against a teacher's top 64
        _kd("fwd", 2048, 2048, 65536, 64, temperature=2.0, name="kd_fwd_2048_d2048_V65536_K64"),
        # a student's gradients against a teacher's top 64 at width 7168
        _kd("bwd", 2048, 7168, 32768, 64, temperature=2.0, name="kd_bwd_2048_d7168_V32768_K64"),
        # a ragged small one: odd vocabulary, rows with fewer entries or none
        _kd("bwd", 300, 520, 10007, 20, ragged=0.3, name="kd_bwd_300_d520_V10007_K20"),
    ]


def _log_uniform(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("layer_norm", "cross_entropy", "distill"))
    direction = rng.choice(("fwd", "bwd"))
    if op == "layer_norm":
        rows, d = _log_uniform(rng, 1, 16384), _log_uniform(rng, 64, 8192)
        if rng.random() < 0.7:
            d = max(64, d // 8 * 8)
        x = rng.choice((BF16, BF16, F32))
        return _ln(direction, rows, d, x=x, w=F32 if x == F32 else rng.choice((BF16, F32)))
    most = 4096 * 7168 * 32768
    while True:
        T, V = _log_uniform(rng, 1, 4096), _log_uniform(rng, 1000, 100000)
        d = max(64, _log_uniform(rng, 64, 7168) // 8 * 8)
        if T * d * V <= most:
            break
    if op == "cross_entropy":
        return _ce(direction, T, d, V, ignored=round(rng.choice((0.0, rng.uniform(0.0, 0.6))), 3))
    return _kd(direction, T, d, V, _log_uniform(rng, 1, 128), temperature=rng.choice((1.0, 2.0)),
               ragged=round(rng.choice((0.0, rng.uniform(0.0, 0.4))), 3))


def _generator(seed, device):
    g = torch.Generator(device=device)
    g.manual_seed(int(seed))
    return g


def prepare(case, seed):
    device = "cuda" if torch.cuda.is_available() else "cpu"
    g = _generator(seed, device)

    def randn(*shape):
        return torch.randn(shape, generator=g, device=device)

    s = {"case": case}
    if case["op"] == "layer_norm":
        rows, d, xt, wt = case["rows"], case["d"], _TORCH[case["x"]], _TORCH[case["w"]]
        # a residual stream: unit spread, a mean of its own per token, a few strong channels
        x = randn(rows, d) + 0.5 * randn(rows, 1) + (randn(d) > 2.5) * 4.0 * randn(rows, d)
        s["x"] = x.to(xt)
        s["w"] = (1.0 + 0.1 * randn(d)).to(wt)
        s["b"] = (0.1 * randn(d)).to(wt)
        if case["direction"] == "bwd":
            s["dy"] = randn(rows, d).to(xt)
            x64 = s["x"].double()
            s["mean"] = x64.mean(1).float()
            s["rstd"] = (x64.var(1, unbiased=False) + EPS).rsqrt().float()
        return s
    T, d, V = case["T"], case["d"], case["V"]
    W = torch.empty((V, d), dtype=torch.bfloat16, device=device)
    step = max(1, (1 << 26) // d)
    for i in range(0, V, step):
        W[i:i + step] = randn(min(step, V - i), d) / math.sqrt(d)
    # normalised activations that lean towards the token they are to predict (a part-trained model)
    target = torch.randint(0, V, (T,), generator=g, device=device)
    s["X"] = (randn(T, d) + 3.0 * W[target].float()).to(torch.bfloat16)
    s["W"] = W
    if case["op"] == "cross_entropy":
        drop = torch.rand(T, generator=g, device=device) < case["ignored"]
        drop[0] = False                       # a batch has a token to learn from
        s["labels"] = torch.where(drop, torch.full_like(target, -100), target)
        valid = (~drop).sum().clamp(min=1)
    else:
        K = case["K"]
        ids = torch.randint(0, V, (T, K), generator=g, device=device)
        # distinct entries: an arithmetic walk from a random start with a random stride below V / K
        stride = 1 + ids[:, 1:2] % max(1, V // K - 1) if K > 1 else ids[:, :1] * 0 + 1
        ids = (target[:, None] + stride * torch.arange(K, device=device)[None, :]) % V
        u = torch.sort(2.5 * randn(T, K), dim=1, descending=True).values
        u[:, 0] += 2.0
        keep = torch.full((T, 1), K, device=device)
        if case["ragged"] > 0:
            short = torch.rand((T, 1), generator=g, device=device) < case["ragged"]
            short[0] = False
            keep = torch.where(short, torch.randint(0, K, (T, 1), generator=g, device=device), keep)
        s["ids"] = torch.where(torch.arange(K, device=device)[None, :] < keep, ids, torch.full_like(ids, -1))
        s["u"] = u.contiguous()
        valid = (keep > 0).sum().clamp(min=1)
    if case["direction"] == "bwd":
        s["dloss"] = torch.full((T,), 1.0, device=device) / valid      # the mean over the tokens that count
        s["lse"] = _lse64(s, case)
    return s


def _lse64(s, case):
    """What the forward pass saved: each row's log of the sum of exponentials."""
    X, W, it = s["X"], s["W"], 1.0 / case.get("temperature", 1.0)
    T, V = case["T"], case["V"]
    m = torch.full((T,), -math.inf, device=X.device, dtype=torch.float64)
    step = max(1, (1 << 27) // max(1, T))
    for i in range(0, V, step):
        z = (X.float() @ W[i:i + step].float().T).double() * it
        m = torch.logaddexp(m, torch.logsumexp(z, 1))
    return torch.where(_active(s), m, torch.zeros_like(m)).float()


def _active(s):
    if "labels" in s:
        return s["labels"] >= 0
    return (s["ids"] >= 0).any(1)


# ------------------------------------------------------------------ the plain forms
def _plain_ln_fwd(s):
    x, w, b = s["x"].float(), s["w"].float(), s["b"].float()
    mean = x.mean(1)
    c = x - mean[:, None]
    rstd = 1.0 / torch.sqrt((c * c).mean(1) + EPS)
    y = c * rstd[:, None] * w + b
    return {"y": y.to(s["x"].dtype), "mean": mean, "rstd": rstd}


def _plain_ln_bwd(s):
    x, w, dy = s["x"].float(), s["w"].float(), s["dy"].float()
    n = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gw = dy * w
    dx = s["rstd"][:, None] * (gw - gw.mean(1, keepdim=True) - n * (gw * n).mean(1, keepdim=True))
    return {"dx": dx.to(s["x"].dtype), "dw": (dy * n).sum(0).to(s["w"].dtype), "db": dy.sum(0).to(s["w"].dtype)}


def _plain_targets(s):
    """The target distribution's entries: (ids clamped into the vocabulary, probabilities, 0 where unused)."""
    if "labels" in s:
        ok = (s["labels"] >= 0)[:, None]
        return s["labels"].clamp(min=0)[:, None], ok.float()
    ok = s["ids"] >= 0
    u = torch.where(ok, s["u"] / s["case"]["temperature"], torch.full_like(s["u"], -math.inf))
    top = torch.where(ok.any(1, keepdim=True), u.max(1, keepdim=True).values, torch.zeros_like(u[:, :1]))
    e = torch.exp(u - top)
    return s["ids"].clamp(min=0), e / e.sum(1, keepdim=True).clamp(min=1e-30)


def _plain_head_fwd(s):
    t = s["case"].get("temperature", 1.0)
    z = (s["X"].float() @ s["W"].float().T) / t
    top = z.max(1, keepdim=True).values
    lse = (top + torch.log(torch.exp(z - top).sum(1, keepdim=True)))[:, 0]
    ids, p = _plain_targets(s)
    logp = torch.where(p > 0, torch.log(p.clamp(min=1e-37)), torch.zeros_like(p))
    loss = t * t * (p * (logp - z.gather(1, ids) + lse[:, None])).sum(1)
    on = _active(s)
    zero = torch.zeros_like(lse)
    return {"loss": torch.where(on, loss, zero), "lse": torch.where(on, lse, zero)}


def _plain_head_bwd(s):
    t = s["case"].get("temperature", 1.0)
    X, W = s["X"].float(), s["W"].float()
    D = torch.exp((X @ W.T) / t - s["lse"][:, None])
    ids, p = _plain_targets(s)
    D.scatter_add_(1, ids, -p)
    D *= torch.where(_active(s), s["dloss"] * t, torch.zeros_like(s["dloss"]))[:, None]
    return {"dX": (D @ W).to(torch.bfloat16), "dW": (D.T @ X).to(torch.bfloat16)}


# ------------------------------------------------------------------ the package's
def _own(s):
    from mixture_experts_layer_19_gb300 import train

    case = s["case"]
    op, fwd = case["op"], case["direction"] == "fwd"
    if op == "layer_norm":
        if fwd:
            y, mean, rstd = train.layer_norm_forward(s["x"], s["w"], s["b"], eps=EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        dx, dw, db = train.layer_norm_backward(s["dy"], s["x"], s["w"], s["mean"], s["rstd"])
        return {"dx": dx, "dw": dw, "db": db}
    if op == "cross_entropy":
        if fwd:
            loss, lse = train.cross_entropy_forward(s["X"], s["W"], s["labels"])
            return {"loss": loss, "lse": lse}
        dX, dW = train.cross_entropy_backward(s["dloss"], s["X"], s["W"], s["labels"], s["lse"])
        return {"dX": dX, "dW": dW}
    if fwd:
        loss, lse = train.distill_forward(s["X"], s["W"], s["u"], s["ids"], temperature=case["temperature"])
        return {"loss": loss, "lse": lse}
    dX, dW = train.distill_backward(s["dloss"], s["X"], s["W"], s["u"], s["ids"], s["lse"],
                                    temperature=case["temperature"])
    return {"dX": dX, "dW": dW}


def run(state):
    if own:
        return _own(state)
    fwd = state["case"]["direction"] == "fwd"
    if state["case"]["op"] == "layer_norm":
        return _plain_ln_fwd(state) if fwd else _plain_ln_bwd(state)
    return _plain_head_fwd(state) if fwd else _plain_head_bwd(state)


def work(case):
    fwd = case["direction"] == "fwd"
    if case["op"] == "layer_norm":
        n, d, xb, wb = case["rows"] * case["d"], case["d"], _BYTES[case["x"]], _BYTES[case["w"]]
        if fwd:
            return {"bytes": 2 * n * xb + 2 * d * wb + 8 * case["rows"], "flops": 7 * n}
        return {"bytes": 3 * n * xb + 3 * d * wb + 8 * case["rows"], "flops": 12 * n}
    T, d, V = case["T"], case["d"], case["V"]
    targets = 8 * T if case["op"] == "cross_entropy" else 12 * T * case["K"]
    # tokens without a loss need no products
    live = T * (1.0 - case["ignored"]) if case["op"] == "cross_entropy" else T
    if fwd:
        return {"bytes": 2 * (T + V) * d + targets + 8 * T, "flops": 2 * live * d * V}
    return {"bytes": 4 * (T + V) * d + targets + 8 * T, "flops": 6 * live * d * V}


# ------------------------------------------------------------------ the definitions in 64 bits
def exact(case, seed):
    if case["op"] != "layer_norm":
        cost = (2 if case["direction"] == "fwd" else 6) * case["T"] * case["d"] * case["V"]
        if cost > EXACT_FLOPS:
            return None
    s = prepare(case, seed)
    return _exact_ln(s) if case["op"] == "layer_norm" else _exact_head(s)


def _exact_ln(s):
    x, w = s["x"].double(), s["w"].double()
    d = x.shape[1]
    if "dy" not in s:
        mean = torch.einsum("rd->r", x) / d
        var = torch.einsum("rd,rd->r", x - mean[:, None], x - mean[:, None]) / d
        rstd = torch.pow(var + EPS, -0.5)
        return {"y": torch.addcmul(s["b"].double(), (x - mean[:, None]) * rstd[:, None], w), "mean": mean, "rstd": rstd}
    # the saved statistics are inputs here
    r, dy = s["rstd"].double(), s["dy"].double()
    n = torch.einsum("rd,r->rd", x - s["mean"].double()[:, None], r)
    c1 = torch.einsum("rd,d->r", dy, w) / d
    c2 = torch.einsum("rd,rd,d->r", dy, n, w) / d
    return {"dx": r[:, None] * (torch.einsum("rd,d->rd", dy, w) - c1[:, None] - c2[:, None] * n),
            "dw": torch.einsum("rd,rd->d", dy, n), "db": torch.einsum("rd->d", dy)}


def _exact_head(s):
    """Row block by row block: the target distribution is laid out over the whole vocabulary."""
    case = s["case"]
    T, V, t = case["T"], case["V"], float(case.get("temperature", 1.0))
    X, W = s["X"].double(), s["W"].double()
    fwd = case["direction"] == "fwd"
    loss = torch.zeros(T, dtype=torch.float64, device=X.device)
    lse = torch.zeros_like(loss)
    dX, dW = torch.zeros_like(X), None if fwd else torch.zeros_like(W)
    rows_all = torch.nonzero(_active(s))[:, 0]
    block = max(1, (1 << 27) // V)
    for i in range(0, rows_all.numel(), block):
        rows = rows_all[i:i + block]
        n = rows.numel()
        z = torch.mm(X[rows], W.t()) / t
        P = torch.zeros((n, V), dtype=torch.float64, device=X.device)
        if case["op"] == "cross_entropy":
            P[torch.arange(n, device=X.device), s["labels"][rows]] = 1.0
            entropy = torch.zeros(n, dtype=torch.float64, device=X.device)
        else:
            at, u = s["ids"][rows], s["u"][rows].double() / t
            p = torch.softmax(u.masked_fill(at < 0, -math.inf), dim=1)
            P.scatter_add_(1, at.clamp(min=0), p)
            entropy = -torch.special.xlogy(p, p).sum(1)
        if fwd:
            logq = torch.log_softmax(z, dim=1)
            loss[rows] = t * t * (-entropy - (P * logq).sum(1))
            lse[rows] = torch.logsumexp(z, dim=1)
        else:
            # the saved sums are inputs here
            D = (torch.exp(z - s["lse"][rows].double()[:, None]) - P) * (t * s["dloss"][rows].double())[:, None]
            dX[rows] = torch.mm(D, W)
            dW.addmm_(D.t(), X[rows])
    return {"loss": loss, "lse": lse} if fwd else {"dX": dX, "dW": dW}
