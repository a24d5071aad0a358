"""The two ends of a language model's training step, as cases to be measured.

Muon updates a model's hidden matrices; the embedding table, the output
projection and the norm weights are the parameters beside them.  The cases
here are the operators that produce those parameters' gradients:

* the embedding lookup with scaling and its gradient by sorted tokens;
* layer norm's forward and backward pass with the parameters' gradients;
* the output projection with its softmax cross entropy, the logits never
  kept, and both gradients.

``own`` False computes them in plain torch operations in 32 bits; True calls
the framework's entry points.
"""

import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-5


def listed():
    return [
        # Output projection of a 124M GPT-2 (d_model 768, its own vocabulary,
        # which is odd), one micro-batch of 16 sequences of 1024 tokens.
        {"name": "xent_train_gpt2", "op": "xent_train", "dtype": "bf16", "n": 16384, "d": 768, "v": 50257},
        # Llama-8B width with a vocabulary of 128000: the largest product.
        {"name": "xent_train_llama", "op": "xent_train", "dtype": "bf16", "n": 8192, "d": 4096, "v": 128000},
        # A ragged packed batch in half precision, expert width 1408.
        {"name": "xent_train_ragged", "op": "xent_train", "dtype": "fp16", "n": 1000, "d": 1408, "v": 32003},
        # Log-probability of one sampled token: every weight read for one row.
        {"name": "xent_score_token", "op": "xent_score", "dtype": "bf16", "n": 1, "d": 4096, "v": 128000},
        # Scoring a short text in full precision, sizes off every tile.
        {"name": "xent_score_fp32", "op": "xent_score", "dtype": "fp32", "n": 300, "d": 1000, "v": 8191},
        # Layer norm of a GPT-2 micro-batch, parameters held in fp32.
        {"name": "norm_fwd_gpt2", "op": "norm_fwd", "dtype": "bf16", "n": 16384, "d": 768, "params": "fp32"},
        # Layer norm of one token while serving: launch latency.
        {"name": "norm_fwd_token", "op": "norm_fwd", "dtype": "bf16", "n": 1, "d": 4096, "params": "bf16"},
        # The backward pass at Llama width, all three gradients.
        {"name": "norm_bwd_llama", "op": "norm_bwd", "dtype": "bf16", "n": 8192, "d": 4096, "params": "bf16"},
        # The backward pass in fp32 with an odd width (no row but the first aligned).
        {"name": "norm_bwd_odd", "op": "norm_bwd", "dtype": "fp32", "n": 5003, "d": 1001, "params": "fp32"},
        # Lookup of a long batch, scaled by sqrt(d).
        {"name": "embed_fwd_llama", "op": "embed_fwd", "dtype": "bf16", "n": 32768, "d": 4096, "v": 128000},
        # The table's gradient, GPT-2 micro-batch: most rows get no token.
        {"name": "embed_bwd_gpt2", "op": "embed_bwd", "dtype": "bf16", "n": 16384, "d": 768, "v": 50257},
        # The table's gradient for a long batch: a few tokens fill thousands of positions.
        {"name": "embed_bwd_long", "op": "embed_bwd", "dtype": "bf16", "n": 65536, "d": 2048, "v": 128000},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: half of them a multiple of 64, the others any number."""
    d = _spread(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 0.5 else d


def draw(rng):
    op = rng.choice(["xent_train", "xent_score", "norm_fwd", "norm_bwd", "embed_fwd", "embed_bwd"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    case = {"op": op, "dtype": dtype}
    if op == "xent_train":
        # fp32 products run at a sixteenth of the 16-bit rate: smaller ones.
        top = 2e10 if dtype == "fp32" else 1e12
        case["d"] = _width(rng, 64, 4096)
        case["v"] = _spread(rng, 500, 128000)
        case["n"] = _spread(rng, 32, max(64, min(16384, top / case["d"] / case["v"])))
    elif op == "xent_score":
        case["d"] = _width(rng, 64, 4096)
        case["v"] = _spread(rng, 500, 128000)
        case["n"] = _spread(rng, 1, max(2, min(4096, 5e10 / case["d"] / case["v"])))
    elif op in ("norm_fwd", "norm_bwd"):
        case["d"] = _width(rng, 64, 8192)
        case["n"] = _spread(rng, 1, min(32768, 64e6 / case["d"]))
        case["params"] = rng.choice([dtype, "fp32"])
    else:
        case["d"] = _width(rng, 64, 4096)
        case["v"] = _spread(rng, 500, 128000)
        case["n"] = _spread(rng, 1, min(65536, 128e6 / case["d"]))
    return case


def _zipf(n, v, gen):
    """n token ids in [0, v) with word-like frequencies 1 / (rank + 2.7), the ranks shuffled over the ids."""
    weight = 1.0 / (torch.arange(v, device="cuda", dtype=torch.float64) + 2.7)
    edges = torch.cumsum(weight / weight.sum(), 0)
    u = torch.rand(n, device="cuda", dtype=torch.float64, generator=gen)
    rank = torch.searchsorted(edges, u).clamp_(max=v - 1)
    return torch.randperm(v, device="cuda", generator=gen)[rank]


def _touched(n, v):
    """Expected number of distinct ids among n of them."""
    p = 1.0 / (np.arange(v) + 2.7)
    return float(np.sum(-np.expm1(n * np.log1p(-p / p.sum()))))


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, n, d, op = DTYPES[case["dtype"]], case["n"], case["d"], case["op"]

    def normal(*shape, scale=1.0, to=dtype):
        return torch.randn(*shape, device="cuda", generator=gen).mul_(scale).to(to)

    s = {"op": op}
    if op.startswith("xent"):
        v = case["v"]
        s["w"] = normal(v, d, scale=1.28 / math.sqrt(d))
        s["targets"] = _zipf(n, v, gen)
        # Normed hidden states that lean towards their target's row, as a
        # model's do once it has learnt something.
        s["h"] = (normal(n, d, to=torch.float32) + 4.0 * s["w"][s["targets"]].float()).to(dtype)
        if op == "xent_train":
            # Prompt and padding positions carry no loss; the loss is the mean of the others.
            s["targets"][torch.rand(n, device="cuda", generator=gen) < 0.1] = -100
            valid = s["targets"] >= 0
            s["dloss"] = valid.float() / valid.sum().clamp(min=1)
    elif op.startswith("norm"):
        # A residual stream: unit rows with an offset and a few large channels.
        s["x"] = (normal(n, d, to=torch.float32) * (1.0 + 4.0 * (torch.rand(d, device="cuda", generator=gen) < 0.01))
                  + 0.5).to(dtype)
        to = DTYPES[case["params"]]
        s["weight"] = (1.0 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(to)
        s["bias"] = normal(d, scale=0.1, to=to)
        if op == "norm_bwd":
            s["dy"] = normal(n, d, scale=1e-3 if dtype != torch.float16 else 1e-2)
            x = s["x"].double()
            s["mean"] = x.mean(1).float()
            s["rstd"] = (1.0 / torch.sqrt(x.var(1, unbiased=False) + EPS)).float()
    else:
        v = case["v"]
        s["v"], s["scale"] = v, math.sqrt(d)
        s["ids"] = _zipf(n, v, gen)
        if op == "embed_fwd":
            s["table"] = normal(v, d, scale=0.02)
        else:
            s["dy"] = normal(n, d, scale=1e-3 if dtype != torch.float16 else 1e-2)
    return s


def run(s):
    op = s["op"]
    if own:
        import newton_schulz_matrix_amd as nsa
        if op == "xent_train":
            loss, lse = nsa.linear_cross_entropy(s["h"], s["w"], s["targets"])
            dh, dw = nsa.linear_cross_entropy_backward(s["h"], s["w"], s["targets"], lse, s["dloss"])
            return {"loss": loss, "lse": lse, "dh": dh, "dw": dw}
        if op == "xent_score":
            loss, lse = nsa.linear_cross_entropy(s["h"], s["w"], s["targets"])
            return {"loss": loss, "lse": lse}
        if op == "norm_fwd":
            y, mean, rstd = nsa.layer_norm(s["x"], s["weight"], s["bias"], eps=EPS)
            return {"y": y, "mean": mean, "rstd": rstd}
        if op == "norm_bwd":
            dx, dweight, dbias = nsa.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["weight"])
            return {"dx": dx, "dweight": dweight, "dbias": dbias}
        if op == "embed_fwd":
            return {"out": nsa.embedding(s["ids"], s["table"], scale=s["scale"])}
        return {"dtable": nsa.embedding_backward(s["ids"], s["dy"], s["v"], scale=s["scale"])}
    if op.startswith("xent"):
        h, w, t = s["h"].float(), s["w"].float(), s["targets"]
        z = h @ w.t()
        top = z.amax(1, keepdim=True)
        lse = top[:, 0] + torch.log(torch.exp(z - top).sum(1))
        valid = t >= 0
        at = t.clamp(min=0)[:, None]
        loss = torch.where(valid, lse - z.gather(1, at)[:, 0], torch.zeros_like(lse))
        if op == "xent_score":
            return {"loss": loss, "lse": lse}
        g = torch.where(valid, s["dloss"], torch.zeros_like(lse))[:, None]
        dz = torch.exp(z - lse[:, None]) * g
        dz.scatter_add_(1, at, -g)
        return {"loss": loss, "lse": lse, "dh": (dz @ w).to(s["h"].dtype), "dw": (dz.t() @ h).to(s["w"].dtype)}
    if op == "norm_fwd":
        x = s["x"].float()
        mean = x.mean(1, keepdim=True)
        x = x - mean
        rstd = torch.rsqrt((x * x).mean(1, keepdim=True) + EPS)
        y = x * rstd * s["weight"].float() + s["bias"].float()
        return {"y": y.to(s["x"].dtype), "mean": mean[:, 0], "rstd": rstd[:, 0]}
    if op == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"][:, None]
        xhat = (s["x"].float() - s["mean"][:, None]) * rstd
        wdy = dy * s["weight"].float()
        dx = (wdy - wdy.mean(1, keepdim=True) - xhat * (wdy * xhat).mean(1, keepdim=True)) * rstd
        to = s["weight"].dtype
        return {"dx": dx.to(s["x"].dtype), "dweight": (dy * xhat).sum(0).to(to), "dbias": dy.sum(0).to(to)}
    if op == "embed_fwd":
        return {"out": (s["table"][s["ids"]].float() * s["scale"]).to(s["table"].dtype)}
    dy = s["dy"]
    total = torch.zeros(s["v"], dy.shape[1], device=dy.device, dtype=torch.float32)
    total.index_add_(0, s["ids"], dy.float())
    return {"dtable": (total * s["scale"]).to(dy.dtype)}


def work(case):
    n, d, b, op = case["n"], case["d"], BYTES[case["dtype"]], case["op"]
    if op.startswith("xent"):
        v = case["v"]
        # Hidden states, weights and targets in, loss and log-sum-exp out;
        # training writes both gradients and takes two more products.
        if op == "xent_score":
            return {"bytes": (n + v) * d * b + 16 * n, "flops": 2.0 * n * v * d + 4.0 * n * v}
        return {"bytes": 2 * (n + v) * d * b + 20 * n, "flops": 6.0 * n * v * d + 8.0 * n * v}
    if op == "norm_fwd":
        return {"bytes": 2 * n * d * b + 2 * d * BYTES[case["params"]] + 8 * n, "flops": 8.0 * n * d}
    if op == "norm_bwd":
        return {"bytes": 3 * n * d * b + 3 * d * BYTES[case["params"]] + 8 * n, "flops": 14.0 * n * d}
    v = case["v"]
    if op == "embed_fwd":
        return {"bytes": 8 * n + (n + _touched(n, v)) * d * b, "flops": 1.0 * n * d}
    return {"bytes": 8 * n + (n + v) * d * b, "flops": 1.0 * n * d}


def _exact_xent(s, train):
    """Row blocks through torch's own 64-bit softmax."""
    h, w, t = s["h"].double(), s["w"].double(), s["targets"]
    n, step = h.shape[0], max(1, (1 << 27) // w.shape[0])
    loss, lse, dh, dw = [], [], [], torch.zeros_like(w) if train else None
    for i in range(0, n, step):
        z = h[i:i + step] @ w.t().contiguous()
        ti = t[i:i + step]
        logp = torch.log_softmax(z, 1)
        lse.append(torch.logsumexp(z, 1))
        rows = torch.nonzero(ti >= 0)[:, 0]
        li = torch.zeros_like(lse[-1])
        li[rows] = -logp[rows, ti[rows]]
        loss.append(li)
        if train:
            p = logp.exp_()
            p[rows, ti[rows]] -= 1.0
            weight = torch.zeros_like(li)
            weight[rows] = s["dloss"][i:i + step].double()[rows]
            p *= weight[:, None]
            dh.append(p @ w)
            dw += p.t().contiguous() @ h[i:i + step]
    out = {"loss": torch.cat(loss), "lse": torch.cat(lse)}
    if train:
        out.update(dh=torch.cat(dh), dw=dw)
    return out


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op.startswith("xent"):
        return _exact_xent(s, op == "xent_train")
    if op == "norm_fwd":
        x = s["x"].double()
        var, mean = torch.var_mean(x, 1, unbiased=False)
        rstd = 1.0 / (var + EPS).sqrt()
        y = torch.addcmul(s["bias"].double(), (x - mean[:, None]) / (var + EPS).sqrt()[:, None], s["weight"].double())
        return {"y": y, "mean": mean, "rstd": rstd}
    if op == "norm_bwd":
        # dx as the projection of w * dy off the ones and off xhat, per row.
        dy, d = s["dy"].double(), s["dy"].shape[1]
        rstd = s["rstd"].double()
        xhat = (s["x"].double() - s["mean"].double()[:, None]).mul_(rstd[:, None])
        a = dy * s["weight"].double()
        c2 = torch.linalg.vecdot(a, xhat) / d
        dx = (a - a.mean(1)[:, None] - c2[:, None] * xhat) * rstd[:, None]
        return {"dx": dx, "dweight": torch.mul(dy, xhat).sum(0), "dbias": dy.sum(0)}
    if op == "embed_fwd":
        return {"out": torch.nn.functional.embedding(s["ids"], s["table"]).double() * s["scale"]}
    total = torch.zeros(s["v"], s["dy"].shape[1], device="cuda", dtype=torch.float64)
    total.index_put_((s["ids"],), s["dy"].double() * s["scale"], accumulate=True)
    return {"dtable": total}
