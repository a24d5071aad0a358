"""A transformer block's feed-forward half and the optimizer beside Muon, as cases to be measured.

Muon updates a block's matrices; the cases here are what the training step
needs around them:

* the gated feed-forward block (gate and up projections, activation, product,
  down projection), forward and with all gradients, and for a few tokens;
* the norms before and after a block with its gate and the scaled residual,
  forward and with all gradients;
* an AdamW step over the tensors that Muon leaves out, in one call, with
  states in 32 bits or in 8.

``own`` False computes them in plain torch operations in 32 bits; True calls
the framework's entry points.
"""

import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
EPS = 1e-6
LR, BETAS, ADAM_EPS, DECAY, STEP = 6e-4, (0.9, 0.95), 1e-8, 0.1, 1000
BLOCK = 256  # elements of an 8-bit state that share a scale
TOP = 448.0  # the largest e4m3 number


def listed():
    return [
        # Feed-forward block of an 8B Llama on one micro-batch: the largest products.
        {"name": "mlp_train_llama", "op": "mlp_train", "dtype": "bf16", "act": "silu", "n": 8192, "d": 4096, "f": 14336},
        # The tokens that one expert (2048 x 1408) got in half precision: a
        # ragged batch, and an odd intermediate width.
        {"name": "mlp_train_ragged", "op": "mlp_train", "dtype": "fp16", "act": "gelu_tanh", "n": 1003, "d": 2048, "f": 1407},
        # A small model in full precision, sizes off every tile.
        {"name": "mlp_train_fp32", "op": "mlp_train", "dtype": "fp32", "act": "gelu", "n": 300, "d": 1000, "f": 2731},
        # One token: every weight read for one row.
        {"name": "mlp_token", "op": "mlp_infer", "dtype": "bf16", "act": "silu", "n": 1, "d": 4096, "f": 14336},
        # One token for each of 48 sequences.
        {"name": "mlp_tokens", "op": "mlp_infer", "dtype": "bf16", "act": "silu", "n": 48, "d": 4096, "f": 14336},
        # Between two blocks of an 8B Llama with norms on both sides and a layer scale.
        {"name": "norm_fwd_llama", "op": "norm_fwd", "dtype": "bf16", "params": "bf16", "n": 8192, "d": 4096, "groups": 1},
        # One token while serving: launch latency.
        {"name": "norm_fwd_token", "op": "norm_fwd", "dtype": "bf16", "params": "bf16", "n": 1, "d": 4096, "groups": 1},
        # The backward pass of a 124M GPT-2's micro-batch of 16 sequences, a gate for each sequence.
        {"name": "norm_bwd_gpt2", "op": "norm_bwd", "dtype": "bf16", "params": "fp32", "n": 16384, "d": 768, "groups": 16},
        # The backward pass in fp32 with an odd width and a gate for each token.
        {"name": "norm_bwd_odd", "op": "norm_bwd", "dtype": "fp32", "params": "fp32", "n": 5003, "d": 1001, "groups": 5003},
        # What Muon leaves out of a 124M GPT-2: fp32 tied embedding and norm
        # vectors, bf16 gradients, the model's bf16 embedding written beside.
        {"name": "adamw_gpt2", "op": "adamw", "bits": 32, "dtype": "fp32", "grads": "bf16", "tables": 1, "rows": 50257, "d": 768, "vectors": 50},
        # The untied output projection and the norms at Llama-8B width, states in 8 bits.
        {"name": "adamw8_llama", "op": "adamw", "bits": 8, "dtype": "bf16", "grads": "bf16", "tables": 1, "rows": 128000, "d": 4096, "vectors": 65},
        # Norm vectors alone: many tiny tensors, launch latency.
        {"name": "adamw_vectors", "op": "adamw", "bits": 32, "dtype": "fp32", "grads": "fp32", "tables": 0, "rows": 0, "d": 768, "vectors": 50},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    """A row width: half of them a multiple of 64, the others any number."""
    d = _spread(rng, lo, hi)
    return max(64, d // 64 * 64) if rng.random() < 0.5 else d


def draw(rng):
    op = rng.choice(["mlp_train", "mlp_train", "mlp_infer", "norm_fwd", "norm_bwd", "adamw"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    case = {"op": op, "dtype": dtype}
    if op.startswith("mlp"):
        case["act"] = rng.choice(["silu", "gelu", "gelu_tanh", "relu"])
        case["d"] = _width(rng, 64, 4096)
        case["f"] = _width(rng, 64, 14336)
        # fp32 products run at a sixteenth of the 16-bit rate: smaller ones.
        most = (2e10 if dtype == "fp32" else 4e11) / case["d"] / case["f"]
        if op == "mlp_train":
            case["n"] = _spread(rng, 32, max(64, min(8192, most)))
        else:
            case["n"] = _spread(rng, 1, max(2, min(512, most)))
    elif op.startswith("norm"):
        case["d"] = _width(rng, 64, 8192)
        case["n"] = _spread(rng, 1, min(32768, 64e6 / case["d"]))
        case["params"] = rng.choice([dtype, "fp32"])
        case["groups"] = rng.choice([1, 1, case["n"], math.gcd(case["n"], 240)])
    else:
        case["bits"] = rng.choice([8, 32])
        case["grads"] = rng.choice([dtype, "bf16"])
        case["d"] = _width(rng, 64, 4096)
        case["tables"] = rng.choice([0, 1, 2])
        case["rows"] = _spread(rng, 500, min(128000, 2e8 / case["d"])) if case["tables"] else 0
        case["vectors"] = _spread(rng, 1, 128)
    return case


def _shapes(case):
    return [(case["rows"], case["d"])] * case["tables"] + [(case["d"],)] * case["vectors"]


def _encode(x, up):
    """An 8-bit state: e4m3 codes in units of the largest magnitude of each block / 448, and those largest magnitudes.

    ``up``: positive numbers below the smallest code take it (a root of the
    second moment that became 0 would make the next update too large)."""
    flat = x.reshape(-1)
    blocks = -(-flat.numel() // BLOCK)
    padded = torch.nn.functional.pad(flat, (0, blocks * BLOCK - flat.numel())).view(blocks, BLOCK)
    top = padded.abs().amax(1).clamp(min=2.0 ** -100)
    q = padded * (TOP / top)[:, None]
    if up:
        q = torch.where((q > 0) & (q < 2.0 ** -9), torch.full_like(q, 2.0 ** -9), q)
    return q.to(torch.float8_e4m3fn).view(-1)[:flat.numel()].view(x.shape), top


def _decode(code, top, to=torch.float32):
    """What an 8-bit state stands for."""
    unit = (top.to(to) / TOP).repeat_interleave(BLOCK)[:code.numel()]
    return code.to(to) * unit.view(code.shape)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    dtype = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0, to=dtype):
        return torch.randn(*shape, device="cuda", generator=gen).mul_(scale).to(to)

    s = {"op": op}
    if op.startswith("mlp"):
        n, d, f = case["n"], case["d"], case["f"]
        s["act"] = case["act"]
        # Normed hidden states and weights that keep the variance.
        s["x"] = normal(n, d)
        s["wg"] = normal(f, d, scale=1 / math.sqrt(d))
        s["wu"] = normal(f, d, scale=1 / math.sqrt(d))
        s["wd"] = normal(d, f, scale=1 / math.sqrt(f))
        if op == "mlp_train":
            s["dy"] = normal(n, d, scale=1e-2)
    elif op.startswith("norm"):
        n, d = case["n"], case["d"]
        to = DTYPES[case["params"]]
        # A residual stream with a few large channels, a branch of another
        # size, gates around a half.
        s["residual"] = (normal(n, d, to=torch.float32)
                         * (1.0 + 4.0 * (torch.rand(d, device="cuda", generator=gen) < 0.01))).to(dtype)
        s["branch"] = normal(n, d, scale=3.0)
        s["gate"] = (0.5 + 0.2 * torch.randn(case["groups"], d, device="cuda", generator=gen)).to(to)
        s["wb"] = (1.0 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(to)
        s["w"] = (1.0 + 0.1 * torch.randn(d, device="cuda", generator=gen)).to(to)
        s["scale"] = 0.9
        if op == "norm_bwd":
            # What the forward pass left.
            b = s["branch"].double()
            rb = (b.square().mean(1) + EPS).rsqrt()
            gate = s["gate"].double().repeat_interleave(n // case["groups"], 0)
            t = s["scale"] * s["residual"].double() + gate * (b * rb[:, None] * s["wb"].double())
            s["stream"] = t.to(dtype)
            s["rb"], s["rs"] = rb.float(), (t.square().mean(1) + EPS).rsqrt().float()
            del s["residual"]
            s["dstream"] = normal(n, d, scale=1e-2)
            s["dy"] = normal(n, d, scale=1e-2)
    else:
        keys = ["p", "g", "m", "v"]
        if case["bits"] == 8:
            keys.append("scales")
        # Masters in fp32 beside 16-bit gradients: the model's own 16-bit tables are written too.
        copies = case["dtype"] == "fp32" and case["grads"] != "fp32"
        if copies:
            keys.append("copies")
        s["lists"] = {k: [] for k in keys}
        s["buffers"] = {k: [] for k in keys}
        s["lr"], s["decay"] = [], []

        def moments(m, v):
            if case["bits"] == 32:
                return {"m": m, "v": v}
            (mc, mt), (vc, vt) = _encode(m, False), _encode(v.sqrt_(), True)
            return {"m": mc, "v": vc, "scales": torch.stack([mt, vt])}

        def add(count, shape, pt, gt, scale, mean, decay):
            """``count`` tensors of a shape, each kind of them behind one another in one buffer."""
            # Gradients whose size differs from column to column; moments as
            # after many steps of such gradients.
            size = 1e-3 * torch.exp(torch.randn(shape[-1], device="cuda", generator=gen))
            kinds = [moments(0.23 * normal(*shape, to=torch.float32) * size,
                             (0.7 + 0.3 * torch.rand(*shape, device="cuda", generator=gen)) * size * size)
                     for _ in range(count)]
            buffers = {k: torch.stack([kind[k] for kind in kinds]) if count > 1 else kinds[0][k][None]
                       for k in kinds[0]}
            buffers["p"] = (mean + normal(count, *shape, scale=scale, to=torch.float32)).to(pt)
            buffers["g"] = (normal(count, *shape, to=torch.float32) * size).to(gt)
            if copies:
                buffers["copies"] = torch.zeros(count, *shape, device="cuda", dtype=gt) if len(shape) > 1 else None
            for k, buffer in buffers.items():
                s["lists"][k] += [None] * count if buffer is None else list(buffer.unbind(0))
                if buffer is not None:
                    s["buffers"][k].append(buffer)
            s["lr"] += [LR] * count
            s["decay"] += [decay] * count

        for _ in range(case["tables"]):
            add(1, (case["rows"], case["d"]), dtype, DTYPES[case["grads"]], 0.02, 0.0, DECAY)
        if case["vectors"]:
            add(case["vectors"], (case["d"],), torch.float32, torch.float32, 0.1, 1.0, 0.0)
        # The coefficient that clips the gradients' norm, made on the device.
        s["clip"] = 0.5 + 0.5 * torch.rand(1, device="cuda", generator=gen)
    return s


def _act(a, name):
    """The activation and its derivative."""
    if name == "silu":
        sig = 1 / (1 + torch.exp(-a))
        return a * sig, sig * (1 + a * (1 - sig))
    if name == "relu":
        return a.clamp(min=0), (a > 0).to(a.dtype)
    if name == "gelu":
        phi = 0.5 * (1 + torch.erf(a * math.sqrt(0.5)))
        return a * phi, phi + a * torch.exp(-0.5 * a * a) * (1 / math.sqrt(2 * math.pi))
    c, k = math.sqrt(2 / math.pi), 0.044715
    t = torch.tanh(c * (a + k * a * a * a))
    return 0.5 * a * (1 + t), 0.5 * (1 + t) + 0.5 * a * (1 - t * t) * c * (1 + 3 * k * a * a)


def _run_own(s):
    import newton_schulz_matrix_amd as nsa
    op = s["op"]
    if op == "mlp_infer":
        return {"y": nsa.gated_mlp(s["x"], s["wg"], s["wu"], s["wd"], activation=s["act"], save=False)[0]}
    if op == "mlp_train":
        y, a, b = nsa.gated_mlp(s["x"], s["wg"], s["wu"], s["wd"], activation=s["act"])
        dx, dwg, dwu, dwd = nsa.gated_mlp_backward(s["dy"], s["x"], s["wg"], s["wu"], s["wd"], a, b,
                                                   activation=s["act"])
        return {"y": y, "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}
    if op == "norm_fwd":
        stream, y, rb, rs = nsa.residual_norm(s["residual"], s["branch"], gate=s["gate"], scale=s["scale"],
                                              branch_weight=s["wb"], weight=s["w"], eps=EPS)
        return {"stream": stream, "y": y, "rb": rb, "rs": rs}
    if op == "norm_bwd":
        dres, dbranch, dgate, dwb, dw = nsa.residual_norm_backward(
            s["dstream"], s["dy"], s["stream"], s["branch"], s["rb"], s["rs"], gate=s["gate"], scale=s["scale"],
            branch_weight=s["wb"], weight=s["w"])
        return {"dresidual": dres, "dbranch": dbranch, "dgate": dgate, "dwb": dwb, "dw": dw}
    t = s["lists"]
    nsa.adamw_step(t["p"], t["g"], t["m"], t["v"], lr=s["lr"], step=STEP, betas=BETAS, eps=ADAM_EPS,
                   weight_decay=s["decay"], scales=t.get("scales"), copies=t.get("copies"), grad_scale=s["clip"])
    return _adamw_outputs(s)


def _adamw_outputs(s):
    """The updated buffers: 8-bit moments as e4m3 numbers beside their scales."""
    return {k: list(s["buffers"][k]) for k in s["buffers"] if k != "g"}


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op.startswith("mlp"):
        x, wg, wu, wd = s["x"].float(), s["wg"].float(), s["wu"].float(), s["wd"].float()
        a, b = x @ wg.t(), x @ wu.t()
        act, slope = _act(a, s["act"])
        h = act * b
        to = s["x"].dtype
        out = {"y": (h @ wd.t()).to(to)}
        if op == "mlp_train":
            dy = s["dy"].float()
            dh = dy @ wd
            da, db = dh * b * slope, dh * act
            out.update(dx=(da @ wg + db @ wu).to(to), dwg=(da.t() @ x).to(to), dwu=(db.t() @ x).to(to),
                       dwd=(dy.t() @ h).to(to))
        return out
    if op.startswith("norm"):
        b, wb, w, groups = s["branch"].float(), s["wb"].float(), s["w"].float(), s["gate"].shape[0]
        gate = s["gate"].float()[:, None]  # groups x 1 x columns, broadcast over a group's rows
        n, d = b.shape
        if op == "norm_fwd":
            rb = torch.rsqrt((b * b).mean(1, keepdim=True) + EPS)
            nb = b * rb * wb
            t = s["scale"] * s["residual"].float() + (gate * nb.view(groups, -1, d)).view(n, d)
            rs = torch.rsqrt((t * t).mean(1, keepdim=True) + EPS)
            to = s["branch"].dtype
            return {"stream": t.to(to), "y": (t * rs * w).to(to), "rb": rb[:, 0], "rs": rs[:, 0]}
        rb, rs, dy = s["rb"][:, None], s["rs"][:, None], s["dy"].float()
        shat, bhat = s["stream"].float() * rs, b * rb
        wdy = w * dy
        g = s["dstream"].float() + rs * (wdy - shat * (wdy * shat).mean(1, keepdim=True))
        dn = (gate * g.view(groups, -1, d)).view(n, d)
        wdn = wb * dn
        dbranch = rb * (wdn - bhat * (wdn * bhat).mean(1, keepdim=True))
        to, pt = s["branch"].dtype, s["w"].dtype
        return {"dresidual": (s["scale"] * g).to(to), "dbranch": dbranch.to(to),
                "dgate": (g * (bhat * wb)).view(groups, -1, d).sum(1).to(pt),
                "dwb": (dn * bhat).sum(0).to(pt), "dw": (dy * shat).sum(0).to(pt)}
    lists = s["lists"]
    for i, p in enumerate(lists["p"]):
        g = lists["g"][i].float() * s["clip"]
        m, v = lists["m"][i], lists["v"][i]
        at = lists["scales"][i] if "scales" in lists else None
        copy = lists["copies"][i] if "copies" in lists else None
        if at is not None:
            m, v = _decode(m, at[0]), _decode(v, at[1]).square()
        m = BETAS[0] * m + (1 - BETAS[0]) * g
        v = BETAS[1] * v + (1 - BETAS[1]) * g * g
        root = torch.sqrt(v)
        x = p.float()
        update = m / (1 - BETAS[0] ** STEP) / (root * (1 / math.sqrt(1 - BETAS[1] ** STEP)) + ADAM_EPS)
        x = x - s["lr"][i] * s["decay"][i] * x - s["lr"][i] * update
        p.copy_(x.to(p.dtype))
        if at is None:
            lists["m"][i].copy_(m)
            lists["v"][i].copy_(v)
        else:
            (mc, mt), (vc, vt) = _encode(m, False), _encode(root, True)
            lists["m"][i].copy_(mc)
            lists["v"][i].copy_(vc)
            at.copy_(torch.stack([mt, vt]))
        if copy is not None:
            copy.copy_(x.to(copy.dtype))
    return _adamw_outputs(s)


def work(case):
    op = case["op"]
    b = BYTES[case["dtype"]]
    if op.startswith("mlp"):
        n, d, f = case["n"], case["d"], case["f"]
        if op == "mlp_infer":
            return {"bytes": (3 * d * f + 2 * n * d) * b, "flops": 6.0 * n * d * f + 8.0 * n * f}
        # Inputs, dy and weights in; y, dx and the weights' gradients out.
        return {"bytes": (6 * d * f + 4 * n * d) * b, "flops": 18.0 * n * d * f + 24.0 * n * f}
    if op.startswith("norm"):
        n, d, g, pb = case["n"], case["d"], case["groups"], BYTES[case["params"]]
        if op == "norm_fwd":
            return {"bytes": 4 * n * d * b + (g + 2) * d * pb + 8 * n, "flops": 10.0 * n * d}
        return {"bytes": 6 * n * d * b + 2 * (g + 2) * d * pb + 8 * n, "flops": 28.0 * n * d}
    count, total = 0, 0.0
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    for shape in _shapes(case):
        k = math.prod(shape)
        vector = len(shape) == 1
        pb, gb = (4, 4) if vector else (b, BYTES[case["grads"]])
        copy = gb if not vector and case["dtype"] == "fp32" and case["grads"] != "fp32" else 0
        total += k * (2 * pb + gb + state + copy)
        count += k
    return {"bytes": total, "flops": 16.0 * count}


def exact(case, seed):
    s = prepare(case, seed)
    op = s["op"]
    if op.startswith("mlp"):
        # The gradients by differentiating the definition in 64 bits.
        train = op == "mlp_train"
        x, wg, wu, wd = (s[k].double().requires_grad_(train) for k in ("x", "wg", "wu", "wd"))
        a = torch.nn.functional.linear(x, wg)
        act = {"silu": torch.nn.functional.silu, "relu": torch.relu, "gelu": torch.nn.functional.gelu,
               "gelu_tanh": lambda t: torch.nn.functional.gelu(t, approximate="tanh")}[s["act"]]
        y = torch.nn.functional.linear(act(a) * torch.nn.functional.linear(x, wu), wd)
        if not train:
            return {"y": y}
        dx, dwg, dwu, dwd = torch.autograd.grad(y, (x, wg, wu, wd), s["dy"].double())
        return {"y": y.detach(), "dx": dx, "dwg": dwg, "dwu": dwu, "dwd": dwd}
    if op.startswith("norm"):
        b, gate, wb, w = (s[k].double() for k in ("branch", "gate", "wb", "w"))
        n, d = b.shape
        rows = torch.arange(n, device=b.device) // (n // gate.shape[0])
        if op == "norm_fwd":
            rb = (torch.linalg.vecdot(b, b) / d + EPS).sqrt().reciprocal()
            t = torch.addcmul(s["scale"] * s["residual"].double(), gate[rows], torch.einsum("ij,i,j->ij", b, rb, wb))
            rs = (torch.linalg.vecdot(t, t) / d + EPS).sqrt().reciprocal()
            return {"stream": t, "y": torch.einsum("ij,i,j->ij", t, rs, w), "rb": rb, "rs": rs}
        # Projections off the normed rows.
        rb, rs, dy = s["rb"].double(), s["rs"].double(), s["dy"].double()
        shat, bhat = s["stream"].double().mul(rs[:, None]), b.mul(rb[:, None])
        u = dy * w
        g = s["dstream"].double() + rs[:, None] * (u - (torch.linalg.vecdot(u, shat) / d)[:, None] * shat)
        q = g * gate[rows] * wb
        dbranch = rb[:, None] * (q - (torch.linalg.vecdot(q, bhat) / d)[:, None] * bhat)
        dgate = torch.zeros_like(gate).index_add_(0, rows, g * bhat * wb)
        return {"dresidual": s["scale"] * g, "dbranch": dbranch, "dgate": dgate,
                "dwb": (g * gate[rows] * bhat).sum(0), "dw": (dy * shat).sum(0)}
    out = {k: [] for k in s["buffers"] if k != "g"}
    lists, first = s["lists"], 0
    for k, buffer in enumerate(s["buffers"]["p"]):
        i = first
        first += buffer.shape[0]
        g = s["buffers"]["g"][k].double().mul_(s["clip"].double())
        if "scales" not in lists:
            m, v = s["buffers"]["m"][k].double(), s["buffers"]["v"][k].double()
        else:
            tops = s["buffers"]["scales"][k]
            m, v = (torch.stack([_decode(c, t[j], torch.float64) for c, t in zip(s["buffers"][name][k], tops)])
                    for j, name in enumerate(("m", "v")))
            v.square_()
        m.lerp_(g, 1 - BETAS[0])
        v.lerp_(g.square_(), 1 - BETAS[1])
        update = (v / (1 - BETAS[1] ** STEP)).sqrt_().add_(ADAM_EPS).reciprocal_().mul_(m).div_(1 - BETAS[0] ** STEP)
        x = buffer.double().mul_(1 - s["lr"][i] * s["decay"][i]).sub_(update, alpha=s["lr"][i])
        out["p"].append(x)
        if "copies" in lists and lists["copies"][i] is not None:
            out["copies"].append(x)
        if "scales" not in lists:
            out["m"].append(m)
            out["v"].append(v)
        else:
            # The codes have no value in 64 bits; their scales do.
            blocks = s["buffers"]["scales"][k].shape[-1]

            def tops_of(t):
                flat = t.abs().view(t.shape[0], -1)
                return torch.nn.functional.pad(flat, (0, blocks * BLOCK - flat.shape[1])).view(-1, blocks, BLOCK).amax(2)

            out["scales"].append(torch.stack([tops_of(m), tops_of(v).sqrt()], 1).clamp_(min=2.0 ** -100))
            out["m"].append(None)
            out["v"].append(None)
    return out
