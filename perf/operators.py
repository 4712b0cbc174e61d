"""Operators around the routed experts: MXFP4 quantisation and grouped products, the block's norms, the router's balance loss.

Each case is one call (or one training step) that a user of the layer makes next to `moe_forward`.  `run` computes it in elementary
torch operations, or, where `own` is set, through the framework's operators.
"""
import math

import torch

own = False

H, I, E, K = 7168, 2048, 256, 8  # the layer of this repository's decode, batched and prefill workloads

TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------------------------------------------ the cases
def listed():
    return [
        # one decoded token's activations, quantised before its experts' products: latency alone
        dict(name="quantize 1x7168 bf16", op="quantize", rows=1, cols=H, type="bf16"),
        # one expert's down projection brought to MXFP4 from its fp32 master copy
        dict(name="quantize 7168x2048 fp32", op="quantize", rows=H, cols=I, type="fp32"),
        # decode of one token: gate and up of its 8 experts with SwiGLU, from bf16 activations
        dict(name="gate/up 1 token", op="product", tokens=1, groups=E, top_k=K, zipf=0.0, cols=H, rows=2 * I, swiglu=True, out="bf16"),
        # batched decode, uneven experts: the down projection, in fp32 for the combine that adds the experts up
        dict(name="down 64 tokens", op="product", tokens=64, groups=E, top_k=K, zipf=1.1, cols=I, rows=H, swiglu=False, out="fp32"),
        # a prefill chunk through gate and up of all experts
        dict(name="gate/up 4096 tokens", op="product", tokens=4096, groups=E, top_k=K, zipf=0.8, cols=H, rows=2 * I, swiglu=True, out="bf16"),
        # the always-on shared expert over a prefill chunk: one dense product, every token in it
        dict(name="shared down 4096 tokens", op="product", tokens=4096, groups=1, top_k=1, zipf=0.0, cols=I, rows=H, swiglu=False, out="bf16"),
        # decode: the experts' output normed, gated and added to the stream, the next block's input normed, for one token
        dict(name="norm 1x7168 bf16", op="norm", rows=1, cols=H, type="bf16", weights="bf16", gate="token", step=False),
        # the same over a training chunk, forward and backward
        dict(name="norm step 4096x7168 bf16", op="norm", rows=4096, cols=H, type="bf16", weights="fp32", gate="feature", step=True),
        # an odd width and odd row count in fp32 with a gate for every value, forward and backward
        dict(name="norm step 777x1003 fp32", op="norm", rows=777, cols=1003, type="fp32", weights="fp32", gate="full", step=True),
        # counts and balance loss of one batched decode step (the popularity that a cache of experts follows)
        dict(name="balance 64x256", op="balance", tokens=64, seqs=1, groups=E, top_k=K, sigmoid=True, masked=0.0, step=False),
        # the router's loss over a training chunk, with its gradient
        dict(name="balance step 4096x256", op="balance", tokens=4096, seqs=1, groups=E, top_k=K, sigmoid=False, masked=0.0, step=True),
        # long packed sequences of different lengths, a loss for each, padding tokens masked out
        dict(name="balance step 65521x256", op="balance", tokens=65521, seqs=37, groups=E, top_k=K, sigmoid=True, masked=0.07, step=True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["quantize", "product", "product", "norm", "norm", "balance"])
    if op == "quantize":
        cols = _log(rng, 33, 16384)
        return dict(op=op, rows=_log(rng, 1, min(16384, H * I // cols)), cols=cols, type=rng.choice(sorted(TYPES)))
    if op == "product":
        groups, cols, swiglu = _log(rng, 1, E), _log(rng, 32, H), rng.random() < 0.5
        rows = 2 * _log(rng, 32, H // 2)
        top_k = min(groups, rng.choice([1, 2, 4, 6, 8]))
        tokens = _log(rng, 1, 4096)
        while groups * cols * rows > E * I * H // 4:
            groups = max(top_k, groups // 2)
            cols = max(32, cols * 3 // 4)
        return dict(op=op, tokens=tokens, groups=groups, top_k=top_k, zipf=rng.choice([0.0, 0.8, 1.1]), cols=cols, rows=rows, swiglu=swiglu,
                    out=rng.choice(["bf16", "fp32"]))
    if op == "norm":
        cols = _log(rng, 17, 16384)
        typ = rng.choice(sorted(TYPES))
        return dict(op=op, rows=_log(rng, 1, min(16384, 4096 * H // cols)), cols=cols, type=typ, weights=rng.choice([typ, "fp32"]),
                    gate=rng.choice(["none", "token", "feature", "full"]), step=rng.random() < 0.6)
    groups, tokens = _log(rng, 4, 1024), _log(rng, 1, 65536)
    tokens = min(tokens, 65521 * E // groups)
    return dict(op=op, tokens=tokens, seqs=rng.randint(1, max(1, min(64, tokens))), groups=groups, top_k=min(groups, rng.choice([1, 2, 6, 8])),
                sigmoid=rng.random() < 0.5, masked=rng.choice([0.0, 0.1]), step=rng.random() < 0.7)


# ------------------------------------------------------------------------------------------------ inputs
def _normal(shape, g, type="fp32", scale=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(TYPES[type])


def _routing(tokens, groups, top_k, zipf, g):
    """Logits with a Zipf popularity, and each token's experts."""
    rank = torch.randperm(groups, generator=g, device="cuda") + 1
    logits = torch.randn((tokens, groups), generator=g, device="cuda") - zipf * torch.log(rank.float())
    return logits, torch.topk(logits, top_k, dim=1).indices.to(torch.int32)


def prepare(case, seed):
    """Activations, weights and routing.  A program keeps its MXFP4 weights laid out for the calls that it makes: the framework's
    operators take their own image of the codes and scales that the plain form reads."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case=case)
    if case["op"] == "quantize":
        s["x"] = _normal((case["rows"], case["cols"]), g, case["type"])
        s["x"] *= torch.exp(torch.randn((case["rows"], 1), generator=g, device="cuda")).to(s["x"].dtype)
    elif case["op"] == "product":
        n, nb = case["rows"], -(-case["cols"] // 32)
        s["x"] = _normal((case["tokens"], case["cols"]), g, "bf16")
        codes = torch.randint(0, 256, (case["groups"], n, nb, 16), generator=g, device="cuda", dtype=torch.uint8)
        scales = torch.randint(116, 120, (case["groups"], n, nb), generator=g, device="cuda", dtype=torch.uint8)
        _, ids = _routing(case["tokens"], case["groups"], case["top_k"], case["zipf"], g)
        flat = ids.reshape(-1).long()
        order = torch.argsort(flat, stable=True)
        s["index"] = (order // case["top_k"]).to(torch.int32)
        counts = torch.bincount(flat, minlength=case["groups"])
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        s["counts"] = counts.tolist()
        if own:
            from routed_expert_ffn_forward_b200 import block
            s["weights"] = block.mx_pack(block.mx_rows(codes, scales, case["cols"]), paired=case["swiglu"])
        else:
            s["codes"], s["scales"] = codes, scales
    elif case["op"] == "norm":
        r, c, t = case["rows"], case["cols"], case["type"]
        s["h"], s["y"] = _normal((r, c), g, t, 2.0), _normal((r, c), g, t, 0.5)
        s["post"] = (1 + _normal((c,), g, scale=0.1)).to(TYPES[case["weights"]])
        s["pre"] = (1 + _normal((c,), g, scale=0.1)).to(TYPES[case["weights"]])
        s["gate"] = {"none": lambda: None, "token": lambda: torch.sigmoid(_normal((r, 1), g)).to(TYPES[t]),
                     "feature": lambda: _normal((c,), g, case["weights"], 0.3), "full": lambda: torch.sigmoid(_normal((r, c), g)).to(TYPES[t])}[case["gate"]]()
        s["d_out"], s["d_next"] = _normal((r, c), g, t), _normal((r, c), g, t)
    else:
        s["logits"], s["ids"] = _routing(case["tokens"], case["groups"], case["top_k"], 0.8, g)
        cuts = torch.rand(case["seqs"] - 1, generator=g, device="cuda").sort().values * (case["tokens"] + 1)
        s["offsets"] = torch.cat([cuts.new_zeros(1), cuts.floor(), cuts.new_full((1,), case["tokens"])]).to(torch.int32) if case["seqs"] > 1 else None
        s["mask"] = torch.rand(case["tokens"], generator=g, device="cuda") >= case["masked"] if case["masked"] else None
        s["d_loss"] = 0.5 + torch.rand((), generator=g, device="cuda")
    return s


EPS, SCALE, COEF = 1e-6, 0.7, 0.01


# ------------------------------------------------------------------------------------------------ MXFP4
def _quantized(x):
    """The values that rows of x stand for in MXFP4: runs of 32 under a power of two, each value to the nearest of E2M1, ties to even."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -cols % 32)).view(rows, -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top).exponent - 3).clamp(-127, 127)  # floor(log2(top)) - 2
    a = torch.ldexp(v.abs(), -e)
    a = a.masked_fill(top == 0, 0.0)
    code = (a > 0.25).int() + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    q = torch.ldexp(torch.tensor(E2M1[:8], device=x.device)[code.long()], e)
    q = torch.where(v < 0, -q, q).masked_fill(~torch.isfinite(top), float("nan"))
    return q.view(rows, -1)[:, :cols]


def _weights(codes, scales, cols):
    """One matrix from its codes (element j of a run of 32: low nibble of byte j, element 16 + j: its high nibble) and E8M0 scales."""
    pairs = torch.tensor([[E2M1[b & 15], E2M1[b >> 4]] for b in range(256)], device=codes.device)
    v = pairs[codes.long()].transpose(-1, -2).reshape(codes.shape[0], -1, 32)
    return torch.ldexp(v, (scales.int() - 127).unsqueeze(-1)).reshape(codes.shape[0], -1)[:, :cols]


def _activated(y, swiglu):
    if not swiglu:
        return y
    gate, up = y.chunk(2, dim=-1)
    return gate / (1 + torch.exp(-gate)) * up


def _product(s):
    case = s["case"]
    x = _quantized(s["x"])[s["index"].long()].split(s["counts"])
    y = torch.cat([_activated(a @ _weights(c, e, case["cols"]).T, case["swiglu"]) for a, c, e in zip(x, s["codes"], s["scales"]) if len(a)])
    return y.to(TYPES[case["out"]])


# ------------------------------------------------------------------------------------------------ the block's norms
def _norm_step(s, wide=torch.float32):
    """out = h + SCALE * gate * (y / rms(y) * post), next = out / rms(out) * pre, and the gradients of all inputs."""
    case = s["case"]
    h, y, post, pre = (s[k].to(wide) for k in ("h", "y", "post", "pre"))
    gate = torch.ones((), device=h.device, dtype=wide) if s["gate"] is None else s["gate"].to(wide)
    ry = torch.rsqrt((y * y).mean(-1, keepdim=True) + EPS)
    ny = y * ry
    z = ny * post
    out = h + SCALE * gate * z
    ro = torch.rsqrt((out * out).mean(-1, keepdim=True) + EPS)
    no = out * ro
    t = TYPES[case["type"]]
    res = dict(out=out.to(t), next=(no * pre).to(t))
    if case["step"]:
        d_next = s["d_next"].to(wide)
        a = d_next * pre
        d = s["d_out"].to(wide) + ro * (a - no * (a * no).mean(-1, keepdim=True))
        dz = SCALE * gate * d
        b = dz * post
        dy = ry * (b - ny * (b * ny).mean(-1, keepdim=True))
        res |= dict(d_h=d.to(t), d_y=dy.to(t), d_post=(dz * ny).sum(0).to(s["post"].dtype), d_pre=(d_next * no).sum(0).to(s["pre"].dtype))
        if s["gate"] is not None:
            dg = SCALE * z * d
            dg = {"token": lambda: dg.sum(1, keepdim=True), "feature": lambda: dg.sum(0), "full": lambda: dg}[case["gate"]]()
            res["d_gate"] = dg.to(s["gate"].dtype)
    return res


# ------------------------------------------------------------------------------------------------ the balance loss
def _balance(s):
    """Per sequence: f_i = groups / (top_k n) * how often expert i was picked, P_i = the mean probability of expert i over its n valid tokens;
    the loss is COEF times the mean over the sequences of sum_i f_i P_i.  The gradient takes the counts as constants."""
    case, logits = s["case"], s["logits"].float()
    tokens, groups = logits.shape
    ends = torch.full((1,), tokens, device=logits.device) if s["offsets"] is None else s["offsets"][1:]
    seqs = len(ends)
    seq = torch.bucketize(torch.arange(tokens, device=logits.device), ends.long(), right=True)
    valid = torch.ones(tokens, device=logits.device, dtype=torch.bool) if s["mask"] is None else s["mask"]
    picked = torch.zeros((seqs, groups), device=logits.device, dtype=torch.int32)
    cells = (seq[:, None] * groups + s["ids"].long()).reshape(-1)
    picked.view(-1).scatter_add_(0, cells, valid[:, None].int().expand_as(s["ids"]).reshape(-1))
    if case["sigmoid"]:
        w = 1 / (1 + torch.exp(-logits))
        p = w / w.sum(-1, keepdim=True)
    else:
        w = torch.exp(logits - logits.amax(-1, keepdim=True))
        p = w / w.sum(-1, keepdim=True)
    total = torch.zeros((seqs, groups), device=logits.device, dtype=torch.float64)  # sums over tens of thousands of tokens
    total.index_add_(0, seq, torch.where(valid[:, None], p, 0.0).double())
    n = torch.zeros(seqs, device=logits.device, dtype=torch.float64).index_add_(0, seq, valid.double())[:, None]
    f = groups / (case["top_k"] * n.clamp(min=1)) * picked
    live = (n > 0).sum().clamp(min=1)
    loss = (COEF / live * (f * total / n.clamp(min=1)).sum()).float()
    if not case["step"]:
        return dict(loss=loss, counts=picked)
    a = (s["d_loss"] * COEF / live * f / n.clamp(min=1)).float()[seq]
    d = p * (a - (p * a).sum(-1, keepdim=True))
    if case["sigmoid"]:
        d = d * (1 - w)
    return dict(loss=loss, counts=picked, d_logits=torch.where(valid[:, None], d, 0.0))


# ------------------------------------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        return _run_own(state, case)
    if case["op"] == "quantize":
        return _quantized(state["x"]).to(torch.bfloat16)  # every one of them is a bf16 number
    if case["op"] == "product":
        return _product(state)
    return _norm_step(state) if case["op"] == "norm" else _balance(state)


def _run_own(s, case):
    from routed_expert_ffn_forward_b200 import block, moe
    if case["op"] == "quantize":
        return block.mx_quantize(s["x"], values=True)[1]
    if case["op"] == "product":
        x = block.mx_quantize(s["x"])
        return block.mx_product(x, s["weights"], s["offsets"], s["index"], out_dtype=TYPES[case["out"]])
    if case["op"] == "norm":
        out, nxt, saved = block.block_norm_forward(s["h"], s["y"], s["post"], s["gate"], SCALE, s["pre"], EPS)
        res = dict(out=out, next=nxt)
        if case["step"]:
            d = block.block_norm_backward(s["d_out"], s["d_next"], s["h"], s["y"], s["post"], s["gate"], SCALE, s["pre"], saved)
            res |= {k: v for k, v in zip(("d_h", "d_y", "d_post", "d_gate", "d_pre"), d) if v is not None}
        return res
    gating = moe.MOE_GATE_SIGMOID_RENORM if case["sigmoid"] else moe.MOE_GATE_SOFTMAX_TOPK
    loss, counts, slope = block.balance_loss_forward(s["logits"], s["ids"], COEF, gating, s["offsets"], s["mask"])
    if not case["step"]:
        return dict(loss=loss, counts=counts)
    return dict(loss=loss, counts=counts, d_logits=block.balance_loss_backward(s["d_loss"], slope, s["logits"], gating, s["offsets"], s["mask"]))


# ------------------------------------------------------------------------------------------------ what a pass cannot do without
def work(case):
    if case["op"] == "quantize":
        n = case["rows"] * case["cols"]
        return dict(bytes=n * (BYTES[case["type"]] + 2 + 17 / 32), flops=4 * n)
    if case["op"] == "product":
        t, k, g, n, c = case["tokens"], case["top_k"], case["groups"], case["rows"], case["cols"]
        p = [r ** -case["zipf"] for r in range(1, g + 1)]
        active = sum(1 - (1 - min(1.0, k * v / sum(p))) ** t for v in p)  # experts with a token, on average
        active = max(active, k)
        outs = t * k * (n // 2 if case["swiglu"] else n)
        return dict(bytes=active * n * c * 17 / 32 + t * c * 2 + outs * BYTES[case["out"]] + t * k * 4, flops=2 * t * k * n * c)
    n = case["rows"] * case["cols"] if case["op"] == "norm" else case["tokens"] * case["groups"]
    if case["op"] == "norm":
        b, full = BYTES[case["type"]], case["gate"] == "full"
        once = 2 + full + 2  # h, y and a whole gate in, out and next out
        back = 4 + full + 2 + full if case["step"] else 0  # their gradients and the inputs again, the inputs' gradients out
        return dict(bytes=n * b * (once + back), flops=n * (12 + (24 if case["step"] else 0)))
    return dict(bytes=n * 4 * (3 if case["step"] else 1) + case["tokens"] * case["top_k"] * 4, flops=n * (5 + (6 if case["step"] else 0)))


# ------------------------------------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "quantize":
        return _mx_exact(s["x"])
    if case["op"] == "product":
        x, at, outs = _mx_exact(s["x"]), 0, []
        level = torch.tensor(E2M1, device="cuda", dtype=f64)
        for e, n in enumerate(s["counts"]):
            if n:
                byte = s["codes"][e].int()
                w = level[torch.cat([byte & 15, byte >> 4], -1)] * torch.exp2(s["scales"][e].double() - 127)[..., None]
                y = x[s["index"][at:at + n].long()] @ w.flatten(1)[:, :case["cols"]].T
                if case["swiglu"]:
                    half = y.shape[1] // 2
                    y = y[:, half:] * y[:, :half] * torch.sigmoid(y[:, :half])
                outs.append(y)
                at += n
        return torch.cat(outs)
    if case["op"] == "norm":
        leaf = {k: s[k].double().requires_grad_(case["step"]) for k in ("h", "y", "post", "pre", "gate") if s[k] is not None}
        z = leaf["y"] / torch.sqrt(leaf["y"].square().mean(1, keepdim=True) + EPS) * leaf["post"] * SCALE
        out = leaf["h"] + (z if s["gate"] is None else z * leaf["gate"])
        nxt = out / torch.sqrt(out.square().mean(1, keepdim=True) + EPS) * leaf["pre"]
        res = dict(out=out.detach(), next=nxt.detach())
        if case["step"]:
            names = sorted(leaf)
            grads = torch.autograd.grad([out, nxt], [leaf[k] for k in names], [s["d_out"].double(), s["d_next"].double()])
            res |= {"d_" + k: v for k, v in zip(names, grads)}
        return res
    logits = s["logits"].double().requires_grad_(case["step"])
    bounds = [0, case["tokens"]] if s["offsets"] is None else s["offsets"].tolist()
    p = torch.sigmoid(logits) if case["sigmoid"] else torch.softmax(logits, 1)
    p = p / p.sum(1, keepdim=True)
    valid = torch.ones(case["tokens"], device="cuda", dtype=torch.bool) if s["mask"] is None else s["mask"]
    terms, counts = [], []
    for lo, hi in zip(bounds, bounds[1:]):
        ok = valid[lo:hi]
        hits = torch.bincount(s["ids"][lo:hi][ok].reshape(-1).long(), minlength=case["groups"])
        counts.append(hits.int())
        if bool(ok.any()):
            n = ok.sum()
            terms.append((hits * case["groups"] / (case["top_k"] * n) * p[lo:hi][ok].sum(0) / n).sum())
    loss = COEF * (torch.stack(terms).mean() if terms else logits.sum() * 0)
    res = dict(loss=loss.detach(), counts=torch.stack(counts))
    if case["step"]:
        res["d_logits"] = torch.autograd.grad(loss, logits, s["d_loss"].double())[0]
    return res


def _mx_exact(x):
    """x's rows in MXFP4, from the distance between neighbouring values at each magnitude."""
    rows, cols = x.shape
    v = torch.nn.functional.pad(x.double(), (0, -cols % 32)).view(rows, -1, 32)
    top = v.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -125))) - 2)
    u = v / scale
    step = torch.where(u.abs() < 2, 0.5, torch.where(u.abs() < 4, 1.0, 2.0)).double()
    return ((torch.round(u / step) * step).clamp(-6, 6) * scale).view(rows, -1)[:, :cols]
