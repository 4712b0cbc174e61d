"""Plain float64 references of the block norms and the balance loss (torch, on
the CPU), differentiable."""
import torch


def block_norm(h, y, post, gate, scale, pre, eps):
    out = h
    if y is not None:
        z = y / torch.sqrt((y * y).mean(1, keepdim=True) + eps) * post
        out = h + scale * (z if gate is None else gate * z)
    nxt = None if pre is None else out / torch.sqrt((out * out).mean(1, keepdim=True) + eps) * pre
    return (None if y is None else out), nxt


def probabilities(logits, sigmoid):
    """softmax, or sigmoid / sum of sigmoid; zeros where no logit is above -infinity."""
    empty = torch.isneginf(logits).all(1, keepdim=True)
    safe = torch.where(empty, torch.zeros_like(logits), logits)
    if sigmoid:
        s = torch.nn.functional.logsigmoid(safe)
        p = torch.exp(s - torch.logsumexp(s, 1, keepdim=True))
    else:
        p = torch.softmax(safe, 1)
    return torch.where(empty, torch.zeros_like(p), p)


def balance_loss(logits, ids, coef, sigmoid, offsets=None, mask=None):
    """(loss, counts [seqs, experts])."""
    tokens, experts = logits.shape
    bounds = [0, tokens] if offsets is None else [min(max(int(o), 0), tokens) for o in offsets]
    p = probabilities(logits, sigmoid)
    terms, counts = [], []
    for lo, hi in zip(bounds, bounds[1:]):
        rows = [t for t in range(lo, hi) if mask is None or bool(mask[t])]
        picked = torch.zeros(experts, dtype=torch.int32)
        for t in rows:
            for e in ids[t].tolist():
                if 0 <= e < experts:
                    picked[e] += 1
        counts.append(picked)
        if rows:
            n = len(rows)
            terms.append((picked.double() * experts / (ids.shape[1] * n) * p[rows].mean(0)).sum())
    loss = coef * torch.stack(terms).mean() if terms else logits.sum() * 0
    return loss, torch.stack(counts)
