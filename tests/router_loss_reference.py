"""The router's training losses from their definitions, in 64 bits on the CPU
(no test functions here).  Written with autograd in mind: with ``logits``
requiring a gradient the losses are differentiable, so that the closed-form
gradients below can be checked against them."""
import math

import torch

F64 = torch.float64


def sequences(T, offsets):
    return [(0, T)] if offsets is None else [(int(a), int(b)) for a, b in zip(offsets[:-1], offsets[1:])]


def counted(T, mask, offsets):
    """Rows that lie in a sequence and are not masked, per sequence."""
    m = torch.ones(T, dtype=torch.bool) if mask is None else mask.bool()
    return [torch.tensor([t for t in range(a, b) if m[t]], dtype=torch.int64) for a, b in sequences(T, offsets)]


def scores(l, scoring):
    if scoring == "sigmoid":
        # exp(min(l,0)) / (1 + exp(-|l|)) about the row's maximum, so that no score is lost
        ls = torch.nn.functional.logsigmoid(l)
        return torch.softmax(ls, 1)
    return torch.softmax(l, 1)


def balance(logits, idx, scoring, mask=None, offsets=None):
    """dict of loss, z_loss, mean_scores, counts, tokens (lists over sequences stacked)."""
    T, E = logits.shape
    k = idx.shape[1]
    out = {"loss": [], "z_loss": [], "mean_scores": [], "counts": [], "tokens": []}
    for rows in counted(T, mask, offsets):
        L = len(rows)
        flat = idx[rows].reshape(-1)
        flat = flat[(flat >= 0) & (flat < E)]
        n = torch.bincount(flat, minlength=E)
        out["counts"].append(n)
        out["tokens"].append(L)
        if L == 0:
            zero = torch.zeros((), dtype=F64)
            out["loss"].append(zero), out["z_loss"].append(zero)
            out["mean_scores"].append(torch.zeros(E, dtype=F64))
            continue
        P = scores(logits[rows], scoring).mean(0)
        out["mean_scores"].append(P)
        out["loss"].append(E * (n.to(F64) / (k * L) * P).sum())
        out["z_loss"].append((torch.logsumexp(logits[rows], 1) ** 2).mean())
    return {"loss": torch.stack(out["loss"]), "z_loss": torch.stack(out["z_loss"]),
            "mean_scores": torch.stack(out["mean_scores"]), "counts": torch.stack(out["counts"]),
            "tokens": torch.tensor(out["tokens"])}


def balance_row_stats(logits, scoring, mask=None, offsets=None):
    T = logits.shape[0]
    st = torch.zeros((T, 2), dtype=F64)
    for rows in counted(T, mask, offsets):
        l = logits[rows]
        if not len(rows):
            continue
        m = l.amax(1)
        soft = torch.stack([m, torch.exp(l - m[:, None]).sum(1)], 1)
        if scoring == "sigmoid":
            sig = torch.stack([torch.zeros_like(m), torch.sigmoid(l).sum(1)], 1)
            soft = torch.where((m >= -20)[:, None], sig, soft)
        st[rows] = soft
    return st


def balance_grad(logits, counts, tokens, k, scoring, dloss, dz=None, mask=None, offsets=None):
    """(gradient, size of the terms it is summed from), both [T,E]."""
    T, E = logits.shape
    d, size = torch.zeros((T, E), dtype=F64), torch.zeros((T, E), dtype=F64)
    for s, rows in enumerate(counted(T, mask, offsets)):
        L = float(tokens[s])
        if not len(rows) or L == 0:
            continue
        l = logits[rows]
        p = scores(l, scoring)
        # about an even load: the scores sum to one, so the constant drops out
        g = dloss[s] * (E * counts[s].to(F64) - k * L) / (k * L * L)
        dot = (p * g).sum(1, keepdim=True)
        v, a = g - dot, g.abs() + (p * g.abs()).sum(1, keepdim=True)
        if dz is not None:
            z = 2 * dz[s] * torch.logsumexp(l, 1, keepdim=True) / L
            v, a = v + z, a + z.abs()
        w = p * torch.sigmoid(-l) if scoring == "sigmoid" else p
        d[rows], size[rows] = w * v, w * a
    return d, size


def targets(l, m, tau):
    """Stable descending order; the rest's logit."""
    order = torch.argsort(-l, dim=1, stable=True)
    s = torch.gather(l, 1, order)
    rest = (torch.full((l.shape[0],), -math.inf, dtype=F64) if m == l.shape[1]
            else tau * torch.logsumexp(s[:, m:] / tau, 1))
    return order[:, :m], s[:, :m], rest


def _row_sides(l, tidx, tl, trest, tau):
    """Of one row: listed experts, their q and log q, q_rest and its log, log p [E]."""
    on = [j for j in range(len(tidx)) if tl[j] != -math.inf]
    a = [tl[j] / tau for j in on] + ([trest / tau] if trest is not None else [])
    logq = torch.log_softmax(torch.stack(a), 0)
    logp = torch.log_softmax(l / tau, 0)
    e = torch.tensor([int(tidx[j]) for j in on], dtype=torch.int64)
    rest = logq[-1] if trest is not None else None
    return e, logq[: len(on)], rest, logp


def distill(logits, tidx, tl, trest, tau, mask=None, offsets=None):
    """(loss [S], tokens [S], row_loss [T], and per row the sum of |q - p|)."""
    T, E = logits.shape
    row = [torch.zeros((), dtype=F64) for _ in range(T)]
    diff = torch.zeros(T, dtype=F64)
    loss, tokens = [], []
    for rows in counted(T, mask, offsets):
        total, n = torch.zeros((), dtype=F64), 0
        for t in rows.tolist():
            if bool((tl[t] == -math.inf).all()) and (trest is None or float(trest[t]) == -math.inf):
                continue
            e, logq, lr, logp = _row_sides(logits[t], tidx[t], tl[t], None if trest is None else trest[t], tau)
            q = logq.exp()
            kl = (q * (logq - logp[e])).sum()
            df = (q - logp[e].exp()).abs().sum()
            out = torch.ones(E, dtype=torch.bool)
            out[e] = False
            if lr is not None and lr > -math.inf:
                lo = torch.logsumexp(logp[out], 0)
                kl = kl + lr.exp() * (lr - lo)
                df = df + (lr.exp() - lo.exp()).abs()
            row[t], diff[t] = kl, df.detach()
            total, n = total + kl, n + 1
        loss.append(total / max(n, 1))
        tokens.append(n)
    return torch.stack(loss), torch.tensor(tokens), torch.stack(row), diff


def distill_grad(logits, tidx, tl, trest, tau, tokens, dloss, mask=None, offsets=None):
    """(gradient, size of its terms), both [T,E]."""
    T, E = logits.shape
    d, size = torch.zeros((T, E), dtype=F64), torch.zeros((T, E), dtype=F64)
    for s, rows in enumerate(counted(T, mask, offsets)):
        for t in rows.tolist():
            if bool((tl[t] == -math.inf).all()) and (trest is None or float(trest[t]) == -math.inf):
                continue
            e, logq, lr, logp = _row_sides(logits[t], tidx[t], tl[t], None if trest is None else trest[t], tau)
            target = torch.zeros(E, dtype=F64)
            target[e] = logq.exp()
            out = torch.ones(E, dtype=torch.bool)
            out[e] = False
            if lr is not None and lr > -math.inf:
                target[out] = torch.softmax(logp[out], 0) * lr.exp()
            c = dloss[s] / (float(tokens[s]) * tau)
            d[t], size[t] = c * (logp.exp() - target), c.abs() * (logp.exp() + target)
    return d, size
