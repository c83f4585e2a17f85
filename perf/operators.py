"""Cases of the router's training losses: the balance loss with its per-expert
counts, and distillation from a teacher's top router logits.

Each case is one pass through one operator.  ``run`` computes it in plain torch
operations, or, with ``own`` set, through this package's calls.  ``exact`` gives
the same outputs from the definitions in 64 bits.

Shapes follow this repository's workloads (64 tokens over 4 experts in FP32,
16384 x 64 top-6, 8192 x 128 top-8, 32 x 256 top-8) and training batches of up
to 2^27 logits.
"""
import math

import torch

own = False

_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "f16": 2, "bf16": 2}
_MAX_LOGITS = 1 << 27


def _case(name, op, T, E, k, dtype, scoring="softmax", z=False, seqs=1, pad=0.0, tail=0, base=False,
          rest=False, temperature=1.0):
    case = dict(op=op, T=T, E=E, k=k, dtype=dtype, scoring=scoring, z=z, seqs=seqs, pad=pad, tail=tail,
                base=base, rest=rest, temperature=temperature)
    return case if name is None else dict(name=name, **case)


def listed():
    return [
        # the smallest training step of the layer: launch latency is everything
        _case("balance_tiny_f32", "balance", 64, 4, 2, "f32", z=True),
        # sequence-wise balance loss of a sigmoid router: FP32 router logits, ragged packed
        # sequences with padding at their ends and unused rows behind the last one
        _case("balance_sigmoid_ragged_f32", "balance", 65537, 256, 8, "f32", scoring="sigmoid", seqs=37,
              pad=0.1, tail=129),
        # the balance loss and z-loss of one large global batch
        _case("balance_large_bf16", "balance", 524288, 256, 8, "bf16", z=True),
        # the balance and z gradient added to the gradient of the routing weights, headline shape
        _case("balance_backward_headline_bf16", "balance_backward", 16384, 64, 6, "bf16", z=True, base=True),
        # the gradient of a sequence-wise loss over a large packed batch
        _case("balance_backward_large_bf16", "balance_backward", 524288, 256, 8, "bf16", seqs=128, pad=0.1),
        # a teacher's targets at the skewed workload's shape
        _case("targets_skewed_bf16", "targets", 8192, 128, 8, "bf16", temperature=2.0),
        # a teacher's targets with long lists, over a large batch
        _case("targets_large_bf16", "targets", 524288, 256, 32, "bf16"),
        # distillation on one decode-sized batch
        _case("distill_decode_f16", "distill", 32, 256, 8, "f16", rest=True),
        # distillation over a large batch
        _case("distill_large_bf16", "distill", 524288, 256, 8, "bf16", rest=True, temperature=2.0),
        # gradient at the headline shape, lists as long as the routed top-k, no rest
        _case("distill_backward_headline_bf16", "distill_backward", 16384, 64, 6, "bf16", base=True),
        # FP32 logits, an expert count that is no power of two, ragged padded sequences
        _case("distill_backward_ragged_f32", "distill_backward", 65537, 100, 16, "f32", rest=True, seqs=37,
              pad=0.3, tail=77, temperature=1.5),
        # gradient over a large batch with long lists
        _case("distill_backward_large_bf16", "distill_backward", 524288, 256, 32, "bf16", rest=True),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "balance_backward", "targets", "distill", "distill_backward"])
    dtype = rng.choice(["f32", "f16", "bf16", "bf16"])
    E = _log_uniform(rng, 2, 1024)
    if rng.random() < 0.5:  # expert counts are mostly multiples of eight
        E = min(1024, max(8, (E + 4) // 8 * 8))
    cap = _MAX_LOGITS // E // (2 if dtype == "f32" else 1)
    T = _log_uniform(rng, 1, min(cap, 524288))
    k = _log_uniform(rng, 1, min(E, 32))
    ragged = rng.random() < 0.5
    seqs = _log_uniform(rng, 1, max(1, min(T // 2, 512))) if ragged else 1
    scoring = rng.choice(["softmax", "sigmoid"]) if op.startswith("balance") else "softmax"
    return _case(None, op, T, E, k, dtype, scoring=scoring,
                 z=op.startswith("balance") and scoring == "softmax" and rng.random() < 0.5, seqs=seqs,
                 pad=rng.choice([0.0, 0.1, 0.3]) if ragged else 0.0,
                 tail=rng.randrange(0, T // 8 + 1) if ragged else 0,
                 base=op.endswith("backward") and rng.random() < 0.5,
                 rest=op.startswith("distill") and rng.random() < 0.7,
                 temperature=rng.choice([1.0, 1.5, 2.0, 4.0]))


def _seed(case, seed):
    return (seed * 1000003 + case["T"] * 8191 + case["E"] * 131 + case["k"]) % (1 << 62)


def prepare(case, seed):
    T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
    dt = _DT[case["dtype"]]
    dev = "cuda"
    gen = torch.Generator(device=dev).manual_seed(_seed(case, seed))
    host = torch.Generator().manual_seed(_seed(case, seed))
    op = case["op"]
    st = {"case": case}

    # router logits: unit normal per token, with experts that are liked more than others
    logits = torch.randn((T, E), generator=gen, device=dev)
    logits += 0.7 * torch.randn((E,), generator=gen, device=dev)
    teacher = None
    if op == "targets":
        st["logits"] = (1.5 * logits).to(dt)
    else:
        if op.startswith("distill"):  # the student is near its teacher
            teacher = (1.5 * logits + 0.5 * torch.randn((T, E), generator=gen, device=dev)).to(dt)
        st["logits"] = logits.to(dt)
        del logits
        if case["seqs"] > 1 or case["tail"] or case["pad"]:
            covered = T - case["tail"]
            cuts = torch.sort(torch.randint(0, covered + 1, (S - 1,), generator=host)).values
            off = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([covered])])
            st["seq_offsets"] = off.to(torch.int32).to(dev)
            if case["pad"]:
                length = off[1:] - off[:-1]
                valid_end = off[:-1] + length - (length.double() * case["pad"]).long()
                row = torch.arange(T)
                seq = torch.bucketize(row, off[1:], right=True).clamp_(max=S - 1)
                st["token_mask"] = (row < valid_end[seq]).to(dev)
        st["dloss"] = 0.01 * (1.0 + 0.25 * torch.rand((S,), generator=gen, device=dev))
        if case["dtype"] == "f16":  # half-precision gradients come with a loss scale
            st["dloss"] *= float(1 << (T - 1).bit_length())
        if case["base"]:
            st["base"] = (torch.randn((T, E), generator=gen, device=dev) * (st["dloss"].mean() / T)).to(dt)
    if op.startswith("balance"):
        idx = torch.topk(st["logits"], k, dim=1).indices
        if op == "balance":
            st["idx"] = idx.to(torch.int32)
        else:  # what the forward hands to the backward
            seq, ok = _rows(st)
            st["tokens"] = torch.bincount(seq[ok], minlength=S).to(torch.int32)
            flat = (seq[:, None] * E + idx)[ok].flatten()
            st["counts"] = torch.bincount(flat, minlength=S * E).to(torch.int32).view(S, E)
            st["row_stats"] = _keep(ok, _scores(st["logits"].float(), case["scoring"])[2])
            if case["z"]:
                st["dz_loss"] = 0.1 * st["dloss"]
    if op.startswith("distill"):
        tau = case["temperature"]
        top = torch.topk(teacher.float(), k, dim=1)
        st["teacher_idx"] = top.indices.to(torch.int32)
        st["teacher_logits"] = top.values.to(dt)
        if case["rest"]:
            others = teacher.float()
            others.scatter_(1, top.indices, float("-inf"))
            st["teacher_rest"] = tau * torch.logsumexp(others / tau, dim=1)
        if op == "distill_backward":
            seq, ok = _rows(st)
            st["tokens"] = torch.bincount(seq[ok], minlength=S).to(torch.int32)
            st["row_stats"] = _distill_stats(st, ok, *_distill_parts(st))
            st["row_loss"] = torch.zeros(T, device=dev)

    if own:
        import top_routing_grouped_fp32_gb300 as moe
        if op == "balance":
            st["workspace"] = moe.moe_balance_loss_workspace(T, E, S, dev)
            st["out"] = moe.BalanceLoss.empty(T, E, S, dev, z_loss=case["z"])
        elif op == "targets":
            st["out"] = moe.DistillTargets.empty(T, k, dt, dev)
        elif op == "distill":
            st["workspace"] = moe.moe_distill_loss_workspace(T, S, dev)
            st["out"] = moe.DistillLoss.empty(T, S, dev)
        else:
            st["dlogits"] = torch.empty_like(st["logits"])
            if op == "balance_backward":
                st["forward"] = moe.BalanceLoss(None, None, None, st["counts"], st["tokens"], st["row_stats"])
            else:
                st["forward"] = moe.DistillLoss(None, st["tokens"], st["row_loss"], st["row_stats"])
        if teacher is not None:
            st["targets"] = moe.DistillTargets(st["teacher_idx"], st["teacher_logits"], st.get("teacher_rest"))
    return st


def _rows(st):
    """(sequence of each row, whether the row counts)."""
    T, S = st["case"]["T"], st["case"]["seqs"]
    dev = st["logits"].device
    row = torch.arange(T, device=dev)
    off = st.get("seq_offsets")
    if off is None:
        seq = torch.zeros(T, dtype=torch.int64, device=dev)
        ok = torch.ones(T, dtype=torch.bool, device=dev)
    else:
        seq = torch.bucketize(row, off[1:].long(), right=True).clamp_(max=S - 1)
        ok = (row >= off[0]) & (row < off[-1])
    if "token_mask" in st:
        ok &= st["token_mask"]
    return seq, ok


def _per_seq(seq, S, values):
    """Sums of values [T,...] over each sequence, in 64 bits (long sums)."""
    if S == 1:
        return values.sum(0, keepdim=True, dtype=torch.float64)
    out = torch.zeros((S,) + values.shape[1:], dtype=torch.float64, device=values.device)
    return out.index_add_(0, seq, values.double())


def _keep(ok, rows):
    """Per-row values [T,n], zero where the row does not count."""
    return torch.where(ok[:, None], rows, torch.zeros((), device=rows.device))


def _scores(l, scoring):
    """Normalised scores, raw sigmoid scores or None, and each row's shift and sum: softmax
    (max, sum exp(l - max)), sigmoid (0, sum sigmoid(l)).  FP32."""
    if scoring == "sigmoid":
        s = 1.0 / (1.0 + torch.exp(-l))
        z = s.sum(1, keepdim=True)
        return s / z, s, torch.cat([torch.zeros_like(z), z], 1)
    m = l.max(1, keepdim=True).values
    e = torch.exp(l - m)
    z = e.sum(1, keepdim=True)
    return e / z, None, torch.cat([m, z], 1)


def _balance(st):
    case = st["case"]
    S, E, k = case["seqs"], case["E"], case["k"]
    seq, ok = _rows(st)
    p, _, stats = _scores(st["logits"].float(), case["scoring"])
    p = torch.where(ok[:, None], p, torch.zeros((), device=p.device))
    tokens = torch.zeros(S, dtype=torch.int32, device=p.device).index_add_(0, seq, ok.int())
    n = torch.clamp(tokens, min=1).double()[:, None]
    scores = _per_seq(seq, S, p) / n
    slot = (seq[:, None] * E + st["idx"]).flatten()
    counts = torch.zeros(S * E, dtype=torch.int32, device=p.device)
    counts.index_add_(0, slot, ok.int()[:, None].expand(-1, k).flatten())
    counts = counts.view(S, E)
    loss = E * (counts.double() / (k * n) * scores).sum(1)
    out = {"loss": loss.float(), "mean_scores": scores.float(), "counts": counts, "tokens": tokens,
           "row_stats": _keep(ok, stats)}
    if case["z"]:
        lse = stats[:, 0] + torch.log(stats[:, 1])
        sq = torch.where(ok, lse * lse, torch.zeros((), device=p.device))
        out["z_loss"] = (_per_seq(seq, S, sq) / n[:, 0]).float()
    return out


def _balance_backward(st):
    case = st["case"]
    E, k = case["E"], case["k"]
    seq, ok = _rows(st)
    l = st["logits"].float()
    p, s, stats = _scores(l, case["scoring"])
    n = torch.clamp(st["tokens"], min=1).double()
    # the share's distance from an even load: exact in 64 bits
    share = (st["counts"].double() * E - (k * n)[:, None]) / (k * n * n)[:, None]
    g = (st["dloss"].double()[:, None] * share).float()[seq]
    g = g - (p * g).sum(1, keepdim=True)
    if s is None:
        d = p * g
        if case["z"]:
            lse = stats[:, 0] + torch.log(stats[:, 1])
            d += p * (lse * (2.0 * st["dz_loss"].double() / n).float()[seq])[:, None]
    else:
        d = p * (1.0 - s) * g
    return _finish(st, ok, d)


def _finish(st, ok, d):
    d = torch.where(ok[:, None], d, torch.zeros((), device=d.device))
    if "base" in st:
        d = d + st["base"].float()
    return d.to(st["logits"].dtype)


def _targets(st):
    case = st["case"]
    k, E, tau = case["k"], case["E"], case["temperature"]
    l = st["logits"].float()
    v, i = torch.sort(l, dim=1, descending=True, stable=True)  # ties stay in order of their ids
    top, others = v[:, :k], v[:, k:] / tau
    if k == E:
        rest = torch.full((case["T"],), float("-inf"), device=l.device)
    else:
        m = others[:, :1]
        rest = tau * (m[:, 0] + torch.log(torch.exp(others - m).sum(1)))
    return {"idx": i[:, :k].to(torch.int32), "logits": top.to(st["logits"].dtype), "rest": rest}


def _distill_parts(st):
    """Exponentials and sums of the teacher's list (and rest) and of the student's row, and the
    student's sum outside the list.  FP32."""
    tau = st["case"]["temperature"]
    a = st["teacher_logits"].float()
    if "teacher_rest" in st:
        a = torch.cat([a, st["teacher_rest"][:, None]], 1)
    am = a.max(1, keepdim=True).values
    a = (a - am) / tau
    ea = torch.exp(a)
    b = st["logits"].float()
    bm = b.max(1, keepdim=True).values
    b = (b - bm) / tau
    eb = torch.exp(b)
    r = eb.scatter(1, st["teacher_idx"].long(), 0.0).sum(1, keepdim=True)
    return a, am, ea, ea.sum(1, keepdim=True), b, bm, eb, eb.sum(1, keepdim=True), r


def _distill_stats(st, ok, a, am, ea, za, b, bm, eb, zb, r):
    """[5,T]: maximum and sum of the student's row, of the teacher's list, and q_rest / p_rest."""
    ratio = torch.zeros_like(zb)
    if st["case"]["rest"]:
        ratio = torch.where(r > 0, (ea[:, -1:] / za) / (r / zb), ratio)
    return _keep(ok, torch.cat([bm, zb, am, za, ratio], 1)).t().contiguous()


def _kl_term(q, p, d):
    """q log(q/p) - q + p, d = log(q/p): q h(d) with h's series where the three nearly cancel."""
    h = 1 / 2 - d * (1 / 6 - d * (1 / 24 - d * (1 / 120 - d * (1 / 720 - d * (1 / 5040 - d / 40320)))))
    t = torch.where(d.abs() < 0.5, q * d * d * h, p - q + q * d)
    return torch.where(q > 0, t, p)


def _distill(st):
    case = st["case"]
    S, m = case["seqs"], case["k"]
    seq, ok = _rows(st)
    parts = _distill_parts(st)
    a, am, ea, za, b, bm, eb, zb, r = parts
    q = ea / za
    ti = st["teacher_idx"].long()
    # sum q log(q/p) = sum (q log(q/p) - q + p) over the list and the rest, as both sides sum to
    # one: every term is >= 0, so that near distributions keep their digits
    logp, pj = torch.gather(b, 1, ti), torch.gather(eb, 1, ti)
    if case["rest"]:
        logp, pj = torch.cat([logp, torch.log(r)], 1), torch.cat([pj, r], 1)
    kl = _kl_term(q, pj / zb, (a - logp) + (torch.log(zb) - torch.log(za))).sum(1)
    if not case["rest"]:
        kl = kl + (r / zb)[:, 0]
    kl = torch.where(ok, kl, torch.zeros((), device=kl.device))
    tokens = torch.zeros(S, dtype=torch.int32, device=kl.device).index_add_(0, seq, ok.int())
    loss = (_per_seq(seq, S, kl) / torch.clamp(tokens, min=1)).float()
    return {"loss": loss, "tokens": tokens, "row_loss": kl,
            "row_stats": _distill_stats(st, ok, *parts)}


def _distill_backward(st):
    case = st["case"]
    m = case["k"]
    seq, ok = _rows(st)
    a, am, ea, za, b, bm, eb, zb, r = _distill_parts(st)
    q = ea / za
    ti = st["teacher_idx"].long()
    d = eb / zb
    if case["rest"]:
        others = eb.scatter(1, ti, 0.0)
        d = d - torch.where(r > 0, others / r * q[:, m:], torch.zeros((), device=d.device))
    d.scatter_add_(1, ti, -q[:, :m])
    c = st["dloss"].double() / torch.clamp(st["tokens"], min=1) / case["temperature"]
    return _finish(st, ok, d * c.float()[seq][:, None])


def run(st):
    case = st["case"]
    op = case["op"]
    if not own:
        return {"balance": _balance, "balance_backward": _balance_backward, "targets": _targets,
                "distill": _distill, "distill_backward": _distill_backward}[op](st)
    import top_routing_grouped_fp32_gb300 as moe
    mask, off = st.get("token_mask"), st.get("seq_offsets")
    if op == "balance":
        r = moe.moe_balance_loss(st["logits"], st["idx"], scoring=case["scoring"], token_mask=mask,
                                 seq_offsets=off, z_loss=case["z"], out=st["out"], workspace=st["workspace"])
        out = {"loss": r.loss, "mean_scores": r.mean_scores, "counts": r.counts, "tokens": r.tokens,
               "row_stats": r.row_stats}
        if case["z"]:
            out["z_loss"] = r.z_loss
        return out
    if op == "balance_backward":
        return moe.moe_balance_loss_backward(st["logits"], st["forward"], case["k"], st["dloss"],
                                             scoring=case["scoring"], seq_offsets=off,
                                             dz_loss=st.get("dz_loss"), base=st.get("base"),
                                             dlogits=st["dlogits"])
    if op == "targets":
        r = moe.moe_distill_targets(st["logits"], case["k"], temperature=case["temperature"], out=st["out"])
        return {"idx": r.idx, "logits": r.logits, "rest": r.rest}
    if op == "distill":
        r = moe.moe_distill_loss(st["logits"], st["targets"], temperature=case["temperature"], token_mask=mask,
                                 seq_offsets=off, out=st["out"], workspace=st["workspace"])
        return {"loss": r.loss, "tokens": r.tokens, "row_loss": r.row_loss, "row_stats": r.row_stats}
    return moe.moe_distill_loss_backward(st["logits"], st["targets"], st["forward"], st["dloss"],
                                         temperature=case["temperature"], seq_offsets=off,
                                         base=st.get("base"), dlogits=st["dlogits"])


def work(case):
    T, E, k, S = case["T"], case["E"], case["k"], case["seqs"]
    size = _SIZE[case["dtype"]]
    op = case["op"]
    valid = int((T - case["tail"]) * (1.0 - case["pad"]))  # rows that count
    row = valid * E * size
    offsets = 4 * (S + 1) if S > 1 or case["tail"] else 0
    per_row = (T if case["pad"] else 0) + offsets
    if op == "balance":
        return {"bytes": row + valid * k * 4 + per_row + 8 * T + S * (2 * E + 2 + case["z"]) * 4,
                "flops": 7 * valid * E}
    if op == "balance_backward":
        return {"bytes": row + 8 * T + T * E * size * (1 + case["base"]) + offsets + S * (E + 2 + case["z"]) * 4,
                "flops": 7 * valid * E}
    if op == "targets":
        return {"bytes": T * E * size + T * k * (4 + size) + 4 * T, "flops": 5 * T * E}
    lists = valid * k * (4 + size)
    if op == "distill":
        return {"bytes": row + lists + valid * 4 * case["rest"] + per_row + 24 * T + 8 * S,
                "flops": 5 * valid * E + 8 * valid * k}
    return {"bytes": row + lists + 20 * T + T * E * size * (1 + case["base"]) + offsets + 8 * S,
            "flops": 4 * valid * E + 6 * valid * k}


def _exact_rows(st, chunk):
    """Row ranges with their sequence ids and whether they count, one pass over the batch."""
    seq, ok = _rows(st)
    for a in range(0, st["case"]["T"], chunk):
        b = min(a + chunk, st["case"]["T"])
        yield a, b, seq[a:b], ok[a:b]


def exact(case, seed):
    st = prepare(case, seed)
    T, E, k, S, tau = case["T"], case["E"], case["k"], case["seqs"], case["temperature"]
    dev = st["logits"].device
    f64 = torch.float64
    op = case["op"]
    chunk = max(1, (1 << 24) // E)
    if op == "targets":
        idx, top, rest = [], [], []
        for a in range(0, T, chunk):
            l = st["logits"][a:a + chunk].to(f64)
            order = torch.argsort(-l, dim=1, stable=True)
            s = torch.gather(l, 1, order)
            idx.append(order[:, :k].to(torch.int32))
            top.append(s[:, :k])
            rest.append(tau * torch.logsumexp(s[:, k:] / tau, 1) if k < E
                        else torch.full((l.shape[0],), float("-inf"), dtype=f64, device=dev))
        return {"idx": torch.cat(idx), "logits": torch.cat(top), "rest": torch.cat(rest)}
    if op == "balance":
        total = torch.zeros((S, E), dtype=f64, device=dev)
        zsum = torch.zeros(S, dtype=f64, device=dev)
        counts = torch.zeros((S, E), dtype=torch.int64, device=dev)
        tokens = torch.zeros(S, dtype=torch.int64, device=dev)
        stats = torch.zeros((T, 2), dtype=f64, device=dev)
        for a, b, seq, ok in _exact_rows(st, chunk):
            l, sq = st["logits"][a:b].to(f64)[ok], seq[ok]
            if case["scoring"] == "sigmoid":
                s = torch.sigmoid(l)
                p = s / s.sum(1, keepdim=True)
                stats[a:b, 1][ok] = s.sum(1)
            else:
                p = torch.softmax(l, 1)
                stats[a:b, 0][ok] = l.amax(1)
                stats[a:b, 1][ok] = 1.0 / p.amax(1)
                zsum.index_add_(0, sq, torch.logsumexp(l, 1) ** 2)
            total.index_add_(0, sq, p)
            hot = torch.zeros((p.shape[0], E), dtype=torch.int64, device=dev)
            hot.scatter_add_(1, st["idx"][a:b].long()[ok], torch.ones_like(hot[:, :1]).expand(-1, k))
            counts.index_add_(0, sq, hot)
            tokens += torch.bincount(sq, minlength=S)
        n = tokens.clamp(min=1).to(f64)
        mean = total / n[:, None]
        out = {"loss": E / k * (counts / n[:, None] * mean).sum(1), "mean_scores": mean,
               "counts": counts.to(torch.int32), "tokens": tokens.to(torch.int32), "row_stats": stats}
        if case["z"]:
            out["z_loss"] = zsum / n
        return out
    if op == "balance_backward":
        out = torch.zeros((T, E), dtype=f64, device=dev)
        n = st["tokens"].clamp(min=1).to(f64)
        for a, b, seq, ok in _exact_rows(st, chunk):
            l = st["logits"][a:b].to(f64)
            w = (st["dloss"].to(f64) * E / (k * n * n))[seq][:, None] * st["counts"].to(f64)[seq]
            if case["scoring"] == "sigmoid":
                s = torch.sigmoid(l)
                tot = s.sum(1, keepdim=True)
                d = s * torch.sigmoid(-l) / tot * (w - (s * w).sum(1, keepdim=True) / tot)
            else:
                p = torch.softmax(l, 1)
                d = p * (w - (p * w).sum(1, keepdim=True))
                if case["z"]:
                    d += p * (2 * st["dz_loss"].to(f64) / n)[seq][:, None] * torch.logsumexp(l, 1, keepdim=True)
            out[a:b] = torch.where(ok[:, None], d, torch.zeros_like(d))
            if "base" in st:
                out[a:b] += st["base"][a:b].to(f64)
        return out
    # distillation
    loss = torch.zeros(S, dtype=f64, device=dev)
    tokens = torch.zeros(S, dtype=torch.int64, device=dev)
    row_loss = torch.zeros(T, dtype=f64, device=dev)
    stats = torch.zeros((5, T), dtype=f64, device=dev)
    grad = torch.zeros((T, E), dtype=f64, device=dev) if op == "distill_backward" else None
    for a, b, seq, ok in _exact_rows(st, chunk):
        t = st["teacher_logits"][a:b].to(f64) / tau
        ti = st["teacher_idx"][a:b].long()
        if case["rest"]:
            t = torch.cat([t, st["teacher_rest"][a:b].to(f64)[:, None] / tau], 1)
        logq = torch.log_softmax(t, 1)
        q = logq.exp()
        b64 = st["logits"][a:b].to(f64) / tau
        logp = torch.log_softmax(b64, 1)
        outside = logp.scatter(1, ti, float("-inf"))
        kl = (q[:, :k] * (logq[:, :k] - torch.gather(logp, 1, ti))).sum(1)
        if case["rest"]:
            part = q[:, k] * (logq[:, k] - torch.logsumexp(outside, 1))
            kl = kl + torch.where(q[:, k] > 0, part, torch.zeros_like(part))
        if grad is None:
            ratio = torch.zeros_like(kl)
            if case["rest"]:
                out_p = torch.logsumexp(outside, 1)
                ratio = torch.where(out_p > float("-inf"), (logq[:, k] - out_p).exp(), ratio)
            new = torch.stack([b64.amax(1) * tau, 1 / logp.amax(1).exp(), t.amax(1) * tau,
                               1 / logq.amax(1).exp(), ratio])
            stats[:, a:b] = torch.where(ok, new, torch.zeros_like(new))
            row_loss[a:b] = torch.where(ok, kl, torch.zeros_like(kl))
            loss.index_add_(0, seq[ok], kl[ok])
            tokens += torch.bincount(seq[ok], minlength=S)
            continue
        target = torch.zeros_like(logp).scatter_(1, ti, q[:, :k])
        if case["rest"] and k < E:
            target = target + torch.softmax(outside, 1) * q[:, k:]
        c = (st["dloss"].to(f64) / st["tokens"].clamp(min=1) / tau)[seq][:, None]
        d = c * (logp.exp() - target)
        grad[a:b] = torch.where(ok[:, None], d, torch.zeros_like(d))
        if "base" in st:
            grad[a:b] += st["base"][a:b].to(f64)
    if grad is not None:
        return grad
    return {"loss": loss / tokens.clamp(min=1), "tokens": tokens.to(torch.int32), "row_loss": row_loss,
            "row_stats": stats}
