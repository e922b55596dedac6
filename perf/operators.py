"""Cases of the router's training operators: the balance loss and the
distillation loss with their gradients, the route's backward pass and the
combine's backward pass.

run() computes one training step's share of an operator: the loss forward and
backward, or the backward pass with every gradient it gives. With `own` false
it is the plain form in elementary torch operations in FP32, with `own` true
the calls of moe_token_routing_amd.
"""
import math

import torch

own = False

DEV = "cuda"
SIGMOID, SOFTMAX = 0, 1   # the router's score functions


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # the balance loss of a handful of tokens (a smoke run, a debug step): latency
        {"name": "balance_tiny", "op": "balance", "T": 16, "E": 16, "k": 4, "S": 1, "score": SIGMOID},
        # a packed training batch of ragged sequences, the last one ending before the batch does,
        # 5% of the tokens invalid (padding, NaN logits); an expert count off the vector width
        {"name": "balance_ragged", "op": "balance", "T": 8111, "E": 254, "k": 8, "S": 13, "score": SIGMOID},
        # many tokens, 22 picks each, softmax scores, one loss over the whole batch
        {"name": "balance_wide_k", "op": "balance", "T": 32768, "E": 512, "k": 22, "S": 1, "score": SOFTMAX},
        # distillation on a single token
        {"name": "distill_token", "op": "distill", "T": 1, "E": 64, "k": 4, "score": SIGMOID, "temperature": 1.0},
        # a batch of 8192 tokens, the teacher's eight picks of 256 experts
        {"name": "distill_batch", "op": "distill", "T": 8192, "E": 256, "k": 8, "score": SIGMOID,
         "temperature": 1.0},
        # thousands of experts, softmax scores, a softened teacher, an odd number of its entries
        {"name": "distill_large_e", "op": "distill", "T": 4093, "E": 2560, "k": 31, "score": SOFTMAX,
         "temperature": 2.0},
        # the route's backward pass of a few tokens in FP32
        {"name": "route_bwd_tiny", "op": "route", "T": 16, "H": 256, "E": 16, "k": 4, "dtype": "f32"},
        # the 8192-token batch in BF16
        {"name": "route_bwd_batch", "op": "route", "T": 8192, "H": 8192, "E": 256, "k": 8, "dtype": "bf16"},
        # thousands of experts, a token count off every tile
        {"name": "route_bwd_large_e", "op": "route", "T": 4001, "H": 4096, "E": 2560, "k": 8, "dtype": "bf16"},
        # the combine's backward pass of a few tokens
        {"name": "combine_bwd_tiny", "op": "combine", "T": 16, "H": 256, "k": 4, "center": 0.0},
        # the 8192-token batch: 65536 expert rows of 8192
        {"name": "combine_bwd_batch", "op": "combine", "T": 8192, "H": 8192, "k": 8, "center": 0.0},
        # narrow rows, 22 per token, the gain stored as an offset from one
        {"name": "combine_bwd_wide_k", "op": "combine", "T": 16411, "H": 1032, "k": 22, "center": 1.0},
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["balance", "distill", "route", "combine"])
    if op in ("balance", "distill"):
        E = _log_uniform(rng, 8, 4096)
        T = _log_uniform(rng, 1, min(32768, (1 << 24) // E))
        case = {"op": op, "T": T, "E": E, "k": rng.randint(1, min(E, 32)), "score": rng.choice([SIGMOID, SOFTMAX])}
        if op == "balance":
            case["S"] = _log_uniform(rng, 1, 64)
        else:
            case["temperature"] = rng.choice([0.5, 1.0, 2.0, 4.0])
        return case
    if op == "route":
        H = 16 * _log_uniform(rng, 1, 512)
        E = _log_uniform(rng, 8, 2560)
        T = _log_uniform(rng, 1, min(8192, (1 << 34) // (H * E)))
        return {"op": op, "T": T, "H": H, "E": E, "k": rng.randint(1, min(E, 32)),
                "dtype": rng.choice(["bf16", "bf16", "f32"])}
    H = 8 * _log_uniform(rng, 1, 1024)
    k = rng.randint(1, 32)
    return {"op": op, "T": _log_uniform(rng, 1, min(32768, (1 << 28) // (H * k))), "H": H, "k": k,
            "center": rng.choice([0.0, 1.0])}


# ----------------------------------------------------------------- inputs ----

def _normal(g, shape, std=1.0):
    return torch.randn(shape, generator=g, device=DEV) * std


def _logits(g, T, E):
    """Router logits: unit spread and a preference of every batch for some experts."""
    return _normal(g, (T, E)) + _normal(g, (1, E), 0.5)


def _mask(g, T):
    """Validity of each token; 5% are invalid (none in batches of a few tokens)."""
    mask = torch.rand(T, generator=g, device=DEV) >= 0.05
    if T < 20:
        mask[:] = True
    return mask


def _picks(logits, mask, k):
    """The k experts of each token in order of score, -1 and weight 0 for invalid tokens."""
    score = torch.sigmoid(logits)
    top, ids = torch.sort(score, dim=1, descending=True, stable=True)
    top, ids = top[:, :k], ids[:, :k].int()
    w = top / top.sum(1, keepdim=True)
    valid = mask[:, None]
    return (torch.where(valid, ids, torch.full_like(ids, -1)).contiguous(),
            torch.where(valid, w, torch.zeros_like(w)).contiguous())


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    op, T, k = case["op"], case["T"], case["k"]
    s = dict(case)
    mask = _mask(g, T)
    if op == "combine":
        H = case["H"]
        R = T * k
        # rows in the order of a dispatch: the valid slots permuted over the first rows, the
        # rest of the expert output never written
        valid = (torch.rand((T, k), generator=g, device=DEV) >= 0.03) & mask[:, None]
        order = torch.argsort(torch.rand(R, generator=g, device=DEV) + 2.0 * (~valid.reshape(-1)))
        slots = torch.empty(R, dtype=torch.int32, device=DEV)
        slots[order] = torch.arange(R, dtype=torch.int32, device=DEV)
        s["slots"] = torch.where(valid, slots.view(T, k), -1).int().contiguous()
        rows = torch.empty((R, H), dtype=torch.bfloat16, device=DEV)
        for r in range(0, R, 8192):
            rows[r:r + 8192] = _normal(g, (min(8192, R - r), H)).bfloat16()
        rows[int(valid.sum()):] = float("nan")
        s["expert_out"] = rows
        w = torch.rand((T, k), generator=g, device=DEV) + 0.05
        s["topk_w"] = w / w.sum(1, keepdim=True)
        s["norm_w"] = torch.rand(H, generator=g, device=DEV) + 0.5 - case["center"]
        s["d_out"] = _normal(g, (T, H), 1e-2).bfloat16()
        s["eps"] = 1e-6
        return s
    E = case["E"]
    logits = _logits(g, T, E)
    s["mask"] = mask.to(torch.uint8)
    if op == "balance":
        s["ids"], _ = _picks(logits, mask, k)
        # ragged sequences, some empty; tokens behind the last one belong to none
        cut = torch.sort(torch.randint(0, T + 1, (case["S"] + 1,), generator=g, device=DEV)).values
        cut[0] = 0
        if case["S"] == 1:
            cut[1] = T
        s["seq_offsets"] = cut.int()
        s["d_losses"] = torch.tensor([1e-2, 1e-3], device=DEV)
    elif op == "distill":
        teacher = logits + _normal(g, (T, E), 0.5)
        z, ids = torch.sort(teacher, dim=1, descending=True, stable=True)
        s["t_logits"], s["t_ids"] = z[:, :k].contiguous(), ids[:, :k].int().contiguous()
        if T >= 20:   # a teacher that kept fewer entries for some tokens, and none for a few
            kept = torch.randint(0, k + 1, (T, 1), generator=g, device=DEV)
            kept = torch.where(torch.rand((T, 1), generator=g, device=DEV) < 0.1, kept, k)
            s["t_ids"][torch.arange(k, device=DEV)[None, :] >= kept] = -1
        s["d_loss"] = torch.tensor([0.5], device=DEV)
    else:
        H = case["H"]
        s["ids"], s["topk_w"] = _picks(logits, mask, k)
        s["hidden"] = torch.empty((T, H), dtype=torch.bfloat16 if case["dtype"] == "bf16" else torch.float32, device=DEV)
        for t in range(0, T, 4096):
            s["hidden"][t:t + 4096] = _normal(g, (min(4096, T - t), H))
        s["hidden"][~mask] = float("nan")
        s["W"] = _normal(g, (E, H), 1.0 / math.sqrt(H))
        s["scale"] = 0.75
        s["d_topk_w"] = _normal(g, (T, k), 1e-2)
        s["d_aux"] = _normal(g, (T, E), 1e-5)   # what the losses of the logits add
    logits[~mask] = float("nan")
    s["logits"] = logits
    return s


# -------------------------------------------------------------- plain form ----

def _log_score(x, score):
    """log of the router's score up to a constant of the row, and the slope of that log."""
    if score == SOFTMAX:
        return x, torch.ones_like(x)
    e = torch.exp(-x.abs())
    return torch.clamp(x, max=0.0) - torch.log(1.0 + e), torch.where(x > 0, e, torch.ones_like(e)) / (1.0 + e)


def _log_softmax(x):
    top = x.max(1, keepdim=True).values
    x = x - top
    total = torch.log(torch.exp(x).sum(1, keepdim=True))
    return x - total, top + total


def _balance(s):
    S, E, k = s["S"], s["E"], s["k"]
    T = s["T"]
    at = torch.arange(T, device=DEV)
    off = s["seq_offsets"].long()
    part = (at[None, :] >= off[:-1, None]) & (at[None, :] < off[1:, None]) & (s["mask"] != 0)[None, :]   # [S,T]
    valid = part.any(0)
    x = torch.where(valid[:, None], s["logits"], torch.zeros_like(s["logits"]))
    ls, slope = _log_score(x, s["score"])
    p = torch.exp(_log_softmax(ls)[0])
    logp, lse = _log_softmax(x)
    member = part.float()
    probs = member @ p
    seq = torch.where(valid, part.int().argmax(0), torch.full_like(at, S))
    cell = torch.where((s["ids"] >= 0) & (s["ids"] < E) & valid[:, None], seq[:, None] * E + s["ids"], S * E)
    counts = torch.zeros(S * E + 1, dtype=torch.int32, device=DEV)
    counts.index_add_(0, cell.reshape(-1).long(), torch.ones(T * k, dtype=torch.int32, device=DEV))
    counts = counts[:-1].view(S, E)
    tokens = part.sum(1)
    n, full = tokens.sum(), (tokens > 0).sum()
    weight = torch.where(tokens > 0, E / (k * tokens.float().square() * full.clamp(min=1)), torch.zeros(S, device=DEV))
    each = (weight[:, None] * counts * probs).sum()
    z = (torch.where(valid[:, None], lse, torch.zeros_like(lse)).square().sum()) / n.clamp(min=1)
    # gradient of d_losses . (balance, z)
    c = torch.cat([weight[:, None] * counts, torch.zeros((1, E), device=DEV)])[seq] * s["d_losses"][0]
    d = p * (c - (p * c).sum(1, keepdim=True)) * slope
    d = d + s["d_losses"][1] * 2.0 * lse / n.clamp(min=1) * torch.exp(logp)
    d = torch.where(valid[:, None], d, torch.zeros_like(d))
    return {"losses": torch.stack([each, z]), "counts": counts, "probs": probs,
            "tokens": torch.cat([tokens, n[None], full[None]]).int(), "d_logits": d}


def _distill(s):
    tau = s["temperature"]
    ok = (s["t_ids"] >= 0) & (s["t_ids"] < s["E"]) & (s["mask"] != 0)[:, None]
    has = ok.any(1, keepdim=True)
    z, _ = _log_score(s["t_logits"] / tau, s["score"])
    z = torch.where(ok, z, torch.full_like(z, float("-inf")))
    z = torch.where(has, z, torch.zeros_like(z))
    logq, _ = _log_softmax(z)
    q = torch.where(ok, torch.exp(logq), torch.zeros_like(logq))
    x = torch.where(has, s["logits"], torch.zeros_like(s["logits"])) / tau
    ls, slope = _log_score(x, s["score"])
    logp, _ = _log_softmax(ls)
    ids = s["t_ids"].long().clamp(0, s["E"] - 1)
    term = q * (logq - torch.gather(logp, 1, ids)) * (tau * tau)
    token_loss = torch.where(ok, term, torch.zeros_like(term)).sum(1)
    n = has.sum()
    d = torch.exp(logp)
    d = d.scatter_add(1, ids, -q) * slope * (s["d_loss"] * tau / n.clamp(min=1))
    d = torch.where(has, d, torch.zeros_like(d))
    return {"loss": (token_loss.sum() / n.clamp(min=1))[None], "token_loss": token_loss, "tokens": n[None].int(),
            "d_logits": d}


def _route(s):
    valid = (s["mask"] != 0)[:, None]
    ids = s["ids"].long().clamp(min=0)
    ok = (s["ids"] >= 0) & valid
    w = torch.where(ok, s["topk_w"], torch.zeros_like(s["topk_w"]))
    dw = torch.where(ok, s["d_topk_w"], torch.zeros_like(s["d_topk_w"]))
    l = torch.where(ok, torch.gather(s["logits"], 1, ids), torch.zeros_like(w))
    d = w * (dw - (w * dw).sum(1, keepdim=True)) / (1.0 + torch.exp(l))
    d_logits = torch.where(valid, s["d_aux"].scatter_add(1, ids, d), torch.zeros_like(s["d_aux"]))
    hidden = torch.where(valid, s["hidden"].float(), torch.zeros((), device=DEV))
    d_hidden = (d_logits @ s["W"]) * s["scale"]
    d_W = (d_logits.t() @ hidden) * s["scale"]
    return {"d_logits": d_logits, "d_hidden": d_hidden.to(s["hidden"].dtype), "d_W": d_W}


def _combine(s):
    T, H, k, R = s["T"], s["H"], s["k"], s["T"] * s["k"]
    slots = s["slots"].long()
    ok = (slots >= 0) & (slots < R)
    x = torch.where(ok[..., None], s["expert_out"][slots.clamp(0, R - 1)].float(), torch.zeros((), device=DEV))
    gain = s["norm_w"] + s["center"]
    rstd = torch.rsqrt(x.square().mean(2, keepdim=True) + s["eps"])
    rstd = torch.where(ok[..., None], rstd, torch.zeros_like(rstd))
    g = s["d_out"].float()[:, None, :]
    a = (x * gain * g).sum(2, keepdim=True)
    w = s["topk_w"][..., None]
    d_norm_w = (g[:, 0] * (x * (w * rstd)).sum(1)).sum(0)
    dx = (w * rstd) * (gain * g - x * (rstd.square() * a / H))
    d_rows = torch.zeros((R + 1, H), dtype=torch.bfloat16, device=DEV)
    d_rows.index_copy_(0, torch.where(ok, slots, R).reshape(-1), dx.reshape(T * k, H).bfloat16())
    return {"d_expert_out": d_rows[:R], "d_topk_w": (rstd * a)[..., 0], "d_norm_w": d_norm_w}


def _own(s):
    import moe_token_routing_amd as m
    op = s["op"]
    if op == "balance":
        losses, counts, probs, tokens = m.balance_loss(s["logits"], s["ids"], s["mask"], score=s["score"],
                                                       seq_offsets=s["seq_offsets"])
        d = m.balance_loss_backward(s["d_losses"], s["logits"], s["mask"], counts, tokens, s["k"], score=s["score"],
                                    seq_offsets=s["seq_offsets"])
        return {"losses": losses, "counts": counts, "probs": probs, "tokens": tokens, "d_logits": d}
    if op == "distill":
        loss, token_loss, tokens = m.distill_loss(s["logits"], s["t_ids"], s["t_logits"], s["mask"], score=s["score"],
                                                  temperature=s["temperature"])
        d = m.distill_loss_backward(s["d_loss"], s["logits"], s["t_ids"], s["t_logits"], s["mask"], tokens,
                                    score=s["score"], temperature=s["temperature"])
        return {"loss": loss, "token_loss": token_loss, "tokens": tokens, "d_logits": d}
    if op == "route":
        d_logits, d_hidden, d_W = m.route_backward(s["d_topk_w"], s["hidden"], s["W"], s["logits"], s["ids"],
                                                   s["topk_w"], s["mask"], s["scale"], d_aux=s["d_aux"])
        return {"d_logits": d_logits, "d_hidden": d_hidden, "d_W": d_W}
    d_rows, d_w, d_norm_w = m.combine_backward(s["d_out"], s["expert_out"], s["slots"], s["topk_w"], s["norm_w"],
                                               s["center"], s["eps"])
    return {"d_expert_out": d_rows, "d_topk_w": d_w, "d_norm_w": d_norm_w}


def run(state):
    if own:
        return _own(state)
    return {"balance": _balance, "distill": _distill, "route": _route, "combine": _combine}[state["op"]](state)


# -------------------------------------------------- what a pass cannot do without ----

def work(case):
    op, T, k = case["op"], case["T"], case["k"]
    if op == "combine":
        H = case["H"]
        rows = T * k * H * 2
        # expert rows and d_out in, row gradients out; slots, weights and their gradients; gains
        return {"bytes": 2 * rows + T * H * 2 + 3 * T * k * 4 + 2 * H * 4, "flops": 13 * T * k * H}
    E = case["E"]
    table = T * E * 4
    if op == "balance":
        S = case["S"]
        return {"bytes": 2 * table + T * k * 4 + T + 2 * S * E * 4 + 8 * S, "flops": 20 * T * E}
    if op == "distill":
        return {"bytes": 2 * table + 2 * T * k * 4 + T + T * 4, "flops": 16 * T * E}
    H = case["H"]
    size = 2 if case["dtype"] == "bf16" else 4
    # logits are read at the picks alone
    return {"bytes": 2 * table + 4 * T * k * 4 + T + 2 * T * H * size + 2 * E * H * 4, "flops": 4 * T * E * H}


# ---------------------------------------------------------------- in 64 bits ----

def exact(case, seed):
    """The gradients by differentiating the operators' definitions in 64 bits."""
    s = prepare(case, seed)
    return {"balance": _exact_balance, "distill": _exact_distill, "route": _exact_route,
            "combine": _exact_combine}[case["op"]](s)


def _exact_scores(l, score):
    """The router's distribution over the experts of each row."""
    return torch.softmax(torch.nn.functional.logsigmoid(l) if score == SIGMOID else l, dim=1)


def _exact_balance(s):
    l = s["logits"].double().requires_grad_()
    S, E, k = s["S"], s["E"], s["k"]
    off = s["seq_offsets"].tolist()
    mask = s["mask"].bool()
    balance, z, n, full = 0.0 * l[:0].sum(), 0.0 * l[:0].sum(), 0, 0
    counts, probs, tokens = [], [], []
    for a, b in zip(off[:-1], off[1:]):
        keep = torch.nonzero(mask[a:b])[:, 0] + a
        rows = l[keep]
        p = _exact_scores(rows, s["score"]).sum(0)
        picked = s["ids"][keep].reshape(-1)
        f = torch.bincount(picked[(picked >= 0) & (picked < E)].long(), minlength=E)
        m = len(keep)
        if m:
            balance = balance + E * (f.double() / (k * m) * (p / m)).sum()
            z = z + torch.logsumexp(rows, 1).square().sum()
            full += 1
        n += m
        counts.append(f.int())
        probs.append(p.detach())
        tokens.append(m)
    balance, z = balance / max(full, 1), z / max(n, 1)
    if n:
        (balance * s["d_losses"][0].double() + z * s["d_losses"][1].double()).backward()
    d = l.grad if l.grad is not None else torch.zeros_like(l)
    return {"losses": torch.stack([balance, z]).detach(), "counts": torch.stack(counts), "probs": torch.stack(probs),
            "tokens": torch.tensor(tokens + [n, full], dtype=torch.int32), "d_logits": d}


def _exact_distill(s):
    tau, E = s["temperature"], s["E"]
    l = s["logits"].double().requires_grad_()
    ok = (s["t_ids"] >= 0) & s["mask"].bool()[:, None]
    keep = torch.nonzero(ok.any(1))[:, 0]
    token_loss = torch.zeros(s["T"], dtype=torch.float64, device=DEV)
    if not len(keep):
        return {"loss": token_loss[:1] * 0, "token_loss": token_loss, "tokens": torch.zeros(1, dtype=torch.int32),
                "d_logits": torch.zeros_like(l)}
    z = (s["t_logits"][keep].double() / tau).masked_fill(~ok[keep], float("-inf"))
    q = _exact_scores(z, s["score"])
    target = torch.zeros((len(keep), E + 1), dtype=torch.float64, device=DEV)
    target.scatter_add_(1, torch.where(ok[keep], s["t_ids"][keep].long(), E), q)
    logp = torch.log(_exact_scores(l[keep] / tau, s["score"]))
    each = tau * tau * (torch.special.xlogy(q, q).sum(1) - (target[:, :E] * logp).sum(1))
    token_loss[keep] = each.detach()
    loss = each.mean()
    (loss * s["d_loss"].double()[0]).backward()
    return {"loss": loss.detach()[None], "token_loss": token_loss,
            "tokens": torch.tensor([len(keep)], dtype=torch.int32), "d_logits": l.grad}


def _exact_route(s):
    mask = s["mask"].bool()
    keep = torch.nonzero(mask)[:, 0]
    hidden, W = s["hidden"][keep].double(), s["W"].double()
    # the weights as a function of the logits of the forward pass
    l = s["logits"][keep].double().requires_grad_()
    picked = torch.sigmoid(torch.gather(l, 1, s["ids"][keep].long()))
    w = picked / picked.sum(1, keepdim=True)
    ((w * s["d_topk_w"][keep].double()).sum() + (l * s["d_aux"][keep].double()).sum()).backward()
    d = torch.zeros(s["logits"].shape, dtype=torch.float64, device=DEV)
    d[keep] = l.grad
    d_hidden = torch.zeros(s["hidden"].shape, dtype=torch.float64, device=DEV)
    d_hidden[keep] = torch.mm(l.grad, W) * s["scale"]
    return {"d_logits": d, "d_hidden": d_hidden, "d_W": torch.mm(l.grad.t().contiguous(), hidden) * s["scale"]}


def _exact_combine(s):
    T, H, k, R = s["T"], s["H"], s["k"], s["T"] * s["k"]
    norm_w = s["norm_w"].double().requires_grad_()
    topk_w = s["topk_w"].double().requires_grad_()
    d_rows = torch.zeros((R, H), dtype=torch.float64, device=DEV)
    step = max(1, (1 << 27) // (k * H))
    for t in range(0, T, step):
        slots = s["slots"][t:t + step].long()
        at = torch.nonzero(slots >= 0)
        rows = slots[at[:, 0], at[:, 1]]
        x = s["expert_out"][rows].double().requires_grad_()
        y = torch.nn.functional.rms_norm(x, (H,), norm_w + s["center"], s["eps"])
        w = topk_w[t:t + step][at[:, 0], at[:, 1]]
        (y * w[:, None] * s["d_out"][t:t + step].double()[at[:, 0]]).sum().backward()
        d_rows[rows] = x.grad
    return {"d_expert_out": d_rows, "d_topk_w": topk_w.grad, "d_norm_w": norm_w.grad}
