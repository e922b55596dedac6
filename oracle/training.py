"""Oracle for the router's training operators: the balance and z losses, the
distillation loss, and the backward passes of the route and the combine.

Definitions: include/moe_training.h. Everything is evaluated in float64 from
the inputs as they are (FP32 arrays, BF16 bits as uint16) and returned in
float64. The backward functions also return the magnitude at which their
rounding is judged: the same formula with every term's absolute value.

Test infrastructure only.
"""
from __future__ import annotations

import numpy as np

from .formats import bf16_bits_to_f64

SIGMOID, SOFTMAX = 0, 1


def _f64(a):
    a = np.asarray(a)
    return bf16_bits_to_f64(a) if a.dtype == np.uint16 else a.astype(np.float64)


def log_score(l, score):
    """log of the router's score: the logit (softmax) or log sigmoid."""
    return l if score == SOFTMAX else np.minimum(l, 0.0) - np.log1p(np.exp(-np.abs(l)))


def slope(l, score):
    """d log_score / dl."""
    if score == SOFTMAX:
        return np.ones_like(l)
    e = np.exp(-np.abs(l))
    return np.where(l > 0, e, 1.0) / (1.0 + e)


def distribution(l, score):
    """p of each row of l; zeros for a row whose every score is zero."""
    ls = log_score(l, score)
    top = ls.max(axis=1, keepdims=True)
    u = np.exp(ls - np.where(np.isfinite(top), top, 0.0))
    total = u.sum(axis=1, keepdims=True)
    return u / np.where(total > 0, total, 1.0)


def logsumexp(l):
    """log sum exp of each row; 0 for a row of -inf, which adds nothing."""
    top = l.max(axis=1, keepdims=True)
    top = np.where(top == -np.inf, 0.0, top)
    total = np.exp(l - top).sum(axis=1, keepdims=True)
    return np.where(total > 0, top + np.log(np.where(total > 0, total, 1.0)), 0.0)[:, 0]


def _members(mask, seq_offsets, T):
    """The valid tokens of each sequence."""
    off = [0, T] if seq_offsets is None else [int(o) for o in seq_offsets]
    mask = np.asarray(mask).astype(bool)
    return [np.flatnonzero(mask[a:b]) + a if a < b else np.zeros(0, np.int64) for a, b in zip(off[:-1], off[1:])]


def balance_loss(logits, topk_ids, token_mask, seq_offsets=None, score=SIGMOID):
    """Returns (losses [2], counts [S,E], probs [S,E], tokens [S+2])."""
    l = _f64(logits)
    T, E = l.shape
    ids = np.asarray(topk_ids)
    k = ids.shape[1]
    seqs = _members(token_mask, seq_offsets, T)
    S = len(seqs)
    counts, probs = np.zeros((S, E), np.int64), np.zeros((S, E))
    balance, z, n, full = 0.0, 0.0, 0, 0
    for s, rows in enumerate(seqs):
        if not len(rows):
            continue
        picked = ids[rows].reshape(-1)
        counts[s] = np.bincount(picked[(picked >= 0) & (picked < E)], minlength=E)
        probs[s] = distribution(l[rows], score).sum(axis=0)
        m = len(rows)
        balance += E * (counts[s] / (k * m) * probs[s] / m).sum()
        z += (logsumexp(l[rows]) ** 2).sum()
        n += m
        full += 1
    losses = np.array([balance / max(full, 1), z / max(n, 1)])
    return losses, counts, probs, np.array([len(r) for r in seqs] + [n, full])


def balance_loss_backward(d_losses, logits, token_mask, counts, tokens, k, seq_offsets=None, score=SIGMOID):
    """Returns (d_logits [T,E], magnitude [T,E])."""
    l = _f64(logits)
    T, E = l.shape
    g = _f64(d_losses)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    n, full = max(int(tokens[-2]), 1), max(int(tokens[-1]), 1)
    for s, rows in enumerate(_members(token_mask, seq_offsets, T)):
        if not len(rows):
            continue
        x = l[rows]
        p, sl = distribution(x, score), slope(x, score)
        m = float(tokens[s])
        c = g[0] * E * np.asarray(counts[s], np.float64)[None, :] / (k * m * m * full)
        dot, adot = (p * c).sum(1, keepdims=True), (p * np.abs(c)).sum(1, keepdims=True)
        lse = logsumexp(x)[:, None]
        soft = np.exp(x - lse)
        zg = g[1] * 2.0 / n
        d[rows] = p * sl * (c - dot) + zg * lse * soft
        mag[rows] = p * sl * (np.abs(c) + adot) + np.abs(zg) * (np.abs(lse) + 1.0) * soft
    return d, mag


def _teacher(teacher_ids, teacher_logits, token_mask, E, score, temperature):
    ids, z = np.asarray(teacher_ids).astype(np.int64), _f64(teacher_logits)
    ok = (ids >= 0) & (ids < E) & (z != -np.inf) & np.asarray(token_mask).astype(bool)[:, None]
    has = ok.any(axis=1)
    with np.errstate(invalid="ignore"):
        ls = np.where(ok, log_score(np.where(ok, z, 0.0) / temperature, score), -np.inf)
    q = np.zeros(z.shape)
    if has.any():
        top = ls[has].max(axis=1, keepdims=True)
        u = np.exp(ls[has] - top)
        q[has] = u / u.sum(axis=1, keepdims=True)
    return ids, ok, has, q


def distill_loss(logits, teacher_ids, teacher_logits, token_mask, score=SIGMOID, temperature=1.0):
    """Returns (loss, token_loss [T], tokens, magnitude [T])."""
    l = _f64(logits)
    T, E = l.shape
    ids, ok, has, q = _teacher(teacher_ids, teacher_logits, token_mask, E, score, temperature)
    loss, mag = np.zeros(T), np.zeros(T)
    rows = np.flatnonzero(has)
    if len(rows):
        with np.errstate(divide="ignore"):
            logp = np.log(distribution(l[rows] / temperature, score))
        at = np.take_along_axis(logp, np.where(ok[rows], ids[rows], 0), axis=1)
        qq = q[rows]
        with np.errstate(divide="ignore", invalid="ignore"):
            logq = np.where(qq > 0, np.log(np.where(qq > 0, qq, 1.0)), 0.0)
            term = np.where(qq > 0, qq * (logq - at), 0.0)
            big = np.where(qq > 0, qq * (np.abs(logq) + np.abs(at) + 1.0), 0.0)
        loss[rows] = temperature ** 2 * term.sum(axis=1)
        mag[rows] = temperature ** 2 * big.sum(axis=1)
    n = int(has.sum())
    return loss.sum() / max(n, 1), loss, n, mag


def distill_loss_backward(d_loss, logits, teacher_ids, teacher_logits, token_mask, tokens, score=SIGMOID,
                          temperature=1.0):
    """Returns (d_logits [T,E], magnitude [T,E])."""
    l = _f64(logits)
    T, E = l.shape
    ids, ok, has, q = _teacher(teacher_ids, teacher_logits, token_mask, E, score, temperature)
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    f = float(d_loss) * temperature / max(int(tokens), 1)
    for t in np.flatnonzero(has):
        x = l[t:t + 1] / temperature
        p, sl = distribution(x, score)[0], slope(x, score)[0]
        share = np.zeros(E)
        np.add.at(share, ids[t][ok[t]], q[t][ok[t]])
        d[t] = f * sl * (p - share)
        mag[t] = abs(f) * sl * (p + share)
    return d, mag


def route_backward(d_topk_w, hidden, W, logits, topk_ids, topk_w, token_mask, scale=1.0, d_aux=None):
    """Returns ((d_logits, d_hidden, d_W), (their magnitudes)); d_hidden and
    d_W are None without hidden."""
    valid = np.asarray(token_mask).astype(bool)
    T = len(valid)
    E = (np.asarray(d_aux) if d_topk_w is None else np.asarray(logits)).shape[1]
    d, mag = np.zeros((T, E)), np.zeros((T, E))
    if d_aux is not None:
        d[valid] = _f64(d_aux)[valid]
        mag[valid] = np.abs(d[valid])
    if d_topk_w is not None:
        ids = np.asarray(topk_ids).astype(np.int64)
        for t in np.flatnonzero(valid):
            ok = (ids[t] >= 0) & (ids[t] < E)
            i = ids[t][ok]
            w, dw = _f64(topk_w)[t][ok], _f64(d_topk_w)[t][ok]
            one_minus = 1.0 / (1.0 + np.exp(_f64(logits[t])[i]))
            np.add.at(d[t], i, w * one_minus * (dw - (w * dw).sum()))
            np.add.at(mag[t], i, w * one_minus * (np.abs(dw) + np.abs(w * dw).sum()))
    if hidden is None:
        return (d, None, None), (mag, None, None)
    h = np.zeros(np.asarray(hidden).shape)
    h[valid] = _f64(np.asarray(hidden)[valid])
    w64 = _f64(W)
    s = float(np.float32(scale))
    return ((d, s * (d @ w64), s * (d.T @ h)),
            (mag, abs(s) * (mag @ np.abs(w64)), abs(s) * (mag.T @ np.abs(h))))


def combine_backward(d_out, expert_out, slots, topk_w, norm_w, gain_center, eps, rows=None):
    """Returns ((d_expert_out [R,H], d_topk_w [T,k], d_norm_w [H]), (their
    magnitudes)). Rows that no slot names are not read."""
    R = expert_out.shape[0] if rows is None else rows
    slots = np.asarray(slots).astype(np.int64)
    T, k = slots.shape
    H = np.asarray(norm_w).shape[0]
    y = _f64(d_out)
    w = _f64(topk_w)
    gain = (np.float32(gain_center) + np.asarray(norm_w, np.float32)).astype(np.float64)
    e = float(np.float32(eps))
    dx, mx = np.zeros((R, H)), np.zeros((R, H))
    dw, mw = np.zeros((T, k)), np.zeros((T, k))
    dn, mn = np.zeros(H), np.zeros(H)
    for j in range(k):
        r = slots[:, j]
        t = np.flatnonzero((r >= 0) & (r < R))
        if not len(t):
            continue
        x = _f64(expert_out[r[t]])
        rstd = 1.0 / np.sqrt((x * x).mean(axis=1, keepdims=True) + e)
        gy = gain * y[t]
        a = (gy * x).sum(axis=1, keepdims=True)
        aa = np.abs(gy * x).sum(axis=1, keepdims=True)
        c = w[t, j][:, None] * rstd
        np.add.at(dx, r[t], c * (gy - x * rstd ** 2 * a / H))
        np.add.at(mx, r[t], np.abs(c) * (np.abs(gy) + np.abs(x) * rstd ** 2 * aa / H))
        dw[t, j] = (rstd * a)[:, 0]
        mw[t, j] = (rstd * aa)[:, 0]
        dn += (c * x * y[t]).sum(axis=0)
        mn += np.abs(c * x * y[t]).sum(axis=0)
    return (dx, dw, dn), (mx, mw, mn)
