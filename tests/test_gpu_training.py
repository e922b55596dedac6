"""The router's training operators against the float64 oracle: sizes from one
token up, odd widths, ragged and empty sequences, masked NaN, repeated and
invalid entries, reused workspaces, graph replay on a side stream, and one
training step's chain of calls.

Tolerances count roundings of 2^-24 (half a step of FP32) at the magnitude of
the sum they happen in:
  * a probability: exp(x) from exp2(x log2 e) is off by |x| 2^-24 for the
    product and 2^-23 for exp2, the row's sum of E terms adds E/64 + 6
    roundings, the reciprocals a few more: P(X, E) = (X + E/64 + 24) 2^-23 with
    X the row's largest |logit - maximum|;
  * a matrix product over K: one rounding per MFMA step and plane product and
    the sums of the splits, (6 K/16 + 64) 2^-24, and the dropped plane
    products: 3 x 2^-24 (two planes for a BF16 result: 3 x 2^-17);
  * a BF16 result: 2^-8 of it (half a step).
"""
import numpy as np
import pytest
import torch

import oracle as O
from oracle import training as OT
import workloads as wl
from gpu_helpers import DEV, dev, host, note, require_gpu

pytestmark = pytest.mark.gpu

m = pytest.importorskip("moe_token_routing_amd")

U = 2.0 ** -24


def _close(got, want, tol, what):
    got = got.astype(np.float64) if got.dtype != np.uint16 else O.bf16_bits_to_f64(got)
    want, tol = np.broadcast_arrays(np.asarray(want, np.float64), np.asarray(tol, np.float64))
    assert got.shape == want.shape, what
    bad = ~(np.abs(got - want) <= tol)
    if bad.any():
        i = tuple(np.argwhere(bad)[0])
        raise AssertionError("%s: %d of %d off, first at %s: got %r want %r tolerance %r" % (
            what, int(bad.sum()), bad.size, i, got[i], want[i], tol[i]))


def _prob_tol(l, mask, E):
    """P(X, E) of the widest valid row."""
    rows = l[np.asarray(mask) != 0].astype(np.float64)
    rows = np.where(np.isfinite(rows), rows, 0.0)
    X = float((rows.max(1) - rows.min(1)).max() + np.abs(rows).max()) if len(rows) else 0.0
    return (X + E / 64 + 24) * 2 * U


def _mask(g, T, frac=0.1):
    mask = (g.uniform(size=T) >= frac).astype(np.uint8)
    if T < 8:
        mask[:] = 1
    return mask


def _logits(g, T, E, mask, spread=1.0, shift=0.0):
    l = (g.standard_normal((T, E)) * spread + g.standard_normal((1, E)) * 0.5 + shift).astype(np.float32)
    l[mask == 0] = np.nan
    return l


def _ids(g, T, E, k, mask):
    ids = np.argsort(g.uniform(size=(T, E)), axis=1)[:, :k].astype(np.int32)
    ids[mask == 0] = -1
    return ids


def _cut(g, T, S):
    off = np.sort(g.integers(0, T + 1, S + 1)).astype(np.int32)
    return off


# ------------------------------------------------------------- balance ----

def _check_balance(g, T, E, k, S, score, spread=1.0, shift=0.0, d_losses=(0.5, 0.25)):
    require_gpu()
    note("balance T=%d E=%d k=%d S=%s score=%d" % (T, E, k, S, score))
    mask = _mask(g, T)
    l = _logits(g, T, E, mask, spread, shift)
    ids = _ids(g, T, E, k, mask)
    if T > 2 and k > 1:
        ids[1, 0] = E          # counts nowhere
    off = None if S is None else _cut(g, T, S)
    with np.errstate(invalid="ignore"):
        ref = OT.balance_loss(l, ids, mask, off, score)
    l_d, ids_d, mask_d = dev(l), dev(ids), dev(mask)
    off_d = None if off is None else dev(off)
    losses, counts, probs, tokens = m.balance_loss(l_d, ids_d, mask_d, score=score, seq_offsets=off_d)
    np.testing.assert_array_equal(host(counts), ref[1], err_msg="counts")
    np.testing.assert_array_equal(host(tokens), ref[3], err_msg="tokens")
    P = _prob_tol(l, mask, E)
    # at most 16 tokens a wave, 4 waves, T/16 / 16 + 16 rows of partial sums
    sums = (40 + T / 256) * U
    _close(host(probs), ref[2], (P + sums) * ref[2] + 1e-37, "probs")
    lse = np.sqrt(max(ref[0][1], 0.0))
    # losses[1]: lse is off by P and by 2 roundings of itself, and enters squared
    _close(host(losses), ref[0], [(P + sums + 16 * U) * ref[0][0],
                                  2 * (lse + 1) * (P + 4 * U * (lse + 1)) + sums * ref[0][1]], "losses")
    g_l = np.array(d_losses, np.float32)
    d = m.balance_loss_backward(dev(g_l), l_d, mask_d, counts, tokens, k, score=score, seq_offsets=off_d)
    with np.errstate(invalid="ignore"):
        want, mag = OT.balance_loss_backward(g_l, l, mask, ref[1], ref[3], k, off, score)
    tol = 4 * P * mag + 1e-37
    _close(host(d), want, tol, "d_logits")
    # accumulate: added to what is there, rows of invalid tokens untouched
    base = g.standard_normal((T, E)).astype(np.float32) * np.float32(np.abs(want).max() + 1e-3)
    base[mask == 0] = np.nan
    acc = dev(base)
    m.balance_loss_backward(dev(g_l), l_d, mask_d, counts, tokens, k, score=score, seq_offsets=off_d, d_logits=acc,
                            accumulate=True)
    got = host(acc)
    assert np.isnan(got[mask == 0]).all()
    v = mask != 0
    _close(got[v], base[v].astype(np.float64) + want[v], tol[v] + U * np.abs(base[v].astype(np.float64) + want[v]) * 2,
           "d_logits accumulated")


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
@pytest.mark.parametrize("T,E,k,S", [(1, 1, 1, None), (1, 64, 4, 1), (3, 5, 2, 3), (16, 16, 4, None), (65, 254, 8, 7),
                                     (200, 257, 3, 66), (333, 1001, 8, 5), (130, 2560, 8, 2), (70, 4096, 32, None),
                                     (67, 4095, 2, 3), (2000, 256, 8, 130), (4500, 33, 4, 3), (50, 1500, 5, 2),
                                     (50, 2000, 5, 2), (50, 700, 5, 2), (40, 1024, 8, 3), (64, 1023, 8, 60),
                                     (66000, 9, 2, 4), (32, 1024, 8, 4), (29, 600, 5, 2), (33, 1024, 8, 4)])
def test_balance(T, E, k, S, score):
    _check_balance(np.random.default_rng(T * 7 + E), T, E, k, S, score)


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
def test_balance_far_logits(score):
    """Logits whose sigmoids all underflow, or whose exponentials overflow:
    the distribution is still that of the definition."""
    g = np.random.default_rng(11)
    _check_balance(g, 40, 48, 4, 2, score, shift=-200.0)
    _check_balance(g, 40, 48, 4, 2, score, shift=300.0)
    _check_balance(g, 40, 48, 4, 2, score, spread=20.0)


def test_balance_only_one_of_the_losses():
    g = np.random.default_rng(12)
    _check_balance(g, 100, 96, 4, 3, OT.SIGMOID, d_losses=(1.0, 0.0))
    _check_balance(g, 100, 96, 4, 3, OT.SIGMOID, d_losses=(0.0, 1.0))


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
def test_balance_masked_experts(score):
    """Experts masked by -inf logits get no probability and no gradient; a row
    of -inf is zero throughout the balance loss."""
    require_gpu()
    g = np.random.default_rng(13)
    T, E, k = 30, 40, 4
    l = g.standard_normal((T, E)).astype(np.float32)
    l[:, ::3] = -np.inf
    ids = _ids(g, T, E, k, np.ones(T))
    mask = np.ones(T, np.uint8)
    ref = OT.balance_loss(l, ids, mask, None, score)
    losses, counts, probs, tokens = m.balance_loss(dev(l), dev(ids), dev(mask), score=score)
    P = (20 + 24) * 2 * U
    _close(host(probs), ref[2], 2 * P * ref[2], "probs")
    assert (host(probs)[:, ::3] == 0).all()
    gl = np.array([1.0, 1.0], np.float32)
    d = host(m.balance_loss_backward(dev(gl), dev(l), dev(mask), counts, tokens, k, score=score))
    want, mag = OT.balance_loss_backward(gl, l, mask, ref[1], ref[3], k, None, score)
    _close(d, want, 4 * P * mag, "d_logits")
    l[5] = -np.inf
    losses, counts, probs, tokens = m.balance_loss(dev(l), dev(ids), dev(mask), score=score)
    assert np.isfinite(host(probs)).all() and np.isfinite(host(losses)[0])


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
@pytest.mark.parametrize("T,E", [(30, 40), (90, 300), (70, 1500)])
def test_losses_of_rows_without_an_expert(T, E, score):
    """Rows whose every logit is -inf: p = 0, nothing in the balance and z
    losses and no gradient of them; the distillation loss is infinite there,
    its gradient finite."""
    require_gpu()
    note("losses, rows of -inf, T=%d E=%d" % (T, E))
    g = np.random.default_rng(16)
    k = 4
    mask = np.ones(T, np.uint8)
    l = g.standard_normal((T, E)).astype(np.float32)
    l[5:T:7] = -np.inf
    ids = _ids(g, T, E, k, mask)
    off = np.array([0, 5, 6, T], np.int32)   # the second sequence has such a row alone
    ref = OT.balance_loss(l, ids, mask, off, score)
    losses, counts, probs, tokens = m.balance_loss(dev(l), dev(ids), dev(mask), score=score, seq_offsets=dev(off))
    P = _prob_tol(l, mask, E)
    _close(host(probs), ref[2], (P + 40 * U) * ref[2], "probs")
    lse = np.sqrt(ref[0][1])
    _close(host(losses), ref[0], [(P + 56 * U) * ref[0][0], 2 * (lse + 1) * (P + 4 * U * (lse + 1)) + 40 * U * ref[0][1]],
           "losses")
    gl = np.array([1.0, 1.0], np.float32)
    d = host(m.balance_loss_backward(dev(gl), dev(l), dev(mask), counts, tokens, k, score=score, seq_offsets=dev(off)))
    want, mag = OT.balance_loss_backward(gl, l, mask, ref[1], ref[3], k, off, score)
    _close(d, want, 4 * P * mag, "d_logits")
    assert (d[5:T:7] == 0).all()
    z = g.standard_normal((T, k)).astype(np.float32)
    loss, each, n = m.distill_loss(dev(l), dev(ids), dev(z), dev(mask), score=score)
    assert np.isposinf(host(each)[5:T:7]).all() and np.isposinf(host(loss)[0]) and int(host(n)[0]) == T
    assert np.isfinite(np.delete(host(each), np.arange(5, T, 7))).all()
    d = host(m.distill_loss_backward(dev(np.ones(1, np.float32)), dev(l), dev(ids), dev(z), dev(mask), n, score=score))
    want, mag = OT.distill_loss_backward(1.0, l, ids, z, mask, T, score)
    _close(d, want, 3 * (P + _prob_tol(z, mask, E)) * mag + 1e-37, "distillation d_logits")


def test_balance_without_tokens():
    require_gpu()
    E, S = 24, 3
    l = torch.empty((0, E), dtype=torch.float32, device=DEV)
    ids = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    mask = torch.empty(0, dtype=torch.uint8, device=DEV)
    off = torch.zeros(S + 1, dtype=torch.int32, device=DEV)
    for t in m.balance_loss(l, ids, mask, seq_offsets=off):
        assert (host(t) == 0).all()
    # tokens, all invalid, in rows of NaN
    T = 9
    l = torch.full((T, E), float("nan"), device=DEV)
    ids = torch.full((T, 2), 3, dtype=torch.int32, device=DEV)
    mask = torch.zeros(T, dtype=torch.uint8, device=DEV)
    losses, counts, probs, tokens = m.balance_loss(l, ids, mask)
    for t in (losses, counts, probs, tokens):
        assert (host(t) == 0).all()
    d = m.balance_loss_backward(torch.ones(2, device=DEV), l, mask, counts, tokens, 2)
    assert (host(d) == 0).all()


def test_balance_offsets_out_of_range_are_clamped():
    require_gpu()
    g = np.random.default_rng(14)
    T, E, k = 50, 32, 4
    mask = np.ones(T, np.uint8)
    l, ids = _logits(g, T, E, mask), _ids(g, T, E, k, mask)
    got = m.balance_loss(dev(l), dev(ids), dev(mask), seq_offsets=dev(np.array([-5, 20, 2 ** 31 - 1], np.int32)))
    want = m.balance_loss(dev(l), dev(ids), dev(mask), seq_offsets=dev(np.array([0, 20, T], np.int32)))
    for a, b in zip(got, want):
        assert torch.equal(a, b)


def test_balance_sums_of_parts_are_the_whole():
    """Counts, probabilities and tokens of two halves add up to the batch's,
    and the backward pass with the sums is the batch's."""
    require_gpu()
    g = np.random.default_rng(15)
    T, E, k = 120, 64, 4
    mask = _mask(g, T)
    l, ids = _logits(g, T, E, mask), _ids(g, T, E, k, mask)
    whole = m.balance_loss(dev(l), dev(ids), dev(mask))
    halves = [m.balance_loss(dev(l[a:b]), dev(ids[a:b]), dev(mask[a:b])) for a, b in ((0, 48), (48, T))]
    counts = halves[0][1] + halves[1][1]
    tokens = halves[0][3] + halves[1][3]
    tokens[-1] = 1   # sequences with a token: the same one
    assert torch.equal(counts, whole[1]) and torch.equal(tokens, whole[3])
    gl = torch.tensor([1.0, 1.0], device=DEV)
    d = m.balance_loss_backward(gl, dev(l), dev(mask), whole[1], whole[3], k)
    part = m.balance_loss_backward(gl, dev(l[48:]), dev(mask[48:]), counts, tokens, k)
    assert torch.equal(d[48:], part)


# ------------------------------------------------------------- distill ----

def _teacher(g, l, K):
    T, E = l.shape
    z = np.where(np.isnan(l), 0.0, l).astype(np.float32) + g.standard_normal((T, E)).astype(np.float32)
    ids = np.argsort(-z, axis=1)[:, :K]
    if K > E:
        ids = np.concatenate([ids, np.full((T, K - E), -1)], axis=1)
    t = np.take_along_axis(z, np.maximum(ids, 0), axis=1).astype(np.float32)
    return ids.astype(np.int32), t


def _check_distill(g, T, E, K, score, temperature, edit=None, spread=1.0, shift=0.0):
    require_gpu()
    note("distill T=%d E=%d K=%d score=%d temperature=%g" % (T, E, K, score, temperature))
    mask = _mask(g, T)
    l = _logits(g, T, E, mask, spread, shift)
    ids, z = _teacher(g, l, K)
    if edit:
        edit(ids, z, E)
    with np.errstate(invalid="ignore"):
        loss, each, n, mag = OT.distill_loss(l, ids, z, mask, score, temperature)
    args = (dev(l), dev(ids), dev(z), dev(mask))
    got = m.distill_loss(*args, score=score, temperature=temperature)
    assert int(host(got[2])[0]) == n
    P = _prob_tol(l / temperature, mask, E) + _prob_tol(np.where(ids >= 0, z, 0) / temperature, mask, E)
    tol = 2 * P * mag + 1e-37
    _close(host(got[1]), each, tol, "token_loss")
    _close(host(got[0]), [loss], [tol.sum() / max(n, 1) + 32 * U * np.abs(each).sum() / max(n, 1)], "loss")
    d = m.distill_loss_backward(dev(np.array([0.5], np.float32)), *args, got[2], score=score, temperature=temperature)
    with np.errstate(invalid="ignore"):
        want, dmag = OT.distill_loss_backward(0.5, l, ids, z, mask, n, score, temperature)
    dtol = 3 * P * dmag + 1e-37
    _close(host(d), want, dtol, "d_logits")
    base = g.standard_normal((T, E)).astype(np.float32) * 1e-3
    acc = dev(base)
    m.distill_loss_backward(dev(np.array([0.5], np.float32)), *args, got[2], score=score, temperature=temperature,
                            d_logits=acc, accumulate=True)
    _close(host(acc), base.astype(np.float64) + want, dtol + 2 * U * np.abs(base.astype(np.float64) + want),
           "d_logits accumulated")


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
@pytest.mark.parametrize("T,E,K,temperature", [(1, 1, 1, 1.0), (1, 64, 4, 1.0), (5, 7, 7, 0.5), (16, 16, 4, 2.0),
                                               (300, 254, 8, 1.0), (131, 1001, 31, 4.0), (70, 2560, 8, 2.0),
                                               (41, 4096, 32, 1.0), (33, 4093, 5, 0.7), (4200, 40, 3, 1.0),
                                               (9, 5, 12, 1.0), (50, 1500, 5, 2.0), (50, 2000, 5, 1.0),
                                               (50, 700, 5, 2.0), (50, 400, 5, 2.0), (132000, 6, 3, 1.0), (32, 1000, 8, 1.0), (33, 900, 4, 1.0)])
def test_distill(T, E, K, temperature, score):
    _check_distill(np.random.default_rng(T + E + K), T, E, K, score, temperature)


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
def test_distill_entries_missing_repeated_and_out_of_range(score):
    def edit(ids, z, E):
        ids[0] = -1
        ids[1, 1:] = -1
        ids[2, 0] = E
        ids[3, 0] = 2 ** 31 - 1
        ids[4, 3] = ids[4, 0]            # named twice
        ids[5, :] = ids[5, 0]            # and by every entry
        z[6, 1] = -np.inf
        z[7, :] = -np.inf
        z[8, 0] = 90.0                   # all but all of the weight

    _check_distill(np.random.default_rng(21), 64, 96, 6, score, 1.5, edit)


def test_distill_far_logits():
    for score in (OT.SIGMOID, OT.SOFTMAX):
        _check_distill(np.random.default_rng(22), 32, 64, 6, score, 1.0, shift=-150.0)
        _check_distill(np.random.default_rng(23), 32, 64, 6, score, 1.0, shift=150.0)


def test_distill_no_entry_at_all():
    require_gpu()
    T, E, K = 6, 32, 3
    l = torch.full((T, E), float("nan"), device=DEV)
    z = torch.full((T, K), float("nan"), device=DEV)
    mask = torch.ones(T, dtype=torch.uint8, device=DEV)
    for ids, mk in ((torch.full((T, K), -1, dtype=torch.int32, device=DEV), mask),
                    (torch.zeros((T, K), dtype=torch.int32, device=DEV), torch.zeros_like(mask))):
        loss, each, n = m.distill_loss(l, ids, z, mk)
        d = m.distill_loss_backward(torch.ones(1, device=DEV), l, ids, z, mk, n)
        for t in (loss, each, n, d):
            assert (host(t) == 0).all()
    empty = m.distill_loss(l[:0], torch.zeros((0, K), dtype=torch.int32, device=DEV), z[:0], mask[:0])
    assert float(empty[0]) == 0 and int(empty[2]) == 0


# --------------------------------------------------------------- route ----

def _check_route(g, T, H, E, k, f32, aux=True, weights=True, scale=0.75, dup=False):
    require_gpu()
    note("route backward T=%d H=%d E=%d k=%d %s" % (T, H, E, k, "f32" if f32 else "bf16"))
    mask = _mask(g, T)
    l = _logits(g, T, E, mask)
    ids = _ids(g, T, E, k, mask)
    if dup and k > 1:
        ids[0, 1] = ids[0, 0]
        ids[min(2, T - 1), 0] = E + 3     # drops out
    s = 1 / (1 + np.exp(-np.take_along_axis(np.nan_to_num(l), np.clip(ids, 0, E - 1).astype(np.int64), 1)))
    w = (s / s.sum(1, keepdims=True)).astype(np.float32)
    dw = g.standard_normal((T, k)).astype(np.float32)
    da = (g.standard_normal((T, E)) * 1e-2).astype(np.float32) if aux else None
    if aux:
        da[mask == 0] = np.nan
    h = g.standard_normal((T, H)).astype(np.float32)
    h[mask == 0] = np.nan
    h = h if f32 else wl.f32_to_bf16_bits(h)
    if not f32:
        h[mask == 0] = wl.BF16_NAN
    W = (g.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32)
    got = m.route_backward(dev(dw) if weights else None, dev(h), dev(W), dev(l), dev(ids), dev(w), dev(mask), scale,
                           d_aux=None if da is None else dev(da))
    want, mag = OT.route_backward(dw if weights else None, h, W, l, ids, w, mask, scale, da)
    _close(host(got[0]), want[0], (k + 12) * 2 * U * mag[0] + 1e-40, "d_logits")
    # a value below 2^-100 loses its low planes; nothing here is that small
    chain = lambda K: (6 * K / 16 + 64 + (k + 12) * 2) * U
    if f32:
        _close(host(got[1]), want[1], (chain(E) + 3 * U) * mag[1], "d_hidden")
    else:
        _close(host(got[1]), want[1], (chain(E) + 3 * 2.0 ** -17) * mag[1] + 2.0 ** -8 * np.abs(want[1]), "d_hidden")
    _close(host(got[2]), want[2], (chain(T) + 3 * U) * mag[2], "d_W")


@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("T,H,E,k", [(1, 16, 1, 1), (1, 256, 64, 4), (16, 256, 16, 4), (33, 272, 130, 8),
                                     (65, 1040, 257, 3), (2, 144, 4000, 7), (5, 8192, 392, 29),
                                     (8, 48, 1000, 32), (31, 528, 500, 11), (32, 2064, 600, 8), (300, 512, 256, 8), (129, 144, 1000, 32), (1000, 528, 40, 4),
                                     (515, 2064, 96, 8)])
def test_route_backward(T, H, E, k, f32):
    _check_route(np.random.default_rng(T + H + E), T, H, E, k, f32)


def test_route_backward_splits_over_tokens():
    """Enough tokens that the weight's gradient is summed in splits."""
    _check_route(np.random.default_rng(31), 5000, 512, 64, 4, False)
    _check_route(np.random.default_rng(32), 3000, 256, 300, 8, True)


@pytest.mark.parametrize("T,f32", [(4200, False), (2100, True)])
def test_route_backward_more_tiles_than_blocks(T, f32):
    """Blocks of the products that take several tiles, whole ones and the
    matrix' edges: 17 x 17 of them."""
    _check_route(np.random.default_rng(37), T, 4112, 40, 4, f32)


def test_route_backward_one_source_only():
    for f32 in (False, True):
        _check_route(np.random.default_rng(33), 70, 64, 48, 4, f32, aux=False)
        _check_route(np.random.default_rng(34), 70, 64, 48, 4, f32, weights=False)


def test_route_backward_repeated_and_dropped_picks():
    _check_route(np.random.default_rng(35), 40, 64, 200, 6, False, dup=True)


@pytest.mark.parametrize("T", [20, 200])
def test_route_backward_parts_and_in_place(T):
    """Logits-in mode, either gradient alone, and d_logits written over d_aux
    give the same values as the whole call."""
    require_gpu()
    g = np.random.default_rng(36)
    H, E, k = 128, 96, 4
    mask = _mask(g, T)
    l, ids = _logits(g, T, E, mask), _ids(g, T, E, k, mask)
    w = np.full((T, k), 1 / k, np.float32)
    dw, da = g.standard_normal((T, k)).astype(np.float32), g.standard_normal((T, E)).astype(np.float32)
    h = wl.f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32))
    W = g.standard_normal((E, H)).astype(np.float32)
    rest = (dev(l), dev(ids), dev(w), dev(mask), 1.0)
    whole = m.route_backward(dev(dw), dev(h), dev(W), *rest, d_aux=dev(da))
    one = m.route_backward(dev(dw), None, None, *rest, d_aux=dev(da))
    assert torch.equal(one[0], whole[0]) and one[1] is None and one[2] is None
    h_only = m.route_backward(dev(dw), dev(h), dev(W), *rest, d_aux=dev(da), need_W=False)
    w_only = m.route_backward(dev(dw), dev(h), None, *rest, d_aux=dev(da), need_hidden=False)
    assert torch.equal(h_only[1], whole[1]) and h_only[2] is None
    assert torch.equal(w_only[2], whole[2]) and w_only[1] is None
    buf = dev(da)
    out = m.route_backward(dev(dw), dev(h), dev(W), *rest, d_aux=buf, d_logits=buf)
    for a, b in zip(out, whole):
        assert torch.equal(a, b)


@pytest.mark.parametrize("T,f32", [(7, False), (30, True), (100, False), (300, False), (300, True)])
def test_route_backward_invalid_rows_beside_a_diverged_weight(T, f32):
    """Invalid tokens' gradients are zeros whatever the weight holds."""
    require_gpu()
    note("route backward, weight with infinities, T=%d" % T)
    g = np.random.default_rng(36 + T)
    H, E, k = 272, 40, 3
    mask = (g.uniform(size=T) >= 0.4).astype(np.uint8)
    mask[:3] = [0, 1, 0]
    l, ids = _logits(g, T, E, mask), _ids(g, T, E, k, mask)
    h = g.standard_normal((T, H)).astype(np.float32)
    h = h if f32 else wl.f32_to_bf16_bits(h)
    W = g.standard_normal((E, H)).astype(np.float32)
    W[4], W[7, ::2] = np.inf, np.nan
    w = np.full((T, k), 1 / k, np.float32)
    _, d_h, d_W = m.route_backward(dev(g.standard_normal((T, k)).astype(np.float32)), dev(h), dev(W), dev(l), dev(ids),
                                   dev(w), dev(mask))
    d_h = d_h.float().cpu().numpy()
    assert (d_h[mask == 0] == 0).all() and np.isnan(d_h[mask != 0]).any()
    assert np.isfinite(host(d_W)).all()


def test_route_backward_without_tokens():
    require_gpu()
    e = lambda *s: torch.empty(s, dtype=torch.float32, device=DEV)
    ids = torch.empty((0, 2), dtype=torch.int32, device=DEV)
    dl, dh, dW = m.route_backward(e(0, 2), e(0, 32), e(8, 32), e(0, 8), ids, e(0, 2),
                                  torch.empty(0, dtype=torch.uint8, device=DEV))
    assert dl.shape == (0, 8) and dh.shape == (0, 32) and (host(dW) == 0).all()
    # tokens, all invalid
    T = 5
    nan = lambda *s: torch.full(s, float("nan"), device=DEV)
    mask = torch.zeros(T, dtype=torch.uint8, device=DEV)
    out = m.route_backward(nan(T, 2), nan(T, 32).bfloat16(), torch.ones((8, 32), device=DEV), nan(T, 8),
                           torch.zeros((T, 2), dtype=torch.int32, device=DEV), nan(T, 2), mask, d_aux=nan(T, 8))
    for t in out:
        assert (t.float().cpu().numpy() == 0).all()


# ------------------------------------------------------------- combine ----

def _check_combine(g, T, H, k, center=0.0, eps=1e-6, R=None, slots=None, what=""):
    require_gpu()
    R = T * k + 3 if R is None else R
    note("combine backward T=%d H=%d k=%d R=%d %s" % (T, H, k, R, what))
    if slots is None:
        slots = g.permutation(max(R, T * k))[:T * k].astype(np.int32).reshape(T, k)
        slots[g.uniform(size=(T, k)) < 0.1] = -1
        if T > 3:
            slots[1] = -1
            slots[2, -1] = R + 5
    x = wl.f32_to_bf16_bits((g.standard_normal((R, H)) * g.uniform(0.1, 4, (R, 1))).astype(np.float32))
    unnamed = np.setdiff1d(np.arange(R), slots[(slots >= 0) & (slots < R)])
    x[unnamed] = wl.BF16_NAN
    y = wl.f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32))
    w = g.uniform(0.01, 0.5, (T, k)).astype(np.float32)
    nw = g.uniform(-0.5, 0.5, H).astype(np.float32)
    got = m.combine_backward(dev(y), dev(x), dev(slots), dev(w), dev(nw), center, eps)
    want, mag = OT.combine_backward(y, x, slots, w, nw, center, eps)
    # sums over a row: 32 values a thread, the wave's 6 exchanges and up to 8
    # waves; the formula's other steps. Slots of one row add a rounding each.
    named = max(int(np.bincount(slots[(slots >= 0) & (slots < R)], minlength=1).max()), 1) if R else 1
    row = (64 + 2 * named + H / 64 * (named > 1)) * 2 * U
    _close(host(got[0]), want[0], row * mag[0] + 2.0 ** -8 * np.abs(want[0]) + 2.0 ** -133, "d_expert_out")
    assert (host(got[0])[unnamed] == 0).all()
    _close(host(got[1]), want[1], row * mag[1], "d_topk_w")
    assert (host(got[1])[(slots < 0) | (slots >= R)] == 0).all()
    # each slot, then a block's tokens, then up to 512 blocks in 32 groups
    _close(host(got[2]), want[2], (row + (k + T / 64 + 64) * 2 * U) * mag[2], "d_norm_w")


@pytest.mark.parametrize("H", [8, 24, 256, 264, 512, 520, 1000, 1024, 1032, 1536, 2048, 2056, 4104, 6144, 8192, 8200,
                               12296, 16384])
def test_combine_backward_widths(H):
    _check_combine(np.random.default_rng(H), 19, H, 5, center=1.0)


@pytest.mark.parametrize("T,H,k", [(1, 64, 1), (1, 8192, 8), (2, 1024, 32), (16, 256, 4), (700, 1024, 22),
                                   (1500, 16, 3), (600, 2304, 2), (530, 4096, 9), (1100, 4104, 3),
                                   (5000, 520, 2), (70000, 16, 2), (600, 16384, 1), (1, 16, 32), (5, 56, 25),
                                   (3, 1032, 31), (100, 520, 13), (90, 4104, 9), (20, 8200, 7), (255, 2048, 6)])
def test_combine_backward_tokens(T, H, k):
    _check_combine(np.random.default_rng(T + H), T, H, k)


@pytest.mark.parametrize("T,H,k", [(37, 200, 4), (9, 2048, 3), (70, 16, 8), (12, 8192, 2)])
def test_combine_backward_rows_named_more_than_once(T, H, k):
    g = np.random.default_rng(41 + T)
    R = T * k
    slots = g.integers(-1, R // 3 + 1, (T, k)).astype(np.int32)
    slots[0, :] = slots[0, 0]
    _check_combine(g, T, H, k, slots=slots, R=R, what="repeated")
    _check_combine(g, T, H, k, slots=np.zeros((T, k), np.int32), R=3, what="one row")


@pytest.mark.parametrize("H", [64, 512, 1024, 2048, 4096, 8192])
def test_combine_backward_tokens_without_a_slot(H):
    """The output's gradient of tokens whose slots are all invalid is padding:
    whatever it and their weights hold, nothing of them reaches a result."""
    require_gpu()
    note("combine backward, padded tokens, H=%d" % H)
    g = np.random.default_rng(43 + H)
    T, k = 13, 3
    slots = np.arange(T * k, dtype=np.int32).reshape(T, k)
    slots[::3] = [-1, T * k, -7]
    x = wl.f32_to_bf16_bits(g.standard_normal((T * k, H)).astype(np.float32))
    y = wl.f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32))
    w = g.uniform(0.01, 0.5, (T, k)).astype(np.float32)
    nw = g.uniform(-0.5, 0.5, H).astype(np.float32)
    want = m.combine_backward(dev(y), dev(x), dev(slots), dev(w), dev(nw), 1.0, 1e-6)
    y[::3], w[::3] = wl.BF16_NAN, np.inf
    got = m.combine_backward(dev(y), dev(x), dev(slots), dev(w), dev(nw), 1.0, 1e-6)
    for a, b in zip(got, want):
        assert torch.isfinite(b.float()).all() and torch.equal(a, b)


def test_combine_backward_zero_sizes():
    require_gpu()
    bf = lambda *s: torch.full(s, float("nan"), dtype=torch.bfloat16, device=DEV)
    nw = torch.ones(64, device=DEV)
    # no token: every row's gradient and the gain's are zero
    dx, dw, dn = m.combine_backward(bf(0, 64), bf(5, 64), torch.empty((0, 2), dtype=torch.int32, device=DEV),
                                    torch.empty((0, 2), device=DEV), nw, 0.0, 1e-6)
    assert (dx.float().cpu().numpy() == 0).all() and dw.shape == (0, 2) and (host(dn) == 0).all()
    # no row: every slot is invalid
    y = torch.ones((3, 64), dtype=torch.bfloat16, device=DEV)
    dx, dw, dn = m.combine_backward(y, bf(0, 64), torch.full((3, 2), 7, dtype=torch.int32, device=DEV),
                                    torch.ones((3, 2), device=DEV), nw, 0.0, 1e-6)
    assert dx.shape == (0, 64) and (host(dw) == 0).all() and (host(dn) == 0).all()
    # rows limits what a slot may address
    x = torch.ones((6, 64), dtype=torch.bfloat16, device=DEV)
    slots = torch.tensor([[0, 4], [1, 2]], dtype=torch.int32, device=DEV)
    w = torch.ones((2, 2), device=DEV)
    dx, dw, dn = m.combine_backward(y[:2], x, slots, w, nw, 0.0, 1e-6, rows=3, need_norm_w=False)
    assert dx.shape == (3, 64) and dn is None and float(dw[0, 1]) == 0.0


# ---------------------------------------------------- streams, graphs, chain ----

def _step_inputs(g, T, H, E, k, mask):
    h = wl.f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32))
    h[mask == 0] = wl.BF16_NAN
    return dict(hidden=h, W=(g.standard_normal((E, H)) / np.sqrt(H)).astype(np.float32),
                bias=g.uniform(-0.05, 0.05, E).astype(np.float32), mask=mask,
                teacher=(g.standard_normal((T, E))).astype(np.float32),
                eo=wl.f32_to_bf16_bits(g.standard_normal((T * k, H)).astype(np.float32)),
                nw=g.uniform(0.5, 1.5, H).astype(np.float32),
                y=wl.f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32)))


def _step(d, k, E, off, gl, gd):
    """One training step's routing: forward, the losses, and every gradient."""
    lg, ids, tw, counts, offsets, perm, dest = m.route_dispatch(d["hidden"], d["W"], d["bias"], d["mask"], k)
    out = m.combine(d["eo"], dest.view(-1, k), tw, d["nw"], 0.0, 1e-6)
    _, t_ids, _ = m.route(None, None, d["bias"], d["mask"], k, logits=d["teacher"])
    t_logits = torch.gather(d["teacher"], 1, t_ids.long().clamp(min=0))
    losses, cnt, probs, tokens = m.balance_loss(lg, ids, d["mask"], seq_offsets=off)
    loss, each, n = m.distill_loss(lg, t_ids, t_logits, d["mask"])
    d_eo, d_tw, d_nw = m.combine_backward(d["y"], d["eo"], dest.view(-1, k), tw, d["nw"], 0.0, 1e-6)
    aux = m.balance_loss_backward(gl, lg, d["mask"], cnt, tokens, k, seq_offsets=off)
    m.distill_loss_backward(gd, lg, t_ids, t_logits, d["mask"], n, d_logits=aux, accumulate=True)
    d_l, d_h, d_W = m.route_backward(d_tw, d["hidden"], d["W"], lg, ids, tw, d["mask"], d_aux=aux)
    return dict(lg=lg, ids=ids, tw=tw, dest=dest, out=out, losses=losses, counts=cnt, loss=loss, d_eo=d_eo,
                d_tw=d_tw, d_nw=d_nw, d_l=d_l, d_h=d_h, d_W=d_W, t_ids=t_ids, t_logits=t_logits)


def test_training_step_chain():
    """route_dispatch, combine and the losses forward, then the gradients back
    to the router's input and weight, against the oracle's chain."""
    require_gpu()
    g = np.random.default_rng(51)
    T, H, E, k = 300, 256, 64, 4
    mask = _mask(g, T)
    d = _step_inputs(g, T, H, E, k, mask)
    off = np.array([0, 100, 100, 290], np.int32)
    gl, gd = np.array([0.02, 0.001], np.float32), np.array([0.1], np.float32)
    note("training step chain")
    r = _step({n: dev(v) for n, v in d.items()}, k, E, dev(off), dev(gl), dev(gd))
    h = {n: host(t) for n, t in r.items()}
    # every row that no slot names has no gradient: a dispatch's tail
    (deo, dtw, dnw), (meo, mtw, mnw) = OT.combine_backward(d["y"], d["eo"], h["dest"].reshape(T, k), h["tw"], d["nw"],
                                                          0.0, 1e-6)
    row = 128 * U
    _close(h["d_eo"], deo, row * meo + 2.0 ** -8 * np.abs(deo) + 2.0 ** -133, "d_eo")
    _close(h["d_tw"], dtw, row * mtw, "d_tw")
    _, counts, _, tokens = OT.balance_loss(h["lg"], h["ids"], mask, off)
    np.testing.assert_array_equal(h["counts"], counts)
    b, bm = OT.balance_loss_backward(gl, h["lg"], mask, counts, tokens, k, off)
    _, _, n, _ = OT.distill_loss(h["lg"], h["t_ids"], h["t_logits"], mask)
    dd, dm = OT.distill_loss_backward(gd[0], h["lg"], h["t_ids"], h["t_logits"], mask, n)
    P = _prob_tol(h["lg"], mask, E) + _prob_tol(d["teacher"], mask, E)
    (dl, dh, dW), (ml, mh, mW) = OT.route_backward(h["d_tw"], d["hidden"], d["W"], h["lg"], h["ids"], h["tw"], mask,
                                                   1.0, b + dd)
    extra = 4 * P * (bm + dm) + 2 * U * (np.abs(b) + np.abs(dd))
    _close(h["d_l"], dl, 40 * U * ml + extra, "d_l")
    _close(h["d_h"], dh, (200 * U + 3 * 2.0 ** -17) * mh + extra @ np.abs(d["W"]) + 2.0 ** -8 * np.abs(dh), "d_h")
    hid = np.abs(np.nan_to_num(O.bf16_bits_to_f64(d["hidden"])))
    _close(h["d_W"], dW, 300 * U * mW + extra.T @ hid, "d_W")


def test_training_step_replayed_from_a_graph_on_a_side_stream():
    """The chain captured on a stream of its own with preallocated buffers:
    replays with new inputs, eager work between, equal eager runs bit for bit."""
    require_gpu()
    g = np.random.default_rng(52)
    T, H, E, k = 260, 512, 96, 4
    masks = [_mask(g, T) for _ in range(3)]
    sets = [{n: dev(v) for n, v in _step_inputs(g, T, H, E, k, mk).items()} for mk in masks]
    off = dev(np.array([0, 90, 250], np.int32))
    gl, gd = torch.tensor([0.02, 0.001], device=DEV), torch.tensor([0.1], device=DEV)
    note("training step graph")
    eager = [_step(s, k, E, off, gl, gd) for s in sets]
    held = {n: t.clone() for n, t in sets[0].items()}
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        _step(held, k, E, off, gl, gd)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        out = _step(held, k, E, off, gl, gd)
    for i in (1, 2, 0, 2, 1):
        for n, t in sets[i].items():
            held[n].copy_(t)
        graph.replay()
        torch.cuda.synchronize()
        for n in eager[i]:
            a, b = out[n], eager[i][n]
            assert torch.equal(a.nan_to_num(7.0) if a.is_floating_point() else a,
                               b.nan_to_num(7.0) if b.is_floating_point() else b), "replay %d: %s" % (i, n)
        again = _step(sets[i], k, E, off, gl, gd)      # eager work between the replays
        assert torch.equal(again["d_W"], eager[i]["d_W"])


def test_training_steps_on_two_streams_at_once():
    """Two chains in flight together, each with its own inputs and buffers."""
    require_gpu()
    note("training steps on two streams")
    g = np.random.default_rng(54)
    k, E = 4, 96
    sets = [{n: dev(v) for n, v in _step_inputs(g, T, H, E, k, _mask(g, T)).items()} for T, H in ((260, 512), (700, 1024))]
    off = dev(np.array([0, 90, 250], np.int32))
    gl, gd = torch.tensor([0.02, 0.001], device=DEV), torch.tensor([0.1], device=DEV)
    alone = [_step(s, k, E, off, gl, gd) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(4):
        for i, stream in enumerate(streams):
            with torch.cuda.stream(stream):
                got[i].append(_step(sets[i], k, E, off, gl, gd))
    torch.cuda.synchronize()
    for i, want in enumerate(alone):
        for r in got[i]:
            for n, b in want.items():
                a, b = (t.nan_to_num(7.0) if t.is_floating_point() else t for t in (r[n], b))
                assert torch.equal(a, b), n


def test_tables_of_more_than_2_32_elements():
    """Long batches and large expert tables, of which only the end is valid,
    against the same work on that end alone."""
    require_gpu()
    T, E, k, H, n = (1 << 20) + 640, 4096, 2, 16, 320
    note("tables of more than 2^32 elements")
    torch.manual_seed(55)
    g = np.random.default_rng(55)
    l = torch.empty((T, E), device=DEV).normal_()
    mask = torch.zeros(T, dtype=torch.uint8, device=DEV)
    tail = _mask(g, n)
    mask[-n:] = dev(tail)
    ids = torch.randint(0, E // k, (T, k), dtype=torch.int32, device=DEV)
    ids[:, 1] += E // k
    assert l.numel() - n * E > 1 << 32
    end = [t[-n:].clone() for t in (l, ids, mask)]
    # balance: the same rows in the same order; sums of up to n tokens
    whole, part = m.balance_loss(l, ids, mask), m.balance_loss(*end)
    assert torch.equal(whole[1], part[1]) and torch.equal(whole[3], part[3])
    p = host(part[2]).astype(np.float64)
    _close(host(whole[2]), p, 2 * n * U * p, "probs")
    b = host(part[0]).astype(np.float64)
    _close(host(whole[0]), b, 4 * n * U * b, "losses")
    gl = torch.ones(2, device=DEV)
    d = m.balance_loss_backward(gl, l, mask, whole[1], whole[3], k)
    assert torch.equal(d[-n:], m.balance_loss_backward(gl, end[0], end[2], part[1], part[3], k))
    assert int(torch.count_nonzero(d[:-n])) == 0
    # distillation
    z = torch.empty((T, k), device=DEV).normal_()
    whole, part = m.distill_loss(l, ids, z, mask), m.distill_loss(end[0], end[1], z[-n:], end[2])
    assert torch.equal(whole[1][-n:], part[1]) and torch.equal(whole[2], part[2])
    assert int(torch.count_nonzero(whole[1][:-n])) == 0
    b = abs(float(part[0])) + float(part[1].abs().sum()) / n
    assert abs(float(whole[0]) - float(part[0])) <= 2 * n * U * b
    d = m.distill_loss_backward(gl[:1], l, ids, z, mask, whole[2], d_logits=d)
    assert torch.equal(d[-n:], m.distill_loss_backward(gl[:1], end[0], end[1], z[-n:], end[2], part[2]))
    assert int(torch.count_nonzero(d[:-n])) == 0
    # route
    w = torch.full((T, k), 0.5, device=DEV)
    h = g.standard_normal((n, H)).astype(np.float32)
    h = wl.f32_to_bf16_bits(h)
    W = g.standard_normal((E, H)).astype(np.float32)
    hidden = torch.full((T, H), float("nan"), dtype=torch.bfloat16, device=DEV)
    hidden[-n:] = dev(h)
    d, d_h, d_W = m.route_backward(z, hidden, dev(W), l, ids, w, mask, d_logits=d)
    (wl_, wh, wW), (ml, mh, mW) = OT.route_backward(host(z[-n:]), h, W, host(end[0]), host(end[1]),
                                                   np.full((n, k), 0.5, np.float32), tail)
    _close(host(d[-n:]), wl_, 40 * U * ml, "d_logits")
    _close(host(d_h[-n:]), wh, ((6 * E / 16 + 64) * U + 3 * 2.0 ** -17) * mh + 2.0 ** -8 * np.abs(wh), "d_hidden")
    # zeros add without a rounding: n tokens' steps count, and the splits
    _close(host(d_W), wW, (40 + 6 * (n / 16 + 1) + 64 + 3) * U * mW, "d_W")
    assert int(torch.count_nonzero(d[:-n])) == 0 and int(torch.count_nonzero(d_h[:-n])) == 0
    del l, d, d_h, z, w, hidden
    # combine
    T, H, R, k = 64, 8192, (1 << 19) + 100, 3
    slots = torch.randperm(R, device=DEV)[:T * k].to(torch.int32)
    slots[:4] = torch.tensor([R - 1, 0, R - 2, 1 << 19], dtype=torch.int32)
    slots = slots.unique()   # ascending
    slots = slots[torch.randperm(len(slots), device=DEV)][:T * k - 6].view(-1, k).contiguous()
    T = slots.shape[0]
    x = torch.empty((R, H), dtype=torch.bfloat16, device=DEV)
    x.fill_(float("nan"))
    rows = slots.flatten().long()
    x[rows] = torch.randn((T * k, H), device=DEV).bfloat16()
    y, tw, nw = torch.randn((T, H), device=DEV).bfloat16(), torch.rand((T, k), device=DEV), torch.rand(H, device=DEV)
    got = m.combine_backward(y, x, slots, tw, nw, 1.0, 1e-6)
    small = torch.arange(T * k, dtype=torch.int32, device=DEV).view(T, k)
    want = m.combine_backward(y, x[rows], small, tw, nw, 1.0, 1e-6)
    assert torch.equal(got[0][rows], want[0]) and torch.equal(got[1], want[1]) and torch.equal(got[2], want[2])
    assert int(torch.count_nonzero(got[0])) == int(torch.count_nonzero(want[0]))


def test_workspace_left_by_a_larger_call():
    """A call that is given a workspace full of another call's values, or of
    NaN, gives the same results: nothing is read before it is written."""
    require_gpu()
    g = np.random.default_rng(53)
    T, H, E, k, R = 90, 272, 70, 4, 400
    mask = _mask(g, T)
    l, ids = _logits(g, T, E, mask), _ids(g, T, E, k, mask)
    off = _cut(g, T, 5)
    w = np.full((T, k), 1 / k, np.float32)
    dw = g.standard_normal((T, k)).astype(np.float32)
    h = wl.f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32))
    W = g.standard_normal((E, H)).astype(np.float32)
    slots = g.permutation(R)[:T * k].astype(np.int32).reshape(T, k)
    y, x = h, wl.f32_to_bf16_bits(g.standard_normal((R, H)).astype(np.float32))
    nw = g.uniform(0.5, 1.5, H).astype(np.float32)
    t_ids, t_l = _teacher(g, l, 5)
    sizes = [m.balance_loss_workspace_bytes(T, E, 5), m.distill_loss_workspace_bytes(T, E),
             m.route_backward_workspace_bytes(T, H, E, m.MOE_DTYPE_BF16), m.combine_backward_workspace_bytes(T, R, H)]
    a = [dev(v) for v in (l, ids, mask, off, dw, h, W, w, slots, y, x, nw, t_ids, t_l)]

    def run(ws):
        out = list(m.balance_loss(a[0], a[1], a[2], seq_offsets=a[3], workspace=ws[0]))
        out += m.distill_loss(a[0], a[12], a[13], a[2], workspace=ws[1])
        out += m.route_backward(a[4], a[5], a[6], a[0], a[1], a[7], a[2], workspace=ws[2])
        out += m.combine_backward(a[9], a[10], a[8], a[7], a[11], 0.0, 1e-6, workspace=ws[3])
        return out

    ref = run([torch.zeros(n, dtype=torch.uint8, device=DEV) for n in sizes])
    got = run([torch.full((n,), 0xFF, dtype=torch.uint8, device=DEV) for n in sizes])
    for p, q in zip(ref, got):
        assert torch.equal(p, q)
