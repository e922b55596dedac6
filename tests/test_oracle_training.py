"""The training oracle against differences of its own losses, closed forms and
the route's and the combine's forward oracles."""
import numpy as np
import pytest

import oracle as O
from oracle import training as OT
import workloads as wl


def _difference(f, x, at, h=1e-5):
    """Central difference of the scalar f along element `at` of x (float64)."""
    a, b = x.copy(), x.copy()
    a[at] += h
    b[at] -= h
    return (f(a) - f(b)) / (2 * h)


def _batch(g, T, E, k):
    logits = g.standard_normal((T, E)) * 1.5
    ids = np.argsort(-logits, axis=1)[:, :k].astype(np.int32)
    mask = g.uniform(size=T) > 0.2
    mask[0] = True
    return logits, ids, mask


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
def test_distribution_is_normalised_scores(score):
    g = np.random.default_rng(1)
    l = g.standard_normal((5, 17)) * 3
    s = 1 / (1 + np.exp(-l)) if score == OT.SIGMOID else np.exp(l)
    np.testing.assert_allclose(OT.distribution(l, score), s / s.sum(1, keepdims=True), rtol=1e-13)
    # far below underflow the proportions stay: sigmoid(l) ~ exp(l)
    np.testing.assert_allclose(OT.distribution(l - 2000, OT.SIGMOID), OT.distribution(l, OT.SOFTMAX), rtol=1e-9)
    assert (OT.distribution(np.full((1, 4), -np.inf), score) == 0).all()


def test_balance_loss_closed_forms():
    # uniform logits and evenly spread picks: the balance loss is 1, z is log(E)^2
    T, E, k = 12, 6, 2
    ids = np.arange(T * k).reshape(T, k) % E
    losses, counts, probs, tokens = OT.balance_loss(np.zeros((T, E)), ids, np.ones(T), None, OT.SIGMOID)
    np.testing.assert_allclose(losses, [1.0, np.log(E) ** 2], rtol=1e-14)
    assert (counts == T * k // E).all() and list(tokens) == [T, T, 1]
    np.testing.assert_allclose(probs, T / E)
    # every token on one expert with all of the probability: the loss is E
    l = np.full((T, E), -60.0)
    l[:, 3] = 60.0
    losses, _, _, _ = OT.balance_loss(l, np.full((T, 1), 3), np.ones(T), None, OT.SOFTMAX)
    np.testing.assert_allclose(losses[0], E)
    # the mean over sequences with a token; empty ones and tokens behind the last count nowhere
    off = [0, 0, 5, 5, 9]
    losses, counts, _, tokens = OT.balance_loss(np.zeros((T, E)), ids, np.ones(T), off, OT.SIGMOID)
    assert list(tokens) == [0, 5, 0, 4, 9, 2]
    assert counts.sum() == 9 * k and (counts[0] == 0).all()


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
def test_balance_gradient_is_the_difference(score):
    g = np.random.default_rng(2)
    T, E, k = 11, 7, 2
    l, ids, mask = _batch(g, T, E, k)
    off = [0, 4, 4, 9]
    gl = np.array([0.7, 0.3])
    _, counts, _, tokens = OT.balance_loss(l, ids, mask, off, score)
    d, mag = OT.balance_loss_backward(gl, l, mask, counts, tokens, k, off, score)
    f = lambda x: (gl * OT.balance_loss(x, ids, mask, off, score)[0]).sum()
    for at in np.ndindex(T, E):
        np.testing.assert_allclose(d[at], _difference(f, l, at), atol=1e-9)
    assert (np.abs(d) <= mag + 1e-15).all()


@pytest.mark.parametrize("score", [OT.SIGMOID, OT.SOFTMAX])
@pytest.mark.parametrize("temperature", [0.5, 1.0, 3.0])
def test_distill_gradient_is_the_difference(score, temperature):
    g = np.random.default_rng(3)
    T, E, K = 9, 6, 4
    l, _, mask = _batch(g, T, E, 2)
    ids = np.stack([g.choice(E, K, replace=False) for _ in range(T)]).astype(np.int32)
    ids[1] = -1
    ids[2, 1:] = E
    ids[3, 1] = ids[3, 0]          # named twice
    z = g.standard_normal((T, K))
    z[4, 0] = -np.inf
    loss, each, n, mag = OT.distill_loss(l, ids, z, mask, score, temperature)
    d, _ = OT.distill_loss_backward(0.8, l, ids, z, mask, n, score, temperature)
    f = lambda x: 0.8 * OT.distill_loss(x, ids, z, mask, score, temperature)[0]
    for at in np.ndindex(T, E):
        np.testing.assert_allclose(d[at], _difference(f, l, at), atol=1e-9)
    assert each[1] == 0 and (d[1] == 0).all()


def test_distill_of_the_same_router_is_zero_at_full_width():
    """All E entries of the same logits: both distributions agree, loss and
    gradient vanish; the sigmoid's shares are a route's weights."""
    g = np.random.default_rng(4)
    T, E = 6, 8
    l = g.standard_normal((T, E)).astype(np.float32)
    ids, w = O.route_from_logits(l, np.zeros(E, np.float32), np.ones(T), E)
    z = np.take_along_axis(l, ids.astype(np.int64), 1)
    loss, each, n, _ = OT.distill_loss(l, ids, z, np.ones(T), OT.SIGMOID)
    assert n == T and np.abs(each).max() < 1e-14
    assert np.abs(OT.distill_loss_backward(1.0, l, ids, z, np.ones(T), n, OT.SIGMOID)[0]).max() < 1e-15
    _, _, _, q = OT._teacher(ids, z, np.ones(T), E, OT.SIGMOID, 1.0)
    np.testing.assert_allclose(q, w, rtol=1e-6)


def test_route_gradient_is_the_difference():
    g = np.random.default_rng(5)
    T, H, E, k = 7, 5, 9, 3
    h, W = g.standard_normal((T, H)), g.standard_normal((E, H))
    scale = 0.75
    mask = np.array([1, 1, 0, 1, 1, 1, 1])
    dw, aux = g.standard_normal((T, k)), g.standard_normal((T, E)) * 0.1
    ids = np.argsort(-(h @ W.T), axis=1)[:, :k].astype(np.int32)
    ids[2] = -1

    def weights(l):
        s = 1 / (1 + np.exp(-np.take_along_axis(l, np.maximum(ids, 0).astype(np.int64), 1)))
        return s / s.sum(1, keepdims=True)

    def loss(h_, W_):
        l = scale * h_ @ W_.T
        v = mask.astype(bool)
        return (weights(l) * dw)[v].sum() + (l * aux)[v].sum()

    l = scale * h @ W.T
    (dl, dh, dW), mags = OT.route_backward(dw, h, W, l, ids, weights(l), mask, scale, aux)
    for at in np.ndindex(T, H):
        np.testing.assert_allclose(dh[at], _difference(lambda x: loss(x, W), h, at), atol=1e-8)
    for at in np.ndindex(E, H):
        np.testing.assert_allclose(dW[at], _difference(lambda x: loss(h, x), W, at), atol=1e-8)
    assert (dl[2] == 0).all()
    for v, m in zip((dl, dh, dW), mags):
        assert (np.abs(v) <= m + 1e-14).all()


def test_combine_gradient_is_the_difference():
    g = np.random.default_rng(6)
    T, H, k, R = 4, 8, 3, 10
    x = wl.f32_to_bf16_bits(g.standard_normal((R, H)).astype(np.float32))
    y = wl.f32_to_bf16_bits(g.standard_normal((T, H)).astype(np.float32))
    slots = g.permutation(R)[:9].reshape(3, 3)
    slots = np.concatenate([slots, [[-1, slots[0, 0], R]]]).astype(np.int32)   # a row named twice, two invalid
    w, nw = g.uniform(0.1, 1, (T, k)), g.uniform(-0.5, 0.5, H).astype(np.float32)
    eps, center = 1e-3, 1.0
    x64, y64 = O.bf16_bits_to_f64(x), O.bf16_bits_to_f64(y)
    e64 = float(np.float32(eps))

    def loss(x_, w_, n_):
        total = 0.0
        for t in range(T):
            for j in range(k):
                r = slots[t, j]
                if 0 <= r < R:
                    v = x_[r]
                    total += (w_[t, j] * v * (center + n_) / np.sqrt((v * v).mean() + e64) * y64[t]).sum()
        return total

    (dx, dw, dn), mags = OT.combine_backward(y, x, slots, w, nw, center, eps)
    n64 = (np.float32(center) + nw).astype(np.float64) - center
    for at in np.ndindex(R, H):
        np.testing.assert_allclose(dx[at], _difference(lambda v: loss(v, w, n64), x64, at), atol=1e-8)
    for at in np.ndindex(T, k):
        np.testing.assert_allclose(dw[at], _difference(lambda v: loss(x64, v, n64), w, at), atol=1e-8)
    for i in range(H):
        np.testing.assert_allclose(dn[i], _difference(lambda v: loss(x64, w, v), n64, i), atol=1e-8)
    assert dw[3, 0] == 0 and dw[3, 2] == 0
    for v, m in zip((dx, dw, dn), mags):
        assert (np.abs(v) <= m + 1e-14).all()
