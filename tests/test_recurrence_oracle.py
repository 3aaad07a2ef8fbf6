"""The recurrence's oracle against independent forms: closed forms, central differences of the
definitions, and values worked by hand."""
import numpy as np
import pytest

import oracle.layer as layer
import oracle.recurrence as ref

SPANS = [(0, 3), (3, 3), (3, 70), (70, 71), (71, 140)]


def inputs(seed, gate, D=3, rows=140):
    rng = np.random.default_rng(seed)
    g = rng.standard_normal((rows, D))
    return rng.standard_normal((rows, D)), -np.abs(g) if gate == "log" else g, rng.standard_normal((len(SPANS), D)), rng


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
def test_scan_is_the_sum_over_earlier_tokens(gate):
    x, g, h0, _ = inputs(0, gate)
    for complement in (False, True):
        y, final, chunks, *bounds = ref.scan(x, g, SPANS, h0, gate, complement)
        a, rest = ref.decays(g, gate)
        for n, (first, end) in enumerate(SPANS):
            for t in range(first, end):
                want = np.prod(a[first:t + 1], 0) * h0[n]
                for s in range(first, t + 1):
                    want = want + np.prod(a[s + 1:t + 1], 0) * x[s] * (rest[s] if complement else 1)
                np.testing.assert_allclose(y[t], want, rtol=1e-12, atol=1e-13)
            np.testing.assert_allclose(final[n], y[end - 1] if end > first else h0[n])
        np.testing.assert_allclose(chunks, [h0[0], y[63], y[127]])
        assert all((b >= 0).all() for b in bounds)


@pytest.mark.parametrize("gate", ["log", "sigmoid"])
@pytest.mark.parametrize("complement", [False, True])
def test_scan_gradients_are_the_differences(gate, complement):
    x, g, h0, rng = inputs(1, gate)
    dy, df = rng.standard_normal(x.shape), rng.standard_normal(h0.shape)

    def loss(x, g, h0):
        y, final, *_ = ref.scan(x, g, SPANS, h0, gate, complement)
        return np.sum(y * dy) + np.sum(final * df)

    chunks = ref.scan(x, g, SPANS, h0, gate, complement)[2]
    grads = ref.scan_backward(dy, x, g, chunks, SPANS, h0, df, gate, complement)[:3]
    args = [x, g, h0]
    for which, grad in enumerate(grads):
        for at in [(0, 0), (2, 1), (4, 2)] + ([(3, 0), (69, 1), (70, 2), (127, 0), (139, 1)] if which < 2 else []):
            moved = []
            for step in (1e-5, -1e-5):
                there = [np.array(v) for v in args]
                there[which][at] += step
                moved.append(loss(*there))
            # central differences: truncation of order step^2, cancellation of order 1e-15 / step
            assert abs((moved[0] - moved[1]) / 2e-5 - grad[at]) <= 1e-7 * (1 + abs(grad[at])), (which, at)


@pytest.mark.parametrize("activation", ["sigmoid", "silu"])
def test_norm_gradients_are_the_differences(activation):
    rng = np.random.default_rng(2)
    x, z, dy, w = rng.standard_normal((4, 7)), rng.standard_normal((4, 7)), rng.standard_normal((4, 7)), rng.standard_normal(7)
    grads = ref.gated_norm_backward(dy, x, z, w, 1e-3, activation)[:3]
    args = [x, z, w]
    for which, grad in enumerate(grads):
        for at in np.ndindex(grad.shape):
            moved = []
            for step in (1e-5, -1e-5):
                there = [np.array(v) for v in args]
                there[which][at] += step
                moved.append(np.sum(layer.gated_norm(there[0], there[1], there[2], 1e-3, activation) * dy))
            assert abs((moved[0] - moved[1]) / 2e-5 - grad[at]) <= 1e-7 * (1 + abs(grad[at])), (which, at)


def test_checkpoint_by_hand():
    x = np.zeros((1, 70))
    x[0, 0], x[0, 1], x[0, 2], x[0, 3] = 127.0, 0.5, -1.5, 126.5         # e = 0: ties to even
    x[0, 32], x[0, 33] = -127.5, 1.0                                      # e = 1
    x[0, 64], x[0, 65] = 2.0 ** -140, -(2.0 ** -149)                      # below the least scale
    codes, exps, values = ref.checkpoint(x)
    assert list(exps[0]) == [127, 128, 0]
    assert list(codes[0, :4]) == [127, 0, -2, 126] and list(codes[0, 32:34]) == [-64, 0] and list(codes[0, 64:]) == [0] * 6
    assert list(values[0, 32:34]) == [-128.0, 0.0]
    x[0, 40] = np.inf
    assert np.isnan(ref.checkpoint(x)[2][0, 32:64]).all() and ref.checkpoint(x)[1][0, 1] == 255


def test_checkpoint_error_is_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 64)) * 10.0 ** rng.uniform(-30, 30, (20, 1))
    codes, exps, values = ref.checkpoint(x)
    scale = np.repeat(2.0 ** (exps.astype(float) - 127), 32, axis=1)
    assert (np.abs(values - x) <= scale / 2).all()
    top = np.abs(x).reshape(20, 2, 32).max(-1)
    assert (scale[:, ::32] / 2 <= top / 127).all()
