"""The fp64 oracle of the fine-tuning operators: its gradients against central differences of its own
forwards, and its hand-checkable corners."""
import numpy as np
import pytest

from oracle import tuning


def _rng(seed=0):
    return np.random.default_rng(seed)


def _difference(f, v, direction, eps=1e-6):
    return (f(v + eps * direction) - f(v - eps * direction)) / (2 * eps)


@pytest.mark.parametrize("renorm", [False, True])
def test_router_gradient_is_the_derivative(renorm):
    r = _rng(1)
    T, E, k = 9, 7, 3
    l = r.normal(size=(T, E))
    idx = np.argsort(-l, axis=1)[:, :k]
    g = r.normal(size=(T, k))
    offsets, mask = [0, 4, 4, 8], np.array([1, 1, 0, 1, 1, 1, 1, 1, 1])

    def value(v):
        p = tuning.softmax_rows(v)
        w = np.take_along_axis(p, idx, 1)
        if renorm:
            w = w / w.sum(1, keepdims=True)
        return float(np.sum(g * w)) + 0.7 * tuning.balance_loss(v, idx, 0.3, offsets, mask)[0]

    _, counts, _, coef = tuning.balance_loss(l, idx, 0.3, offsets, mask)
    got = tuning.router_backward(l, idx, g, renorm, (counts, coef, 0.7, offsets, mask))
    for seed in range(5):
        d = _rng(seed + 10).normal(size=l.shape)
        assert np.isclose(np.sum(got * d), _difference(value, l, d), rtol=1e-6, atol=1e-9)


def test_balance_loss_of_an_even_router_is_alpha():
    # every expert equally likely and equally chosen: f = P = 1 / E, alpha * E * E / E^2
    loss, counts, prob, coef = tuning.balance_loss(np.zeros((8, 4)), np.arange(8)[:, None] % 4, 0.25)
    assert np.isclose(loss, 0.25) and np.all(counts == 2) and np.allclose(prob, 0.25)
    assert np.isclose(coef[0], 0.25 * 4 / (1 * 64 * 1))


def test_balance_loss_leaves_out_what_the_mask_and_the_sequences_do():
    l = _rng(2).normal(size=(6, 3))
    l[1] = np.nan
    l[5] = np.inf
    idx = np.array([[0], [1], [2], [0], [1], [2]])
    loss, counts, prob, coef = tuning.balance_loss(l, idx, 1.0, [0, 2, 2, 5], [1, 0, 1, 1, 1, 1])
    assert np.isfinite(loss) and counts.tolist() == [[1, 0, 0], [0, 0, 0], [1, 1, 1]]
    assert coef[1] == 0 and np.all(prob[1] == 0)


def test_adapter_gradients_are_the_derivative():
    r = _rng(3)
    T, d, N, R, n = 11, 6, 5, 2, 3
    x, A, B = r.normal(size=(T, d)), r.normal(size=(n, R, d)), r.normal(size=(n, N, R))
    row, scale = np.array([0, 2, -1, 2, 2, 0, -1, 0, 2, 2, 0]), r.normal(size=n)
    g, base = r.normal(size=(T, N)), r.normal(size=(T, N))

    def value(x_, A_, B_):
        return float(np.sum(g * tuning.lora(x_, A_, B_, row, scale, base)[0]))

    h = tuning.lora(x, A, B, row, scale)[1]
    dx, dA, dB = tuning.lora_backward(g, x, h, A, B, row, scale)
    u, v, w = (r.normal(size=t.shape) for t in (x, A, B))
    assert np.isclose(np.sum(dx * u), _difference(lambda t: value(t, A, B), x, u), rtol=1e-6, atol=1e-8)
    assert np.isclose(np.sum(dA * v), _difference(lambda t: value(x, t, B), A, v), rtol=1e-6, atol=1e-8)
    assert np.isclose(np.sum(dB * w), _difference(lambda t: value(x, A, t), B, w), rtol=1e-6, atol=1e-8)
    assert not dA[1].any() and not dB[1].any()


def test_combine_gradient_is_the_derivative():
    r = _rng(4)
    T, k, d = 4, 2, 3
    Y, w = r.normal(size=(T * k + T, d)), r.normal(size=(T, k))
    t2r = r.permutation(T * k).reshape(T, k)
    t2r[1, 1] = -1
    g = r.normal(size=(T, d))

    def out(Y_, w_):
        o = Y_[T * k:].copy()
        for t in range(T):
            for j in range(k):
                if t2r[t, j] >= 0:
                    o[t] += w_[t, j] * Y_[t2r[t, j]]
        return float(np.sum(g * o))

    dY, dw = tuning.combine_backward(g, Y, t2r, w, T * k)
    u, v = r.normal(size=Y.shape), r.normal(size=w.shape)
    assert np.isclose(np.sum(dY * u), _difference(lambda t: out(t, w), Y, u), rtol=1e-6, atol=1e-9)
    assert np.isclose(np.sum(dw * v), _difference(lambda t: out(Y, t), w, v), rtol=1e-6, atol=1e-9)


# The tiles of the adapters' kernels: every position of the plan lies in exactly one, inside its adapter.
def _find_tile(off, n, rows, mt, u):
    held = lambda a: rows if a > n else min(max(off[a], 0), rows)  # noqa: E731
    lo, size = 0, n + 1
    while size > 1:
        step = (size + 31) // 32
        le = [l for l in range(32) if l * step < size and held(lo + l * step) // mt + lo + l * step <= u]
        top = le[-1] if le else 0
        size = min(step, size - top * step)
        lo += top * step
    b, e = held(lo), held(lo + 1)
    s = b + (u - b // mt - lo) * mt
    return None if s < b or s >= e else (lo, s, min(e, s + mt))


@pytest.mark.parametrize("n", [1, 2, 31, 32, 33, 100, 1024])
@pytest.mark.parametrize("mt", [16, 64, 512])
def test_tiles_cover_every_row_once(n, mt):
    r = _rng(n * 1000 + mt)
    for rows in (1, mt - 1, mt, mt + 1, 5 * mt + 3):
        cuts = np.sort(r.integers(0, rows + 1, size=n))
        off = [0] + cuts.tolist()
        seen = np.full(rows, -2)
        for u in range(rows // mt + n + 1):
            t = _find_tile(off, n, rows, mt, u)
            if t:
                assert np.all(seen[t[1]:t[2]] == -2) and t[2] - t[1] <= mt
                seen[t[1]:t[2]] = t[0]
        want = np.concatenate([np.full(off[a + 1] - off[a], a) for a in range(n)] + [np.full(rows - off[n], n)])
        assert np.array_equal(seen, want)


def test_tiles_of_bad_offsets_stay_in_bounds():
    r = _rng(7)
    for _ in range(300):
        n, rows = int(r.integers(1, 70)), int(r.integers(1, 200))
        off = r.integers(-50, 300, size=n + 1).tolist()
        for u in range(rows // 16 + n + 1):
            t = _find_tile(off, n, rows, 16, u)
            assert t is None or (0 <= t[1] < t[2] <= rows and t[2] - t[1] <= 16 and 0 <= t[0] <= n)
