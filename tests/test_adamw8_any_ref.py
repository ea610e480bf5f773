"""The form of the 8-bit AdamW step for any gradient: it is adamw8_ref's on
ordinary ones, the formula in 64 bits on large ones, and NaN in one element
alone where one is not finite (CPU)."""
import numpy as np
import pytest

import adamw8_any_ref as ra
import adamw8_ref as r8

F = np.float32


def _state(n, rng):
    nb = -(-n // 256)
    return (rng.integers(0, 127, n).astype(np.uint8) | (rng.integers(0, 2, n).astype(np.uint8) << 7),
            rng.integers(0, 127, n).astype(np.uint8), (rng.random(nb) * 1e-5).astype(F), (rng.random(nb) * 1e-5).astype(F))


@pytest.mark.parametrize("n", [1, 300, 2048])
def test_ordinary_gradients_give_the_same_bits(n):
    rng = np.random.default_rng(n)
    theta = rng.normal(size=n).astype(F)
    g = r8.bf16(rng.normal(size=n) * 2.0 ** rng.integers(-40, 60, n)).float().numpy()
    state = _state(n, rng)
    args = (2, 11, 1e-3, 0.9, 0.999, 1e-8, 0.01, 5)
    for a, b in zip(ra.step(theta, g, *state, *args), r8.step(theta, g, *state, *args)):
        assert np.array_equal(a.view(np.uint8), b.view(np.uint8))


def test_large_gradients_against_64_bits():
    rng = np.random.default_rng(7)
    n = 512
    theta = rng.normal(size=n).astype(F)
    g = r8.bf16(rng.normal(size=n) * 2.0 ** rng.integers(60, 125, n)).float().numpy()
    g[0] = 2.0**127 * (2 - 2.0**-7)      # bf16's largest
    cm, cu, dm, du = _state(n, rng)
    dm, du = dm * F(2.0**100), du * F(2.0**100)
    b1, b2 = 0.9, 0.999
    th, ncm, ncu, ndm, ndu = ra.step(theta, g, cm, cu, dm, du, 0, 1, 1e-3, b1, b2, 1e-8, 0.0, 9)
    rep = lambda d: np.repeat(d.astype(np.float64), 256)[:n]  # noqa: E731
    m = b1 * r8.decode(cm) * rep(dm) + (1 - b1) * g.astype(np.float64)
    mm = b1 * np.abs(r8.decode(cm)) * rep(dm) + (1 - b1) * np.abs(g.astype(np.float64))
    u = np.sqrt(b2 * (r8.decode(cu) * rep(du)) ** 2 + (1 - b2) * g.astype(np.float64) ** 2)
    upd = 1e-3 / (1 - b1**9) / (u / np.sqrt(1 - b2**9) + 1e-8)
    # as for ordinary gradients: two roundings of theta's size and one of the result, about ten of the update's terms
    assert np.all(np.abs(th - (theta - upd * m)) <= 2.0**-24 * (3 * np.abs(theta) + 12 * upd * mm) + 1e-30)
    top = lambda x: np.abs(x).reshape(-1, 256).max(1)  # noqa: E731
    assert np.allclose(ndm, top(m) / 448, rtol=2.0**-20, atol=0) and np.allclose(ndu, top(u) / 448, rtol=2.0**-20, atol=0)
    assert np.isfinite(r8.decode(ncm)).all() and np.isfinite(r8.decode(ncu)).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_one_bad_element_keeps_to_itself(bad):
    rng = np.random.default_rng(3)
    n, at = 512, 77
    out = []
    for x in (bad, 0.0):
        r = np.random.default_rng(3)
        theta = r.normal(size=n).astype(F)
        state = (np.zeros(n, np.uint8), np.zeros(n, np.uint8), np.zeros(2, F), np.zeros(2, F))
        for t in (1, 2, 3):
            g = r8.bf16(r.normal(size=n)).float().numpy()
            g[at] = x if t == 1 else 0.0
            theta, *state = ra.step(theta, g, *state, 0, t, 1e-3, 0.9, 0.999, 1e-8, 0.0, t)
        out.append((theta, *state))
    rest = np.arange(n) != at
    for a, b in zip(*out):
        if a.size == n:
            a, b = a[rest], b[rest]
        assert np.array_equal(a, b) and np.isfinite(a.astype(F)).all()
    assert np.isnan(out[0][0][at]) and out[0][1][at] == out[0][2][at] == ra.NAN_CODE
