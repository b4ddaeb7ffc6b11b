"""The 64-bit references of the row operators against closed forms and central differences (CPU)."""
import numpy as np
import pytest

from tests.rows_ref import Norms, Recurrence

STEP = 1e-6
# a central difference with step 1e-6 of a 64-bit loss: truncation ~ 1e-12 times the third
# derivative, cancellation ~ 1e-16 / 1e-6 times the loss
TOL = 1e-6


def test_recurrence_is_the_bidiagonal_solve():
    rng = np.random.default_rng(1)
    x, r, i, lam = (rng.standard_normal(s) for s in ((9, 3), (9, 3), (9, 3), (3,)))
    h0 = rng.standard_normal((1, 3))
    ref = Recurrence(x, r, i, lam, 2.0, [(0, 9)], h0)
    for c in range(3):
        A = np.eye(9) - np.diag(ref.a[1:, c], -1)
        rhs = ref.u[:, c].copy()
        rhs[0] += ref.a[0, c] * h0[0, c]
        assert np.abs(np.linalg.solve(A, rhs) - ref.h[:, c]).max() < 1e-13
        rhs = rng.standard_normal(9)
        g = np.linalg.solve(A.T, rhs)
        full = np.zeros((9, 3))
        full[:, c] = rhs
        ref.backward(full)
        assert np.abs(ref.dx[:, c] - g * ref.s[:, c] * ref.si[:, c]).max() < 1e-13


def _differences(loss, arrays):
    out = []
    for a in arrays:
        g = np.zeros_like(a)
        for k in np.ndindex(a.shape):
            keep = a[k]
            a[k] = keep + STEP
            up = loss()
            a[k] = keep - STEP
            g[k] = (up - loss()) / (2 * STEP)
            a[k] = keep
        out.append(g)
    return out


def test_recurrence_gradients_against_differences():
    rng = np.random.default_rng(2)
    spans = [(0, 4), (4, 4), (4, 5), (6, 9)]
    x, r, i = (rng.standard_normal((9, 2)) for _ in range(3))
    lam, h0 = rng.standard_normal(2), rng.standard_normal((4, 2))
    dh, dhT = rng.standard_normal((9, 2)), rng.standard_normal((4, 2))
    dh[5] = 0  # row 5 belongs to no sequence

    def loss():
        ref = Recurrence(x, r, i, lam, 3.0, spans, h0)
        return (ref.h * dh).sum() + (ref.hT * dhT).sum()

    ref = Recurrence(x, r, i, lam, 3.0, spans, h0).backward(dh, dhT)
    for got, want in zip((ref.dx, ref.dr, ref.di, ref.dlam, ref.dh0),
                         _differences(loss, (x, r, i, lam, h0))):
        assert np.abs(got - want).max() < TOL * max(1.0, np.abs(want).max())


@pytest.mark.parametrize("gate", [0, 1, 2])
@pytest.mark.parametrize("post", [True, False])
def test_norm_gradients_against_differences(gate, post):
    rng = np.random.default_rng(3)
    f, z, x = (rng.standard_normal((3, 5)) for _ in range(3))
    w, c, p = (1 + 0.3 * rng.standard_normal(5) for _ in range(3))
    dy, du = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def make():
        return Norms(f, z, x, w if post else None, c, p, 1e-3, gate)

    def loss():
        ref = make()
        return (ref.y * dy).sum() + (ref.u * du).sum()

    ref = make().backward(dy, du)
    got = [ref.df, ref.dz, ref.dx, ref.dscale, ref.dw_pre] + ([ref.dw_post] if post else [])
    for g, want in zip(got, _differences(loss, [f, z, x, c, p] + ([w] if post else []))):
        assert np.abs(g - want).max() < TOL * max(1.0, np.abs(want).max())
