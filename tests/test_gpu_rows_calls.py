"""Calls of the row operators on the GPU that are rare in use."""
import numpy as np
import pytest
import torch

import dense_linear_solvers_gb300 as bs

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.rows_ref import EPS  # noqa: E402


@pytest.mark.parametrize("eps", [1e-44, 1e-40, 1e-38, 1e-36])
@pytest.mark.parametrize("width", [40, 700, 9000])
def test_norms_of_small_rows_under_a_small_eps(eps, width):
    """Rows whose squares vanish beside eps, a subnormal number included: n = f / sqrt(eps) w. An
    inverse root and three products, a few EPS."""
    eps = float(np.float32(eps))
    rng = np.random.default_rng(1)
    f = torch.from_numpy(rng.standard_normal((3, width)) * 1e-26).float().cuda()
    w = torch.full((width,), 0.5, device="cuda")
    dy = torch.from_numpy(rng.standard_normal((3, width)) * 1e-6).float().cuda()
    y, df = torch.empty_like(f), torch.empty_like(f)
    bs.bs_gnorm_batched(f, y, w_post=w, eps=eps)
    want = f.double() / eps ** 0.5 * 0.5
    assert bool(((y.double() - want).abs() <= 8 * EPS * want.abs()).all())
    bs.bs_gnorm_backward_batched(f, dy, df, w_post=w, eps=eps)
    # the second term, n mean(dn n), is below 1e-8 of the first: n is at most 1e-3 here
    want = dy.double() / eps ** 0.5 * 0.5
    n = f.double() / eps ** 0.5
    want -= n * (dy.double() * 0.5 * n).mean(1, keepdim=True) / eps ** 0.5
    size = dy.double().abs().amax(1, keepdim=True) / eps ** 0.5
    assert bool(((df.double() - want).abs() <= 16 * EPS * size).all())


def test_a_gate_past_32_bits_is_refused():
    f = torch.ones(2, 8, device="cuda")
    for gate in (1 << 32, (1 << 32) + 1, -(1 << 32), 3, -1):
        with pytest.raises(bs.BsolveError, match="INVALID_ARG"):
            bs.bs_gnorm_batched(f, torch.empty_like(f), gate=gate)
        with pytest.raises(bs.BsolveError, match="INVALID_ARG"):
            bs.bs_gnorm_backward_batched(f, f, torch.empty_like(f), gate=gate)


def test_views_with_a_pending_sign_are_refused():
    """Memory that torch reads with the other sign: its values are not the tensor's."""
    x, lam = torch.ones(2, 10, 8, device="cuda"), torch.zeros(8, device="cuda")
    neg = torch._neg_view
    with pytest.raises(ValueError, match="sign"):
        bs.bs_grec_batched(neg(x), x, x, lam, torch.empty_like(x))
    with pytest.raises(ValueError, match="sign"):
        bs.bs_grec_batched(x, x, x, neg(lam), torch.empty_like(x))
    with pytest.raises(ValueError, match="sign"):
        bs.bs_gnorm_batched(x, neg(torch.empty_like(x)))
