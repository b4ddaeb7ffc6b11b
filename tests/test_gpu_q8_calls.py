"""Calls of the 8-bit norm output and the 8-bit product that the documentation allows and few programs make."""
import pytest
import torch

import dense_linear_solvers_gb300 as bs

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

E4M3 = torch.float8_e4m3fn


@pytest.mark.parametrize("m, n", [(1, 1), (5, 40), (200, 129)])
def test_a_product_of_no_depth(m, n):
    """Operands as torch makes them for no element a row: rows one element apart."""
    a, w = (torch.empty(r, 0, device="cuda").to(E4M3) for r in (m, n))
    sa, sw = (torch.empty(r, 0, device="cuda") for r in (m, -(-n // 128)))
    y = torch.full((m, n + 3), 7.0, device="cuda")
    bs.bs_gemm_q8(a, sa, w, sw, y[:, 1:n + 1])
    assert bool((y[:, 1:n + 1] == 0).all()) and bool((y[:, :1] == 7).all()) and bool((y[:, n + 1:] == 7).all())
