"""Every form of the gated delta rule's chains and of the 8-bit product's kernels on the GPU against 64 bits, at the
shapes that reach them (which those are is tested on the host)."""
import pytest
import torch

import dense_linear_solvers_gb300 as bs

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.delta_forms import CHAINS, CUTS, PACKED, PRODUCTS, allowed  # noqa: E402
from tests.test_gpu_gdelta import (KINDS, backward, check_gradients, forward, inputs, reference,  # noqa: E402
                                   tape_of)
from tests.test_gpu_q8 import E4M3, check  # noqa: E402


def near(name, got, want, bound):
    far = float((got.double() - want).norm() / want.norm())
    assert far <= bound, (name, far, bound)


def check_near(ref, got, kind, length):
    """What is returned in FP32 is as near as two terms an operand make it."""
    for name, t in got.items():
        if t.dtype == torch.float32:
            near(name, t, getattr(ref, name), allowed(length, name not in ("o", "hT")))


@pytest.mark.parametrize("shape", [s for s, _ in CHAINS], ids=lambda s: "-".join(map(str, s)))
def test_chains(shape):
    kind, batch, length, hk, hv, dk, dv, pad = shape
    x = inputs(kind, batch * length, hk, hv, dk, dv, seed=length, pad=pad)
    do = torch.randn(batch * length, hv, dv, device="cuda").to(KINDS[kind])
    h0, dhT = (torch.randn(batch, hv, dk, dv, device="cuda") for _ in range(2))
    hT, dh0, tape = torch.empty_like(h0), torch.empty_like(h0), tape_of(x, batch)
    o = forward(*x, batch, h0=h0, hT=hT, tape=tape)
    got = backward(x, tape, do, batch, dhT=dhT, dh0=dh0)
    spans = [(b * length, (b + 1) * length) for b in range(batch)]
    ref = reference(*x, spans, h0=h0.double()).backward(do.double(), dhT.double())
    assert ref.close("o", o, KINDS[kind])[0] and ref.close("hT", hT, torch.float32)[0]
    check_gradients(ref, dict(got, dh0=dh0), KINDS[kind])
    check_near(ref, dict(got, dh0=dh0, o=o, hT=hT), kind, length)
    # without a tape, the state in place; the same bits again
    state, grad = h0.clone(), dhT.clone()
    assert torch.equal(forward(*x, batch, h0=state, hT=state), o) and torch.equal(state, hT)
    again = backward(x, tape, do, batch, dhT=grad, dh0=grad)
    assert all(torch.equal(again[n], got[n]) for n in got) and torch.equal(grad, dh0)


@pytest.mark.parametrize("kind, hk, hv, dk, dv", PACKED)
def test_packed_chains(kind, hk, hv, dk, dv):
    """An empty sequence, one of a row, of 64 and 128 rows and others; rows of none keep what was there."""
    rows, batch, offsets = CUTS[-1] + 5, len(CUTS) - 1, torch.tensor(CUTS, device="cuda")
    x = inputs(kind, rows, hk, hv, dk, dv, seed=21)
    do = torch.randn(rows, hv, dv, device="cuda").to(KINDS[kind])
    for t in (*x, do):
        t[:CUTS[0]], t[CUTS[-1]:] = float("nan"), float("nan")
    h0, dhT = (torch.randn(batch, hv, dk, dv, device="cuda") for _ in range(2))
    hT, dh0, tape = torch.empty_like(h0), torch.empty_like(h0), tape_of(x, batch)
    o = forward(*x, batch, offsets, h0=h0, hT=hT, tape=tape)
    got = backward(x, tape, do, batch, offsets, dhT=dhT, dh0=dh0)
    ref = reference(*x, list(zip(CUTS[:-1], CUTS[1:])), h0=h0.double()).backward(do.double(), dhT.double())
    for t in (o, *got.values()):
        assert bool((t[:CUTS[0]] == 7).all()) and bool((t[CUTS[-1]:] == 7).all())
        t[:CUTS[0]], t[CUTS[-1]:] = 0, 0
    assert ref.close("o", o, KINDS[kind])[0] and ref.close("hT", hT, torch.float32)[0]
    check_gradients(ref, dict(got, dh0=dh0), KINDS[kind])
    longest = max(b - a for a, b in zip(CUTS[:-1], CUTS[1:]))
    check_near(ref, dict(got, dh0=dh0, o=o, hT=hT), kind, longest)
    assert torch.equal(hT[0], h0[0]) and torch.equal(dh0[0], dhT[0])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", [s for s, _ in PRODUCTS], ids=lambda s: "-".join(map(str, s)))
def test_products(shape, kind):
    """Operands as windows of matrices that hold NaN around them, y as one of a matrix that keeps what it held."""
    m, n, k, ld = shape
    gen = torch.Generator("cuda").manual_seed(m + n)
    wide = -(-k // 16) * 16 + 32
    ops, scales = [], []
    for rows, parts in ((m, m), (n, -(-n // 128))):
        t = torch.full((rows, wide), 0x7F, dtype=torch.uint8, device="cuda")
        t[:, 16:16 + k] = torch.randn(rows, k, generator=gen, device="cuda").to(E4M3).view(torch.uint8)
        ops.append(t[:, 16:16 + k].view(E4M3))
        s = torch.full((parts, -(-k // 128) + 2), float("nan"), device="cuda")
        s[:, 1:-1] = 0.5 + torch.rand(parts, s.shape[1] - 2, generator=gen, device="cuda")
        scales.append(s[:, 1:-1])
    held = torch.full((m + 2, n + 2 * ld), 7.0, device="cuda").to(KINDS[kind])
    y = held[1:-1, ld:n + ld]
    bs.bs_gemm_q8(ops[0], scales[0], ops[1], scales[1], y)
    check(ops[0], scales[0], ops[1], scales[1], y, kind)
    again = torch.empty(m, n, device="cuda").to(KINDS[kind])
    bs.bs_gemm_q8(ops[0], scales[0], ops[1], scales[1], again)
    assert torch.equal(again, y)
    y.fill_(7)
    assert bool((held == 7).all())
