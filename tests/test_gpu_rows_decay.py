"""Channels of the recurrence that forget quickly, on the GPU: a decay far below one keeps its digits, in
the states that are handed on and in every gradient that they reach.

The rows' inputs are zero, so that a state is the initial one times the decays in front of it and every
gradient a sum of positive products: errors are relative. One decay e^-t of t = rate sigma(r) carries
t times t's own relative error, as in tests/rows_ref.py (8 + 2 |r| operations' EPS for the logistic
function, four more for the rate and the product), and at most four EPS of its own operations and of the
product it goes into. What lies in a channel's products is at most the sum of that over its rows;
besides come the operations of a gradient's own factors and the order of a sum over rows."""
import numpy as np
import pytest
import torch

import dense_linear_solvers_gb300 as bs
from tests.rows_ref import EPS, Recurrence, rounded

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def near(got, want, relative, kind, what):
    off = np.abs(got.double().cpu().numpy().reshape(want.shape) - want)
    most = rounded(want, relative * np.abs(want), kind)
    bad = ~(off <= most)
    assert not bad.any(), (what, int(bad.sum()), bad.size, float((off / most).max()))


def exact(v, kind="f32"):
    return torch.from_numpy(v).to(DT[kind]).double().numpy()


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("length,channels", [(1, 130), (3, 130), (200, 96), (1100, 65)])
def test_quick_decays_keep_their_digits(kind, length, channels):
    """Up to three rows of a sequence forget (t up to 22 each), the others hand on what they get."""
    rng = np.random.default_rng(length)
    batch, rows = 3, 3 * length
    lam = exact(rng.uniform(1.0, 3.0, channels))
    r = np.full((batch, length, channels), -30.0)
    for t in sorted({0, length // 2, length - 1}):
        r[:, t] = rng.uniform(-1.5, 1.5, (batch, channels))
    r = exact(r, kind).reshape(rows, channels)
    i = exact(rng.standard_normal((rows, channels)), kind)
    x = np.zeros((rows, channels))
    h0 = exact(rng.uniform(0.5, 2.0, (batch, channels)))
    dh = np.zeros((rows, channels))
    dT = exact(rng.uniform(0.5, 2.0, (batch, channels)))
    spans = [(b * length, (b + 1) * length) for b in range(batch)]
    ref = Recurrence(x, r, i, lam, 8.0, spans, h0).backward(dh, dT)
    t = -ref.l
    own = EPS * (4 + (12 + 2 * np.abs(r)) * t)
    of = own.reshape(batch, length, channels).sum(1)             # of a sequence's products
    over = (rows + 8) * 2.0 ** -24                               # the sum over rows

    def put(v):
        return torch.from_numpy(v).to(DT[kind]).cuda().view(batch, length, channels)

    def f32(v):
        return torch.from_numpy(v).float().cuda()

    tx, tr, ti, tdh = (put(v) for v in (x, r, i, dh))
    h, dx, dr, di = (torch.empty_like(tx) for _ in range(4))
    hT, dh0 = torch.empty(batch, channels, device="cuda"), torch.empty(batch, channels, device="cuda")
    dlam = torch.empty(channels, device="cuda")
    tape = torch.empty(bs.bs_grec_tape_rows(batch, rows), channels, device="cuda")
    work = torch.empty(bs.bs_grec_backward_workspace(channels, batch, rows), dtype=torch.uint8,
                       device="cuda")
    bs.bs_grec_batched(tx, tr, ti, f32(lam), h, h0=f32(h0), hT=hT, tape=tape)
    bs.bs_grec_backward_batched(tx, tr, ti, f32(lam), tape, tdh, dx, dr, di, dlam, work,
                                dhT=f32(dT), dh0=dh0)
    near(hT, ref.hT, of + 4 * EPS, "f32", "hT")
    near(h, ref.h, np.repeat(of, length, 0) + 4 * EPS, kind, "h")
    near(dh0, ref.dh0, of + 4 * EPS, "f32", "dh0")
    # a row's factors beside the products: t, and 1 - sigma(r) for dr
    rest = np.repeat(of, length, 0) + EPS * (32 + 4 * np.abs(r))
    near(dr, ref.dr, rest, kind, "dr")
    near(dlam, ref.dlam, rest.max(0) + over + 16 * EPS, "f32", "dlam")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_a_step_keeps_the_digits_of_a_quick_decay(kind):
    rng = np.random.default_rng(2)
    batch, channels = 9, 130
    lam = exact(rng.uniform(1.0, 3.0, channels))
    r = exact(rng.uniform(-1.5, 1.5, (batch, channels)), kind)
    state = exact(rng.uniform(0.5, 2.0, (batch, channels)))
    zero = np.zeros((batch, channels))
    ref = Recurrence(zero, r, zero, lam, 8.0, [(b, b + 1) for b in range(batch)], state)
    put = lambda v, k: torch.from_numpy(v).to(DT[k]).cuda()  # noqa: E731
    s, y = put(state, "f32"), torch.empty(batch, channels, dtype=DT[kind], device="cuda")
    bs.bs_grec_step_batched(put(zero, kind), put(r, kind), put(zero, kind), put(lam, "f32"), s, y)
    own = EPS * (8 + (12 + 2 * np.abs(r)) * -ref.l)
    near(s, ref.hT, own, "f32", "state")
    near(y, ref.h, own, kind, "y")
