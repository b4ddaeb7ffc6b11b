"""The row operators' refusals on the host: bad arguments return a status before anything is
launched, the Python binding raises on tensors that do not fit (no GPU needed)."""
import pytest
import torch

import dense_linear_solvers_gb300 as bs
from dense_linear_solvers_gb300 import _build

OK, BAD, NO = bs.BS_OK, bs.BS_ERR_INVALID_ARG, bs.BS_ERR_UNSUPPORTED
M = 0x1000000
P = [0x10000000 + k * M for k in range(24)]  # distinct operands, never dereferenced


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return bs.lib()


FORWARD = dict(dtype=bs.BS_BF16, channels=64, batch=2, rows=200, offsets=None, x=P[0], ldx=64,
               r=P[1], ldr=64, i=P[2], ldi=64, lam=P[3], kappa=8.0, h0=P[4], h=P[5], ldh=64,
               hT=P[6], tape=P[7], stream=None)
BACKWARD = dict(dtype=bs.BS_BF16, channels=64, batch=2, rows=200, offsets=None, x=P[0], ldx=64,
                r=P[1], ldr=64, i=P[2], ldi=64, lam=P[3], kappa=8.0, tape=P[4], dh=P[5], lddh=64,
                dhT=P[6], dx=P[7], lddx=64, dr=P[8], lddr=64, di=P[9], lddi=64, dlam=P[10],
                dh0=P[11], work=P[12], work_bytes=M, stream=None)
STEP = dict(dtype=bs.BS_BF16, channels=64, batch=2, x=P[0], ldx=64, r=P[1], ldr=64, i=P[2],
            ldi=64, lam=P[3], kappa=8.0, state=P[4], num_slots=5, slots=P[5], y=P[6], ldy=64,
            stream=None)
NORM = dict(dtype=bs.BS_BF16, rows=9, width=64, f=P[0], ldf=64, z=P[1], ldz=64, x=P[2], ldx=64,
            w_post=P[3], scale=P[4], w_pre=P[5], eps=1e-6, gate=0, y=P[6], ldy=64, u=P[7], ldu=64,
            stream=None)
NORM_BACK = dict(dtype=bs.BS_BF16, rows=9, width=64, f=P[0], ldf=64, z=P[1], ldz=64, x=P[2],
                 ldx=64, w_post=P[3], scale=P[4], w_pre=P[5], eps=1e-6, gate=0, dy=P[6], lddy=64,
                 du=P[7], lddu=64, df=P[8], lddf=64, dz=P[9], lddz=64, dx=P[10], lddx=64,
                 dw_post=P[11], dscale=P[12], dw_pre=P[13], work=P[14], work_bytes=M, stream=None)


def call(entry, args, **change):
    assert set(change) <= set(args)
    return entry(*{**args, **change}.values())


def test_forward_refusals(lib):
    f = lib.bs_grec_batched
    assert call(f, FORWARD, batch=0, rows=0) == OK
    for change in (dict(batch=-1), dict(rows=-1), dict(channels=-1), dict(rows=201), dict(ldx=63),
                   dict(ldr=63), dict(ldi=0), dict(ldh=-64), dict(kappa=0.0), dict(kappa=-1.0),
                   dict(kappa=float("inf")), dict(kappa=float("nan")), dict(kappa=1e300),
                   dict(x=None), dict(r=None), dict(i=None), dict(h=None), dict(lam=None),
                   dict(x=P[0] + 1), dict(h=P[5] + 1), dict(lam=P[3] + 2), dict(h0=P[4] + 2),
                   dict(hT=P[6] + 1), dict(tape=P[7] + 2), dict(offsets=P[8] + 4),
                   dict(h=P[0]), dict(h=P[0] + 128), dict(hT=P[4] + 4), dict(tape=P[5]),
                   dict(tape=P[6]), dict(hT=P[3]), dict(h0=P[6] + 8), dict(h0=P[5], hT=P[5]),
                   dict(h=P[1], ldh=128), dict(offsets=P[5])):
        assert call(f, FORWARD, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(dtype=9), dict(channels=0),
                   dict(channels=(1 << 20) + 1), dict(ldx=(1 << 21) + 1),
                   dict(batch=1 << 31, rows=1 << 31)):
        assert call(f, FORWARD, **change) == NO, change


def test_windows_of_one_matrix_may_interleave(lib):
    """Outputs as column windows of one wide matrix pass the overlap check while they are
    disjoint; a call with a bad work size behind that check shows which it was."""
    f = lib.bs_grec_backward_batched
    wide = dict(dx=P[7], lddx=192, dr=P[7] + 128, lddr=192, di=P[7] + 256, lddi=192)
    # the inputs' own matrix may hold the gradients of other rows' columns too
    for change, want in ((dict(wide, dr=P[7] + 126), BAD), (dict(wide, di=P[7] + 258), BAD),
                         (dict(wide, lddi=200), BAD), (dict(wide, dr=P[7]), BAD),
                         (dict(wide, x=P[7] + 64, ldx=192), BAD)):
        assert call(f, BACKWARD, **change) == want, change


def test_backward_refusals(lib):
    f = lib.bs_grec_backward_batched
    need = bs.bs_grec_backward_workspace(64, 2, 200)
    assert need > 0
    for change in (dict(batch=-1), dict(rows=201), dict(lddh=63), dict(lddx=1), dict(lddr=63),
                   dict(lddi=63), dict(kappa=0.0), dict(x=None), dict(dh=None), dict(dx=None),
                   dict(dr=None), dict(di=None), dict(dlam=None), dict(lam=None), dict(tape=None),
                   dict(work=None), dict(work=P[12] + 8), dict(work_bytes=need - 1),
                   dict(dh=P[5] + 1), dict(dx=P[7] + 1), dict(dlam=P[10] + 2), dict(dh0=P[11] + 1),
                   dict(dhT=P[6] + 2), dict(dx=P[0]), dict(dx=P[5]), dict(di=P[8]),
                   dict(dlam=P[3]), dict(dh0=P[6]), dict(dh0=P[4]), dict(work=P[4]),
                   dict(work=P[10])):
        assert call(f, BACKWARD, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(channels=0), dict(lddx=(1 << 21) + 1)):
        assert call(f, BACKWARD, **change) == NO, change


def test_step_refusals(lib):
    f = lib.bs_grec_step_batched
    assert call(f, STEP, batch=0) == OK
    for change in (dict(batch=-1), dict(num_slots=-1), dict(kappa=0.0), dict(x=None), dict(y=None),
                   dict(lam=None), dict(state=None), dict(ldy=63), dict(x=P[0] + 1),
                   dict(state=P[4] + 2), dict(slots=P[5] + 2), dict(y=P[0]), dict(y=P[4]),
                   dict(state=P[3]), dict(state=P[5])):
        assert call(f, STEP, **change) == BAD, change
    assert call(f, STEP, dtype=bs.BS_FP64) == NO
    assert call(f, STEP, channels=0) == NO


def test_norm_refusals(lib):
    f = lib.bs_gnorm_batched
    assert call(f, NORM, rows=0) == OK
    for change in (dict(rows=-1), dict(width=-1), dict(eps=0.0), dict(eps=-1.0), dict(eps=1e-60),
                   dict(eps=float("nan")), dict(eps=float("inf")), dict(gate=-1), dict(gate=3),
                   dict(f=None), dict(y=None, u=None, w_pre=None), dict(u=None), dict(w_pre=None),
                   dict(ldf=63), dict(ldz=63), dict(ldx=63), dict(ldy=63), dict(ldu=63),
                   dict(f=P[0] + 1), dict(u=P[7] + 1), dict(w_post=P[3] + 2), dict(y=P[0]),
                   dict(u=P[6]), dict(u=P[2] + 128), dict(y=P[5])):
        assert call(f, NORM, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(width=0), dict(width=65537),
                   dict(ldf=(1 << 21) + 1)):
        assert call(f, NORM, **change) == NO, change


def test_norm_backward_refusals(lib):
    f = lib.bs_gnorm_backward_batched
    need = bs.bs_gnorm_backward_workspace(64, 9)
    assert need > 0
    for change in (dict(rows=-1), dict(width=-2), dict(eps=0.0), dict(gate=7), dict(f=None),
                   dict(df=None), dict(dy=None, du=None, w_pre=None, dw_pre=None), dict(du=None),
                   dict(w_pre=None), dict(z=None), dict(x=None), dict(w_post=None),
                   dict(scale=None), dict(work=None), dict(work=P[14] + 4),
                   dict(work_bytes=need - 1), dict(lddy=63), dict(lddf=63), dict(df=P[8] + 1),
                   dict(dw_pre=P[13] + 2), dict(df=P[0]), dict(dz=P[8]), dict(dx=P[6]),
                   dict(dw_post=P[3]), dict(dscale=P[11]), dict(work=P[5])):
        assert call(f, NORM_BACK, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(width=0), dict(lddz=(1 << 21) + 1)):
        assert call(f, NORM_BACK, **change) == NO, change


def test_queries(lib):
    assert bs.bs_grec_tape_rows(3, 130) == 130 // 32 + 3
    assert bs.bs_grec_tape_rows(-1, 5) == 0
    assert lib.bs_grec_backward_workspace(0, 1, 1) == 0
    assert lib.bs_gnorm_backward_workspace(0, 1) == 0
    for dtype, want in ((bs.BS_FP32, 1), (bs.BS_BF16, 1), (bs.BS_FP16, 1), (bs.BS_FP64, 0), (4, 0)):
        assert lib.bs_grec_supported(dtype, 64) == want
        assert lib.bs_gnorm_supported(dtype, 64) == want
    assert lib.bs_grec_supported(bs.BS_BF16, 0) == 0
    assert lib.bs_gnorm_supported(bs.BS_BF16, 65537) == 0
    # the solvers take neither 16-bit type
    assert lib.bs_getrf_getrs_supported(bs.BS_BF16, 0, 8, 1) == 0
    assert lib.bs_bdsv_supported(bs.BS_FP16, 4, 4) == 0


def test_tape_parts_do_not_overlap():
    """Sequence s that starts at row a has its tape at a // 32 + s: ceil(length / 32) rows fit in front
    of the next one's, and the last inside bs_grec_tape_rows."""
    import random
    rng = random.Random(0)
    for _ in range(200):
        cuts = sorted(rng.randrange(2000) for _ in range(rng.randrange(2, 12)))
        end = 0
        for s, (a, b) in enumerate(zip(cuts[:-1], cuts[1:])):
            base = a // 32 + s
            assert base >= end
            end = base + -(-(b - a) // 32)
        assert end <= bs.bs_grec_tape_rows(len(cuts) - 1, cuts[-1])


def test_binding_raises(lib):
    """Host tensors, other types and other shapes are refused before the library is called."""
    x = torch.zeros(2, 10, 8)
    lam = torch.zeros(8)
    with pytest.raises(ValueError, match="device"):
        bs.bs_grec_batched(x, x, x, lam, x)
    with pytest.raises(ValueError, match="device"):
        bs.bs_gnorm_batched(x, x)
    with pytest.raises(TypeError, match="unsupported"):
        bs.bs_grec_batched(x.double(), x, x, lam, x)
    with pytest.raises(TypeError, match="unsupported"):
        bs.bs_gnorm_batched(x.double(), x)
    with pytest.raises(ValueError, match="shape"):
        bs.bs_gnorm_batched(x[0, 0], x[0, 0])
    with pytest.raises((TypeError, AttributeError)):
        bs.bs_grec_step_batched(None, x[0], x[0], lam, x[0], x[0])
