"""Refusals of the gated delta rule, the 8-bit norm output and the 8-bit product on the host: bad arguments
return a status before anything is launched, the Python binding raises on tensors that do not fit (no GPU
needed)."""
import random

import pytest
import torch

import dense_linear_solvers_gb300 as bs
from dense_linear_solvers_gb300 import _build

OK, BAD, NO = bs.BS_OK, bs.BS_ERR_INVALID_ARG, bs.BS_ERR_UNSUPPORTED
M = 0x10000000
P = [0x100000000 + k * M for k in range(24)]  # distinct operands, never dereferenced
HEADS = dict(dtype=bs.BS_BF16, heads_k=2, heads_v=4, dk=64, dv=128)


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return bs.lib()


GIVEN = dict(q=P[0], ldq=128, k=P[1], ldk=128, v=P[2], ldv=512, g=P[3], ldg=4, beta=P[4], ldbeta=4,
             scale=0.1)
FORWARD = dict(HEADS, batch=2, rows=200, offsets=None, **GIVEN, h0=P[5], o=P[6], ldo=512, hT=P[7],
               tape=P[8], work=P[9], work_bytes=M, stream=None)
BACKWARD = dict(HEADS, batch=2, rows=200, offsets=None, **GIVEN, tape=P[8], d_o=P[6], lddo=512, dhT=P[5],
                dq=P[10], lddq=128, d_k=P[11], lddk=128, d_v=P[12], lddv=512, dg=P[13], lddg=4,
                dbeta=P[14], lddbeta=4, dh0=P[15], work=P[9], work_bytes=M, stream=None)
STEP = dict(HEADS, batch=2, **GIVEN, state=P[5], num_slots=5, slots=P[6], o=P[7], ldo=512, stream=None)
NORM = dict(dtype=bs.BS_BF16, rows=9, width=300, f=P[0], ldf=300, z=P[1], ldz=300, x=P[2], ldx=300,
            w_post=P[3], scale=P[4], w_pre=P[5], eps=1e-6, gate=0, y=P[6], ldy=300, q=P[7], ldq=300,
            scales=P[8], lds=3, stream=None)
PRODUCT = dict(dtype=bs.BS_BF16, m=9, n=300, k=256, a=P[0], lda=256, sa=P[1], ldsa=2, w=P[2], ldw=256,
               sw=P[3], ldsw=2, y=P[4], ldy=300, stream=None)


def call(entry, args, **change):
    assert set(change) <= set(args)
    return entry(*{**args, **change}.values())


def test_forward_refusals(lib):
    f = lib.bs_gdelta_batched
    need = bs.bs_gdelta_workspace(4, 2, 200)
    assert call(f, FORWARD, batch=0, rows=0) == OK
    for change in (dict(batch=-1), dict(rows=-1), dict(rows=201), dict(heads_k=-1), dict(heads_v=-4),
                   dict(dk=-1), dict(dv=-1), dict(heads_k=3), dict(ldq=127), dict(ldk=127),
                   dict(ldv=511), dict(ldo=0), dict(ldg=3), dict(ldbeta=-4), dict(scale=float("nan")),
                   dict(scale=float("inf")), dict(scale=1e300), dict(q=None), dict(k=None),
                   dict(v=None), dict(g=None), dict(beta=None), dict(o=None), dict(work=None),
                   dict(work=P[9] + 8), dict(work_bytes=need - 1), dict(tape=P[8] + 8),
                   dict(q=P[0] + 1), dict(o=P[6] + 1), dict(g=P[3] + 2), dict(beta=P[4] + 1),
                   dict(h0=P[5] + 2), dict(hT=P[7] + 2), dict(offsets=P[16] + 4), dict(o=P[0]),
                   dict(o=P[2]), dict(o=P[2] + 256), dict(hT=P[5] + 4), dict(hT=P[6]), dict(tape=P[7]),
                   dict(tape=P[9]), dict(work=P[3]), dict(work=P[0]), dict(offsets=P[6]), dict(g=P[7])):
        assert call(f, FORWARD, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(dtype=9), dict(heads_k=0, heads_v=0), dict(dk=0),
                   dict(dk=129), dict(dv=0), dict(dv=1025, ldv=1 << 14, ldo=1 << 14),
                   dict(heads_v=65536, ldv=1 << 24), dict(ldq=(1 << 21) + 1), dict(batch=1 << 23),
                   dict(rows=(1 << 30) + 2)):
        assert call(f, FORWARD, **change) == NO, change


def test_backward_refusals(lib):
    f = lib.bs_gdelta_backward_batched
    need = bs.bs_gdelta_backward_workspace(4, 64, 128, 2, 200)
    assert need > bs.bs_gdelta_workspace(4, 2, 200) > 0
    assert call(f, BACKWARD, batch=0, rows=0) == OK
    for change in (dict(rows=201), dict(lddo=511), dict(lddq=127), dict(lddk=1), dict(lddv=511),
                   dict(lddg=3), dict(lddbeta=3), dict(scale=float("inf")), dict(d_o=None),
                   dict(dq=None), dict(d_k=None), dict(d_v=None), dict(dg=None), dict(dbeta=None),
                   dict(v=None), dict(tape=None), dict(work=None), dict(work=P[9] + 4),
                   dict(work_bytes=need - 1), dict(tape=P[8] + 4), dict(dq=P[10] + 1),
                   dict(dbeta=P[14] + 2), dict(dh0=P[15] + 1), dict(dhT=P[5] + 2), dict(dq=P[0]),
                   dict(d_k=P[1]), dict(d_v=P[6]), dict(dg=P[3]), dict(dbeta=P[13]), dict(dh0=P[8]),
                   dict(dh0=P[5] + 64), dict(work=P[8]), dict(work=P[5])):
        assert call(f, BACKWARD, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(dk=129), dict(lddv=(1 << 21) + 1)):
        assert call(f, BACKWARD, **change) == NO, change
    # column windows of one matrix may interleave while they are disjoint: another refusal shows which it was
    wide = dict(dq=P[10], lddq=768, d_k=P[10] + 256, lddk=768, d_v=P[10] + 512, lddv=768)
    for change in (dict(wide, d_k=P[10] + 254), dict(wide, d_v=P[10] + 1024), dict(wide, lddk=770)):
        assert call(f, BACKWARD, **change) == BAD, change


def test_step_refusals(lib):
    f = lib.bs_gdelta_step_batched
    assert call(f, STEP, batch=0) == OK
    for change in (dict(batch=-1), dict(num_slots=-1), dict(q=None), dict(o=None), dict(state=None),
                   dict(slots=None, num_slots=1), dict(ldo=511), dict(q=P[0] + 1), dict(state=P[5] + 2),
                   dict(slots=P[6] + 2), dict(o=P[2]), dict(o=P[5]), dict(state=P[0]), dict(state=P[6]),
                   dict(heads_k=3)):
        assert call(f, STEP, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(dk=129), dict(num_slots=(1 << 30) + 1)):
        assert call(f, STEP, **change) == NO, change


def test_norm_refusals(lib):
    f = lib.bs_gnorm_q8_batched
    assert call(f, NORM, rows=0) == OK
    for change in (dict(rows=-1), dict(width=-1), dict(eps=0.0), dict(eps=float("nan")), dict(gate=3),
                   dict(f=None), dict(q=None), dict(scales=None), dict(ldf=299), dict(ldq=299),
                   dict(lds=2), dict(ldy=299), dict(f=P[0] + 1), dict(scales=P[8] + 2),
                   dict(w_pre=P[5] + 1), dict(q=P[0]), dict(q=P[6]), dict(scales=P[7]),
                   dict(scales=P[5]), dict(y=P[0])):
        assert call(f, NORM, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(width=0), dict(width=65537, ldf=70000, ldz=70000,
                                                               ldx=70000, ldy=70000, ldq=70000, lds=600),
                   dict(ldq=(1 << 21) + 1)):
        assert call(f, NORM, **change) == NO, change


def test_product_refusals(lib):
    f = lib.bs_gemm_q8
    assert call(f, PRODUCT, m=0) == OK and call(f, PRODUCT, n=0) == OK
    for change in (dict(m=-1), dict(n=-1), dict(k=-1), dict(lda=255), dict(lda=264), dict(ldw=264),
                   dict(ldsa=1), dict(ldsw=1), dict(ldy=299), dict(a=None), dict(sa=None), dict(w=None),
                   dict(sw=None), dict(y=None), dict(a=P[0] + 8), dict(w=P[2] + 1), dict(sa=P[1] + 2),
                   dict(sw=P[3] + 1), dict(y=P[4] + 1), dict(y=P[0]), dict(y=P[1]), dict(y=P[2]),
                   dict(y=P[3])):
        assert call(f, PRODUCT, **change) == BAD, change
    for change in (dict(dtype=bs.BS_FP64), dict(m=(1 << 30) + 1), dict(n=(1 << 21) + 1),
                   dict(ldy=(1 << 21) + 1)):
        assert call(f, PRODUCT, **change) == NO, change


def test_queries(lib):
    assert bs.bs_gdelta_workspace(0, 1, 1) == 0 and bs.bs_gdelta_workspace(4, -1, 1) == 0
    assert bs.bs_gdelta_workspace(1 << 10, 1 << 15, 1) == 0
    assert bs.bs_gdelta_tape(4, 129, 64, 1, 1) == 0 and bs.bs_gdelta_tape(4, 64, 0, 1, 1) == 0
    assert bs.bs_gdelta_backward_workspace(4, 64, 64, 1, -1) == 0
    assert bs.bs_gdelta_tape(4, 64, 64, 1, 64) < bs.bs_gdelta_tape(4, 65, 64, 1, 64)
    for dtype, want in ((bs.BS_FP32, 1), (bs.BS_BF16, 1), (bs.BS_FP16, 1), (bs.BS_FP64, 0), (4, 0)):
        assert lib.bs_gdelta_supported(dtype, 2, 4, 64, 128) == want
    assert lib.bs_gdelta_supported(bs.BS_BF16, 3, 4, 64, 128) == 0
    assert lib.bs_gdelta_supported(bs.BS_BF16, 1, 1, 129, 128) == 0


def test_places_do_not_overlap():
    """Sequence s that starts at row a has its chunks at a // 64 + s: ceil(length / 64) of them fit in front of the
    next one's, and the last inside rows // 64 + batch."""
    rng = random.Random(0)
    for _ in range(300):
        cuts = sorted(rng.randrange(3000) for _ in range(rng.randrange(2, 12)))
        end = 0
        for s, (a, b) in enumerate(zip(cuts[:-1], cuts[1:])):
            assert a // 64 + s >= end
            end = a // 64 + s + -(-(b - a) // 64)
        assert end <= cuts[-1] // 64 + len(cuts) - 1


def test_binding_raises(lib):
    """Host tensors, other types and other shapes are refused before the library is called."""
    q, v, g = torch.zeros(2, 10, 2, 8), torch.zeros(2, 10, 4, 6), torch.zeros(2, 10, 4)
    work = torch.zeros(16, dtype=torch.uint8)
    with pytest.raises(ValueError, match="device"):
        bs.bs_gdelta_batched(q, q, v, g, g, v, work)
    with pytest.raises(TypeError, match="unsupported"):
        bs.bs_gdelta_batched(q.double(), q, v, g, g, v, work)
    with pytest.raises(ValueError, match="shape"):
        bs.bs_gdelta_batched(q[0], q[0], v[0], g[0], g[0], v[0], work)
    with pytest.raises(ValueError, match="shape"):
        bs.bs_gdelta_step_batched(q, q, v, g, g, v, v)
    with pytest.raises(ValueError, match="device"):
        bs.bs_gnorm_q8_batched(q[0], q[0], q[0])
    with pytest.raises(ValueError, match="device"):
        bs.bs_gemm_q8(q[0], q[0], q[0], q[0], q[0])
    with pytest.raises((TypeError, AttributeError)):
        bs.bs_gemm_q8(q[0], q[0], q[0], q[0], None)
