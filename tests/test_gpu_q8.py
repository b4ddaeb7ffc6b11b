"""The norms' output in 8 bits and the product that reads it, on the GPU against 64 bits."""
import numpy as np
import pytest
import torch

import dense_linear_solvers_gb300 as bs

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.rows_ref import HALF_ULP, Norms, rounded  # noqa: E402

KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF_STEP, SMALL = 2.0 ** -4, 2.0 ** -10   # e4m3: half a step, half the spacing of its smallest numbers
E4M3 = torch.float8_e4m3fn


def host(t):
    return None if t is None else t.double().cpu().numpy()


def window(t, pad, fill=float("nan")):
    """The tensor as columns of a wider one, `pad` of its elements in front."""
    wide = torch.empty(t.shape[0], t.shape[1] + 2 * pad, dtype=t.dtype, device="cuda")
    wide.fill_(fill)
    wide[:, pad:pad + t.shape[1]] = t
    return wide[:, pad:pad + t.shape[1]]


def quantised(v):
    """e4m3 numbers and scales of (rows, width) values, by the definition."""
    rows, width = v.shape
    full = torch.zeros(rows, -(-width // 128) * 128, dtype=torch.float32, device="cuda")
    full[:, :width] = v
    full = full.unflatten(1, (-1, 128))
    s = full.abs().amax(2).clamp_min(2.0 ** -100) / 448
    return (full / s[..., None]).flatten(1)[:, :width].to(E4M3), s


def spread(s, width):
    return np.repeat(s, 128, 1)[:, :width]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows, width, parts, pad", [
    (1, 2048, "zxwcpy", 0), (5, 128, "w", 0), (3, 64, "xpy", 0), (9, 40, "zwy", 0), (4, 1, "p", 0),
    (2, 300, "zxwcpy", 0), (3, 129, "zxwcpy", 3), (6, 7, "cp", 1), (7, 1000, "xp", 0),
    (2, 4419, "zxwcpy", 1), (700, 96, "zwp", 0), (2, 8192, "xwp", 0), (2, 16384, "zxwcpy", 0),
    (3, 16400, "zxwcpy", 0), (1, 20001, "wy", 1), (5, 512, "", 0)])
@pytest.mark.parametrize("gate", [0, 2])
def test_norms(kind, rows, width, parts, pad, gate):
    rng = np.random.default_rng(width)
    dt = KINDS[kind]
    new = lambda *s: torch.from_numpy(rng.standard_normal(s)).float().cuda()  # noqa: E731
    f = window(new(rows, width).to(dt), pad)
    z = window(new(rows, width).to(dt), pad) if "z" in parts else None
    x = window(new(rows, width).to(dt), pad) if "x" in parts else None
    w, c, p = ((1 + 0.1 * new(width)) if k in parts else None for k in "wcp")
    y = window(torch.zeros(rows, width, device="cuda").to(dt), pad, 7.0) if "y" in parts else None
    q = window(torch.zeros(rows, width, device="cuda").to(E4M3).view(torch.uint8), pad, 99).view(E4M3)
    s = window(torch.zeros(rows, -(-width // 128), device="cuda"), pad, 7.0)
    bs.bs_gnorm_q8_batched(f, q, s, y=y, z=z, x=x, w_post=w, scale=c, w_pre=p, gate=gate)
    ref = Norms(host(f), host(z), host(x), host(w), host(c), host(p), gate=gate)
    v, err = (ref.u, ref.err["u"]) if p is not None else (ref.y, ref.err["y"])
    if y is not None:
        assert (np.abs(host(y) - ref.y) <= rounded(ref.y, ref.err["y"], kind)).all()
    blocks = -(-width // 128)
    full = np.zeros((2, rows, blocks * 128))
    full[0, :, :width], full[1, :, :width] = np.abs(v), err
    top, far = full.reshape(2, rows, blocks, 128).max(3)
    # the largest magnitude, a division
    assert (np.abs(host(s) - top / 448) <= far / 448 + 2.0 ** -22 * top / 448).all()
    back = host(q.float()) * spread(host(s), width)
    assert (np.abs(back - v) <= err + (HALF_STEP + 2.0 ** -20) * (np.abs(v) + err)
            + SMALL * spread(host(s), width)).all()
    # nothing around the outputs is written
    if pad:
        assert bool((q._base.view(torch.uint8)[:, :pad] == 99).all()) if q._base is not None else True
        assert bool((s._base[:, :pad] == 7).all()) and bool((s._base[:, -pad:] == 7).all())


def test_zeros_and_what_is_not_finite():
    f = torch.zeros(4, 300, device="cuda")
    f[1, 130], f[2, 5], f[3] = float("nan"), float("inf"), 1e-36
    q, s = torch.empty(4, 300, device="cuda").to(E4M3), torch.empty(4, 3, device="cuda")
    bs.bs_gnorm_q8_batched(f, q, s)
    floor = float(np.float32(2.0 ** -100) / np.float32(448))
    assert bool((q[0].float() == 0).all()) and s[0].tolist() == [floor] * 3
    assert s[1].isnan().tolist() == [False, True, False]
    assert s[2, 0] == float("inf") and s[2, 1:].tolist() == [floor] * 2
    assert s[3].tolist() == [floor] * 3     # 1e-36 is below 2^-100 / 448 / 2^10
    assert bool((q[3].float() == 0).all())


def product(m, n, k, kind="f32", seed=0, ld=0, batch=None):
    gen = torch.Generator("cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    a, sa = quantised(new(m, k)) if m else (new(0, k).to(E4M3), new(0, -(-k // 128)))
    w = new(n, k).to(E4M3)
    sw = 0.5 + torch.rand(-(-n // 128), -(-k // 128), generator=gen, device="cuda")
    if ld:  # rows further apart than they are long
        a, w = (window(t.view(torch.uint8), 16, 0x7F).view(E4M3) for t in (a, w))
        sa, sw = window(sa, 3), window(sw, 1)
    y = torch.full((m, n + 2 * ld), 7.0, device="cuda").to(KINDS[kind])
    y = y[:, ld:n + ld]
    bs.bs_gemm_q8(a, sa, w, sw, y)
    return a, sa, w, sw, y


def check(a, sa, w, sw, y, kind):
    (m, k), n = a.shape, w.shape[0]
    A = a.float().double() * sa.double().repeat_interleave(128, 1)[:, :k]
    W = w.float().double() * sw.double().repeat_interleave(128, 1)[:, :k].repeat_interleave(128, 0)[:n]
    want, size = A @ W.T, A.abs() @ W.abs().T
    # 128 products of a block added in some order, the blocks, two scales; a sum's step is 2^-23 at most
    blocks = -(-k // 128)
    bound = (128 + blocks + 4) * 2.0 ** -23 * size
    bound = bound + HALF_ULP[kind] * (want.abs() + bound) + (2.0 ** -25 if kind == "f16" else 0)
    assert bool(((y.double() - want).abs() <= bound).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("m, n, k, ld", [
    (1, 1, 16, 0), (1, 128, 128, 0), (1, 4096, 2048, 0), (2, 130, 144, 0), (16, 256, 1024, 8), (17, 100, 64, 0),
    (33, 200, 400, 5), (64, 384, 512, 0), (65, 129, 4112, 0), (129, 640, 256, 1), (300, 1000, 1552, 0),
    (515, 300, 96, 0), (1000, 2000, 640, 0), (257, 257, 272, 3), (4100, 128, 128, 0)])
def test_product(kind, m, n, k, ld):
    a, sa, w, sw, y = product(m, n, k, kind, m + n + k, ld)
    check(a, sa, w, sw, y, kind)
    if ld:
        assert bool((y._base[:, :ld] == 7).all()) and bool((y._base[:, -ld:] == 7).all())
    # the same bits every time
    again = torch.empty_like(y)
    bs.bs_gemm_q8(a, sa, w, sw, again)
    assert torch.equal(again, y)


def test_product_of_a_long_depth():
    check(*product(40, 256, 32768 + 48, "f32", 3), "f32")


def test_product_shapes():
    """Rows as (batch, length); no depth; an odd depth with rows 16 bytes apart; no rows."""
    a, sa, w, sw, y = product(12, 200, 256)
    z = torch.empty(3, 4, 200, device="cuda")
    bs.bs_gemm_q8(a.view(3, 4, 256), sa.view(3, 4, 2), w, sw, z)
    assert torch.equal(z.view(12, 200), y)
    short = [t[:, :201] for t in (a, w)]
    bs.bs_gemm_q8(short[0], sa, short[1], sw, y)
    check(short[0], sa, short[1], sw, y, "f32")
    bs.bs_gemm_q8(a[:, :0], sa[:, :0], w[:, :0], sw[:, :0], y)
    assert bool((y == 0).all())
    bs.bs_gemm_q8(a[:0], sa[:0], w, sw, y[:0])


def test_product_keeps_what_is_not_finite_in_its_row():
    a, sa, w, sw, y = product(50, 300, 384, "bf16", 5)
    want = y.clone()
    sa[7, 1], sa[30, 2] = float("nan"), float("inf")
    bs.bs_gemm_q8(a, sa, w, sw, y)
    rows = torch.ones(50, dtype=torch.bool, device="cuda")
    rows[7] = rows[30] = False
    assert torch.equal(y[rows], want[rows])
    assert bool(y[7].isnan().all()) and not bool(y[30].isfinite().any())


@pytest.mark.parametrize("kind", KINDS)
def test_norm_then_product(kind):
    """As a block uses them: the norm's numbers and scales straight into the product."""
    gen = torch.Generator("cuda").manual_seed(1)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    f, x = new(2, 33, 640).to(KINDS[kind]), new(2, 33, 640).to(KINDS[kind])
    w_pre, y = 1 + 0.1 * new(640), torch.empty_like(x)
    q = torch.empty(f.shape, device="cuda").to(E4M3)
    s = torch.empty(2, 33, 5, device="cuda")
    bs.bs_gnorm_q8_batched(f, q, s, y=y, x=x, w_pre=w_pre)
    w, sw = new(256, 640).to(E4M3), 0.5 + torch.rand(2, 5, generator=gen, device="cuda")
    out = torch.empty(2, 33, 256, device="cuda").to(KINDS[kind])
    bs.bs_gemm_q8(q, s, w, sw, out)
    check(q.flatten(0, 1), s.flatten(0, 1), w, sw, out.flatten(0, 1), kind)
    exact = f.double() + x.double()
    exact = exact * torch.rsqrt((exact ** 2).mean(-1, keepdim=True) + 1e-6) * w_pre.double()
    W = w.float().double() * sw.double().repeat_interleave(128, 1).repeat_interleave(128, 0)
    want = exact @ W.T
    # each of 640 products is off by half a step of its 8-bit operand, 2^-4 at most, at random: two thirds
    # of the largest error in the root mean square are more than it can be
    far = (out.double() - want).norm() / (exact.norm(dim=-1, keepdim=True) * W.norm(dim=-1)).norm()
    assert float(far) <= 2.0 ** -4 * 2 / 3
