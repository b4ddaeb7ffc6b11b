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


def near_ties(rows, width, seed):
    """Values that lie on midpoints of two e4m3 numbers times their block's scale, and one to three steps of
    FP32 beside them."""
    gen = torch.Generator().manual_seed(seed)
    blocks = -(-width // 128)
    top = 0.5 + torch.rand(rows, blocks, 1, generator=gen)
    # halfway between two numbers of three fraction bits, from the subnormal ones up to 240
    exponent = torch.randint(-7, 7, (rows, blocks, 128), generator=gen)
    fraction = torch.randint(0, 8, (rows, blocks, 128), generator=gen) + 0.5
    unit = torch.exp2(exponent.clamp_min(-6).float() - 3)
    middle = unit * (fraction + 8 * (exponent > -7))
    v = middle * (top / 448)
    for _ in range(3):  # up or down a step, or not
        to = torch.randint(-1, 2, v.shape, generator=gen).float()
        v = torch.where(to == 0, v, torch.nextafter(v, to * torch.inf))
    v = torch.where(torch.rand(v.shape, generator=gen) < 0.5, v, -v)
    v[..., 0] = top[..., 0]
    return v.flatten(1)[:, :width].contiguous()


@pytest.mark.parametrize("rows, width, pad", [(300, 128, 0), (40, 4096, 0), (64, 1000, 0), (300, 129, 1), (9, 2051, 1),
                                              (2, 20008, 0)])
def test_numbers_are_quotients(rows, width, pad):
    """scales = max / 448 and q = v / scales, both divisions of FP32, q then to nearest even: to the bit, for
    rows that take vectors, that take elements, and that are longer than a block of threads holds."""
    v = near_ties(rows, width, seed=rows + width)
    wide = torch.zeros(rows, width + 2 * pad)
    wide[:, pad:pad + width] = v
    f = wide.cuda()[:, pad:pad + width]
    blocks = -(-width // 128)
    full = torch.zeros(rows, blocks * 128)
    full[:, :width] = v
    full = full.unflatten(1, (blocks, 128))
    s = full.abs().amax(2) / torch.full((rows, blocks), 448.0)
    want = (full / s[..., None]).flatten(1)[:, :width].to(E4M3)
    q, scales = torch.empty(rows, width, device="cuda").to(E4M3), torch.empty(rows, blocks, device="cuda")
    bs.bs_gnorm_q8_batched(f, q, scales)
    assert torch.equal(scales.cpu(), s)
    assert int((q.cpu().view(torch.uint8) != want.view(torch.uint8)).sum()) == 0


@pytest.mark.parametrize("width, pad", [(256, 0), (256, 1), (70000 // 4, 0)])
def test_numbers_of_blocks_that_are_not_finite(width, pad):
    """Under an infinite scale a finite number is 0 and an infinity no number; under no number everything is none.
    The largest and smallest finite blocks keep their quotients."""
    wide = torch.randn(4, width + 2 * pad, device="cuda")
    f = wide[:, pad:pad + width]
    f[0, 3], f[1, 7] = float("inf"), float("nan")
    f[2] *= 2.0 ** 124
    f[3] *= 2.0 ** -98
    f[2].clamp_(-3e38, 3e38)
    blocks = -(-width // 128)
    q, s = torch.empty(4, width, device="cuda").to(E4M3), torch.empty(4, blocks, device="cuda")
    bs.bs_gnorm_q8_batched(f, q, s)
    got, first = q.cpu().float(), min(width, 128)
    assert s[0, 0] == float("inf") and bool(s[1, 0].isnan())
    assert bool(got[0, 3].isnan()) and bool((got[0, :3] == 0).all()) and bool((got[0, 4:first] == 0).all())
    assert bool(got[1, :first].isnan().all()) and bool(got[:2, 128:].isfinite().all())
    v, by = f.cpu()[2:], s.cpu()[2:].repeat_interleave(128, 1)[:, :width]
    assert torch.equal(got[2:], (v / by).to(E4M3).float())


@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows, width, front, ld", [
    (5, 299, 16, 336), (9, 300, 32, 352), (3, 37, 16, 64), (700, 131, 16, 160), (2, 4093, 16, 4128),  # 16-byte rows
    (6, 130, 3, 139), (3, 2050, 1, 2053),                                                           # any rows
    (2, 17001, 16, 17040)])                                                                         # long ones
def test_norms_write_their_rows_only(kind, rows, width, front, ld):
    """y, the numbers and the scales as windows of matrices that keep what they held on both sides, among them rows
    that end inside a vector of 16 bytes."""
    gen = torch.Generator("cuda").manual_seed(width)
    blocks = -(-width // 128)

    def window(like, n, at, total, fill):
        wide = torch.full((rows, total), fill, device="cuda").to(like)
        return wide, wide[:, at:at + n]

    f, x = (torch.randn(rows, ld, generator=gen, device="cuda").to(kind)[:, front:front + width] for _ in range(2))
    w = 1 + 0.1 * torch.randn(width, generator=gen, device="cuda")
    held_y, y = window(kind, width, front, ld, 7.0)
    held_q, q = window(torch.uint8, width, front, ld, 99)
    held_s, s = window(torch.float32, blocks, 2, blocks + 5, 7.0)
    q = q.view(E4M3)
    bs.bs_gnorm_q8_batched(f, q, s, y=y, x=x, w_pre=w)
    for held, n, at, fill in ((held_y, width, front, 7), (held_q, width, front, 99), (held_s, blocks, 2, 7)):
        assert bool((held[:, :at] == fill).all()) and bool((held[:, at + n:] == fill).all())
    # and right ones: half a step of e4m3 (or half its smallest number) around values whose sums and products in FP32
    # are off by far less than 2^-18 of themselves
    v = f.double() + x.double()
    assert bool(((y.double() - v).abs() <= torch.finfo(kind).eps / 2 * v.abs() + 2.0 ** -23 * v.abs()).all())
    v = v * torch.rsqrt((v ** 2).mean(1, keepdim=True) + 1e-6) * w.double()
    by = s.double().repeat_interleave(128, 1)[:, :width]
    far = (q.float().double() * by - v).abs()
    assert bool((far <= (2.0 ** -4 + 2.0 ** -17) * v.abs() + 2.0 ** -10 * by).all())


def test_rows_of_an_odd_width():
    """A contiguous tensor's are refused with the reason; columns of a wider one are taken, straight from the norm."""
    width, n = 1000, 40
    f, w = torch.randn(9, width, device="cuda"), torch.randn(n, 1008, device="cuda").to(E4M3)[:, :width]
    s, sw, y = torch.empty(9, 8, device="cuda"), torch.ones(1, 8, device="cuda"), torch.empty(9, n, device="cuda")
    q = torch.empty(9, width, device="cuda").to(E4M3)
    with pytest.raises(ValueError, match="a: rows 1000 bytes apart"):
        bs.bs_gemm_q8(q, s, w, sw, y)
    wide = torch.empty(9, -(-width // 16) * 16, dtype=E4M3, device="cuda")[:, :width]
    with pytest.raises(ValueError, match="w: rows 1000 bytes apart"):
        bs.bs_gemm_q8(wide, s, w.float().contiguous().to(E4M3), sw, y)
    bs.bs_gnorm_q8_batched(f, wide, s)
    bs.bs_gemm_q8(wide, s, w, sw, y)
    want = (wide.float().double() * s.double().repeat_interleave(128, 1)[:, :width]) @ w.float().double().T
    assert float((y - want).norm() / want.norm()) <= 2.0 ** -20  # a few FP32 roundings of independent terms
