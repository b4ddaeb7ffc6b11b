"""Calls of the row operators on the GPU that are rare in use."""
import itertools
import threading
import time

import numpy as np
import pytest
import torch

import dense_linear_solvers_gb300 as bs

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.rows_ref import EPS  # noqa: E402
from tests.test_gpu_rows import run_norms  # noqa: E402


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


def test_other_threads_run_while_a_launch_waits():
    """A launch behind a full queue waits for the GPU; the other threads of the program do not."""
    f = torch.ones(2, 8, device="cuda")
    y = torch.empty_like(f)
    bs.bs_gnorm_batched(f, y)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    with torch.cuda.stream(stream):
        start.record()
        torch.cuda._sleep(1_500_000_000)  # about 0.8 seconds
        end.record()

    def launch():
        for _ in range(4000):  # more than a queue holds
            bs.bs_gnorm_batched(f, y, stream=stream)

    other = threading.Thread(target=launch)
    longest, last = 0.0, time.perf_counter()
    other.start()
    while other.is_alive():
        time.sleep(0.001)
        now = time.perf_counter()
        longest, last = max(longest, now - last), now
    other.join()
    torch.cuda.synchronize()
    assert longest < 0.4e-3 * start.elapsed_time(end), longest


def test_threads_on_their_own_streams():
    """First calls of an instance from several threads at once, then many more."""
    torch.manual_seed(0)
    data = [torch.randn(2, 300, 4 * 72, device="cuda").half() for _ in range(4)]
    lam = torch.rand(72, device="cuda") * 4 - 5

    def calls(p, stream):
        x, r, i, z = p.split(72, -1)
        with torch.cuda.stream(stream):
            h, y = (torch.empty(2, 300, 72, dtype=p.dtype, device="cuda") for _ in range(2))
            tape = torch.empty(bs.bs_grec_tape_rows(2, 600), 72, device="cuda")
            g, dlam = [torch.empty_like(h) for _ in range(3)], torch.empty_like(lam)
            work = torch.empty(bs.bs_grec_backward_workspace(72, 2, 600), dtype=torch.uint8,
                               device="cuda")
            bs.bs_grec_batched(x, r, i, lam, h, tape=tape)
            bs.bs_gnorm_batched(h, y, z=z)
            bs.bs_grec_backward_batched(x, r, i, lam, tape, y, *g, dlam, work)
            stream.synchronize()
        return [h, y, *g, dlam]

    torch.cuda.synchronize()
    streams, seen = [torch.cuda.Stream() for _ in data], [[] for _ in data]

    def thread(k):
        for _ in range(20):
            seen[k].append(calls(data[k], streams[k]))

    threads = [threading.Thread(target=thread, args=(k,)) for k in range(len(data))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for k, p in enumerate(data):
        want = calls(p, torch.cuda.current_stream())
        assert len(seen[k]) == 20
        for got in seen[k]:
            assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["bf16", "f16"])
@pytest.mark.parametrize("width", [136, 100, 4096, 12000])
@pytest.mark.parametrize("parts", ["".join(p) for n in range(7)
                                   for p in itertools.combinations("zxwcpy", n)
                                   if ("y" in p or "p" in p) and n < 6])
def test_norms_parts_in_16_bits(kind, width, parts):
    """Aligned and unaligned rows, of one warp's part, a block and the looped kernels of the backward
    pass."""
    run_norms(np.random.default_rng(width), kind, 5, width, parts=parts)
