"""Calls of the gated delta rule, the 8-bit norm output and the 8-bit product that are rare in tests and common in
programs: captured and replayed, on several streams, with operands far apart, and one after another as
a layer uses them."""
import pytest
import torch

import dense_linear_solvers_gb300 as bs

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.gdelta_ref import Delta  # noqa: E402
from tests.test_gpu_gdelta import backward, check_gradients, forward, inputs, reference, tape_of  # noqa: E402
from tests.test_gpu_q8 import E4M3, check, quantised  # noqa: E402


def test_captured_training_pass():
    """Forward and backward pass in one graph, replayed on other inputs; twice the same bits."""
    x = inputs("bf16", 2 * 150, 2, 4, 128, 64, seed=1)
    x = [t.clone() for t in x]
    do = torch.randn(300, 4, 64, device="cuda").bfloat16()
    tape, hT, dh0 = tape_of(x, 2), torch.empty(2, 4, 128, 64, device="cuda"), torch.empty(2, 4, 128, 64,
                                                                                          device="cuda")
    forward(*x, 2, hT=hT, tape=tape)  # modules are loaded outside the capture
    backward(x, tape, do, 2, dh0=dh0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = forward(*x, 2, hT=hT, tape=tape)
        got = backward(x, tape, do, 2, dh0=dh0)
    for seed in (2, 3):
        for a, b in zip(x, inputs("bf16", 300, 2, 4, 128, 64, seed=seed)):
            a.copy_(b)
        graph.replay()
        first = [t.clone() for t in (o, hT, dh0, *got.values())]
        ref = reference(*x, [(0, 150), (150, 300)]).backward(do.double())
        assert ref.close("o", o, torch.bfloat16)[0] and ref.close("hT", hT, torch.float32)[0]
        check_gradients(ref, dict(got, dh0=dh0), torch.bfloat16)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(first, (o, hT, dh0, *got.values())))


def test_captured_serving_step():
    """A token's pass: norm, product, one row of the delta rule, norm behind it, product; the state advances
    with every replay."""
    gen = torch.Generator("cuda").manual_seed(5)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    batch, width, hk, hv, d = 3, 256, 1, 2, 128
    x, w_pre = new(batch, width).bfloat16(), 1 + 0.1 * new(width)
    w_in, s_in = new((2 * hk + hv) * d, width).to(E4M3), 0.05 + 0.01 * torch.rand(4, 2, device="cuda")
    w_out, s_out = new(width, hv * d).to(E4M3), 0.05 + 0.01 * torch.rand(2, 2, device="cuda")
    q8, s8 = torch.empty(batch, width, device="cuda").to(E4M3), torch.empty(batch, 2, device="cuda")
    p = torch.empty(batch, (2 * hk + hv) * d, dtype=torch.bfloat16, device="cuda")
    keys = torch.empty(batch, 2 * hk * d, dtype=torch.bfloat16, device="cuda")
    one = torch.full((d,), d ** -0.5, device="cuda")
    g, beta = -torch.rand(batch, hv, generator=gen, device="cuda"), torch.rand(batch, hv, generator=gen,
                                                                              device="cuda")
    state = 0.1 * new(batch, hv, d, d)
    o, z = torch.empty(batch, hv, d, dtype=torch.bfloat16, device="cuda"), new(batch * hv, d).bfloat16()
    r8, t8 = torch.empty(batch * hv, d, device="cuda").to(E4M3), torch.empty(batch * hv, 1, device="cuda")
    w_post = 1 + 0.1 * new(d)
    y = torch.empty(batch, width, dtype=torch.bfloat16, device="cuda")

    def step():
        bs.bs_gnorm_q8_batched(x, q8, s8, w_pre=w_pre)
        bs.bs_gemm_q8(q8, s8, w_in, s_in, p)
        # q and k of length one: the norm over heads of d elements
        bs.bs_gnorm_batched(p[:, :2 * hk * d].reshape(-1, d), keys.view(-1, d), w_post=one)  # rows at one distance
        q, k = keys.view(batch, 2 * hk, d).split(hk, 1)
        bs.bs_gdelta_step_batched(q, k, p[:, 2 * hk * d:].unflatten(1, (hv, d)), g, beta, state, o)
        bs.bs_gnorm_q8_batched(o.view(batch * hv, d), r8, t8, z=z, w_post=w_post)
        bs.bs_gemm_q8(r8.view(batch, hv * d), t8.view(batch, hv), w_out, s_out, y)

    kept = state.clone()
    step()
    state.copy_(kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    state.copy_(kept)
    before = kept.double()
    for _ in range(3):
        graph.replay()
        k = keys.view(batch, 2 * hk, d)
        assert float((k.double().norm(dim=-1) - 1).abs().max()) <= 2.0 ** -7
        check(q8, s8, w_in, s_in, p, "bf16")
        ref = Delta(k[:, :hk].double(), k[:, hk:].double(), p[:, 2 * hk * d:].unflatten(1, (hv, d)).double(),
                    g.double(), beta.double(), [(b, b + 1) for b in range(batch)], h0=before)
        assert ref.close("o", o, torch.bfloat16)[0] and ref.close("hT", state, torch.float32)[0]
        check(r8.view(batch, hv * d), t8.view(batch, hv), w_out, s_out, y, "bf16")
        before = state.double()


def test_streams_side_by_side():
    """Calls on two streams with workspaces of their own do not disturb each other."""
    cases = [inputs("bf16", 400, 1, 4, 64, 64, seed=s) for s in (1, 2)]
    want = [forward(*x, 2) for x in cases]
    a, sa = quantised(torch.randn(200, 512, device="cuda"))
    w, sw = torch.randn(300, 512, device="cuda").to(E4M3), torch.rand(3, 4, device="cuda")
    y = torch.empty(200, 300, device="cuda")
    bs.bs_gemm_q8(a, sa, w, sw, y)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    out = [[], []]
    for _ in range(5):
        for n, s in enumerate(streams):
            with torch.cuda.stream(s):
                out[n].append(forward(*cases[n], 2))
                z = torch.empty_like(y)
                bs.bs_gemm_q8(a, sa, w, sw, z)
                out[n].append(z)
    torch.cuda.synchronize()
    for n in range(2):
        assert all(torch.equal(t, want[n]) for t in out[n][::2])
        assert all(torch.equal(t, y) for t in out[n][1::2])


def test_a_given_stream():
    x = inputs("f32", 100, 1, 1, 32, 16, seed=3)
    want = forward(*x, 1)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    o = torch.empty_like(want)
    work = torch.empty(bs.bs_gdelta_workspace(1, 1, 100), dtype=torch.uint8, device="cuda")
    s.wait_stream(torch.cuda.current_stream())
    bs.bs_gdelta_batched(*(t[None] for t in x), o[None], work, stream=s)
    s.synchronize()
    assert torch.equal(o, want)


def test_rows_beyond_32_bits():
    """Rows 2^21 elements apart: the last ones start behind the 2^31st element."""
    rows, ld = 1100, 1 << 21
    q, k, v, g, beta = inputs("bf16", rows, 1, 1, 64, 64, seed=4)
    wide = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    far = []
    for n, t in enumerate((q, k, v)):
        wide[:, n * 64:(n + 1) * 64] = t.flatten(1)
        far.append(wide[:, n * 64:(n + 1) * 64].unflatten(1, (1, 64)))
    o = wide[:, 192:256].unflatten(1, (1, 64))
    work = torch.empty(bs.bs_gdelta_workspace(1, 1, rows), dtype=torch.uint8, device="cuda")
    tape = tape_of((q, k, v), 1)
    bs.bs_gdelta_batched(*(t[None] for t in far), g[None], beta[None], o[None], work, tape=tape)
    assert torch.equal(o, forward(q, k, v, g, beta, 1))
    do = torch.randn(rows, 1, 64, device="cuda").bfloat16()
    want = backward((q, k, v, g, beta), tape, do, 1)
    into = [wide[:, 256 + 64 * n:320 + 64 * n].unflatten(1, (1, 64)) for n in range(3)]
    into += [torch.empty_like(g), torch.empty_like(beta)]
    got = backward((*far, g, beta), tape, do, 1, into=into)
    assert all(torch.equal(got[n], want[n]) for n in want)
    # the 8-bit calls
    a, sa = quantised(torch.randn(rows, 64, device="cuda"))
    bytes_ = torch.empty(rows, ld, dtype=torch.uint8, device="cuda")
    bytes_[:, :64] = a.view(torch.uint8)
    w, sw = torch.randn(40, 64, device="cuda").to(E4M3), torch.ones(1, 1, device="cuda")
    y, z = torch.empty(rows, 40, device="cuda"), wide[:, 1 << 20:(1 << 20) + 40]
    bs.bs_gemm_q8(a, sa, w, sw, y)
    bs.bs_gemm_q8(bytes_[:, :64].view(E4M3), sa, w, sw, z)
    assert torch.equal(z, y.bfloat16())
    f = wide[:, 512:576]
    f.copy_(v.flatten(1))
    q8, s8 = torch.empty(rows, 64, device="cuda").to(E4M3), torch.empty(rows, 1, device="cuda")
    bs.bs_gnorm_q8_batched(f, q8, s8)
    want8, wants = quantised(v.flatten(1).float())
    # torch divides by a number as a product with its rounded inverse: two half steps from the quotient, the call's
    # own half a step
    assert bool(((s8 - wants).abs() <= 3 * 2.0 ** -24 * wants).all())
    assert float((q8.float() - want8.float()).abs().max()) <= 32  # a step of its largest numbers


def test_one_tensor_as_query_and_key():
    x = inputs("f32", 90, 2, 2, 64, 32, seed=6)
    got = forward(x[1], x[1], *x[2:], 1)
    assert torch.equal(got, forward(x[1].clone(), *x[1:], 1))


def test_a_layer_over_a_prompt_and_its_next_token():
    """Norm, product, delta rule, norm behind it, product over packed prompts; then one token more of each from the
    kept states, in a larger pool."""
    gen = torch.Generator("cuda").manual_seed(7)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    cuts, width, hk, hv, d = [0, 70, 70, 201, 264], 384, 1, 2, 128
    rows, batch = cuts[-1], len(cuts) - 1
    x, w_pre = new(rows, width).bfloat16(), 1 + 0.1 * new(width)
    w, s = new((2 * hk + hv) * d, width).to(E4M3), 0.05 + 0.01 * torch.rand(4, 3, device="cuda")
    q8, s8 = torch.empty(rows, width, device="cuda").to(E4M3), torch.empty(rows, 3, device="cuda")
    p = torch.empty(rows, (2 * hk + hv) * d, dtype=torch.bfloat16, device="cuda")
    bs.bs_gnorm_q8_batched(x, q8, s8, w_pre=w_pre)
    bs.bs_gemm_q8(q8, s8, w, s, p)
    check(q8, s8, w, s, p, "bf16")
    keys = torch.empty(rows, 2 * hk, d, dtype=torch.bfloat16, device="cuda")
    bs.bs_gnorm_batched(p[:, :2 * hk * d].reshape(-1, d), keys.view(-1, d),
                        w_post=torch.full((d,), d ** -0.5, device="cuda"))
    g, beta = -torch.rand(rows, hv, generator=gen, device="cuda"), torch.rand(rows, hv, generator=gen,
                                                                             device="cuda")
    v = p[:, 2 * hk * d:].unflatten(1, (hv, d))
    pool, at = torch.zeros(9, hv, d, d, device="cuda"), torch.tensor([7, 2, 5, 0], device="cuda")
    hT = torch.empty(batch, hv, d, d, device="cuda")
    o = forward(keys[:, :hk], keys[:, hk:], v, g, beta, batch, torch.tensor(cuts, device="cuda"), hT=hT)
    spans = list(zip(cuts[:-1], cuts[1:]))
    ref = reference(keys[:, :hk], keys[:, hk:], v, g, beta, spans)
    assert ref.close("o", o, torch.bfloat16)[0] and ref.close("hT", hT, torch.float32)[0]
    pool[at] = hT
    token = [t[:batch].contiguous() for t in (keys[:, :hk], keys[:, hk:], v, g, beta)]
    y = torch.empty(batch, hv, d, dtype=torch.bfloat16, device="cuda")
    bs.bs_gdelta_step_batched(*token, pool, y, slots=at.to(torch.int32))
    ref = reference(*token, [(b, b + 1) for b in range(batch)], h0=hT.double())
    assert ref.close("o", y, torch.bfloat16)[0] and ref.close("hT", pool[at], torch.float32)[0]


@pytest.mark.parametrize("m, n, k", [(1, 40, 100), (1, 1, 7), (3, 1, 100), (1, 300, 129), (70, 1, 1)])
def test_single_rows_of_any_depth(m, n, k):
    """A single row of an operand has no distance to a next one that could be a wrong one."""
    deep = -(-k // 16) * 16
    new = lambda rows: torch.randn(rows, deep, device="cuda").to(E4M3)[:, :k]  # noqa: E731
    a, w = (new(r) if r > 1 else torch.randn(1, k, device="cuda").to(E4M3) for r in (m, n))
    sa, sw = (torch.rand(r, -(-k // 128), device="cuda") for r in (m, -(-n // 128)))
    y = torch.empty(m, n, device="cuda")
    bs.bs_gemm_q8(a, sa, w, sw, y)
    check(a, sa, w, sw, y, "f32")
