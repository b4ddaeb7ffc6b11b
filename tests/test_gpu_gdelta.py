"""The gated delta rule on the GPU against its definition in 64 bits: whole sequences and single rows."""
import pytest
import torch

import dense_linear_solvers_gb300 as bs

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

from tests.gdelta_ref import Delta  # noqa: E402

KINDS = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


def inputs(kind, rows, hk, hv, dk, dv, seed=0, pad=0, rate=1.0):
    """q, k of length one, v, g, beta; q, k, v as windows of one matrix with `pad` columns more."""
    gen = torch.Generator("cuda").manual_seed(seed)
    new = lambda *s: torch.randn(*s, generator=gen, device="cuda")  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)               # noqa: E731
    wide = torch.full((rows, 2 * hk * dk + hv * dv + pad), float("nan"), device="cuda").to(KINDS[kind])
    at = pad // 2
    out = []
    for t in (unit(new(rows, hk, dk)), unit(new(rows, hk, dk) + new(hk, dk)), new(rows, hv, dv)):
        n = t[0].numel() if rows else t.shape[1] * t.shape[2]
        wide[:, at:at + n] = t.flatten(1)
        out.append(wide[:, at:at + n].unflatten(1, t.shape[1:]))
        at += n
    g = -rate * torch.rand(rows, hv, generator=gen, device="cuda") ** 3
    return (*out, g, torch.sigmoid(new(rows, hv)))


def forward(q, k, v, g, beta, batch, offsets=None, **more):
    rows = q.shape[0]
    o = torch.full(v.shape, 7.0, device="cuda").to(v.dtype)
    work = torch.empty(bs.bs_gdelta_workspace(v.shape[1], batch, rows), dtype=torch.uint8, device="cuda")
    as_given = (lambda t: t) if offsets is not None else (lambda t: t.unflatten(0, (batch, -1)))  # noqa: E731
    bs.bs_gdelta_batched(*(as_given(t) for t in (q, k, v, g, beta, o)), work, offsets=offsets, **more)
    return o


def backward(x, tape, do, batch, offsets=None, dhT=None, dh0=None, into=None, **more):
    """dq, dk, dv, dg, dbeta; into: given outputs."""
    q, v = x[0], x[2]
    out = into or [torch.full(t.shape, 7.0, device="cuda").to(t.dtype) for t in x]
    work = torch.empty(bs.bs_gdelta_backward_workspace(v.shape[1], q.shape[2], v.shape[2], batch,
                                                       q.shape[0]), dtype=torch.uint8, device="cuda")
    as_given = (lambda t: t) if offsets is not None else (lambda t: t.unflatten(0, (batch, -1)))  # noqa: E731
    bs.bs_gdelta_backward_batched(*(as_given(t) for t in x), tape, as_given(do),
                                  *(as_given(t) for t in out), work, dhT=dhT, dh0=dh0, offsets=offsets,
                                  **more)
    return dict(zip(("dq", "dk", "dv", "dg", "dbeta"), out))


def tape_of(x, batch):
    return torch.empty(bs.bs_gdelta_tape(x[2].shape[1], x[0].shape[2], x[2].shape[2], batch,
                                         x[0].shape[0]), dtype=torch.uint8, device="cuda")


def check_gradients(ref, got, kind):
    for name, t in got.items():
        ok, worst = ref.close(name, t, kind if name in ("dq", "dk", "dv") else torch.float32)
        assert ok, (name, worst)


def reference(q, k, v, g, beta, spans, **more):
    return Delta(*(t.double() for t in (q, k, v, g, beta)), spans, **more)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch, length, hk, hv, dk, dv, pad", [
    (1, 1, 1, 1, 64, 64, 0), (2, 63, 1, 2, 64, 64, 16), (2, 64, 2, 2, 128, 128, 0),
    (1, 65, 1, 3, 128, 256, 8), (3, 130, 2, 4, 93, 77, 0), (1, 200, 1, 1, 128, 16, 3),
    (2, 70, 1, 1, 1, 1, 0), (1, 300, 1, 2, 40, 1024, 0), (40, 64, 4, 4, 64, 48, 0)])
def test_forward(kind, batch, length, hk, hv, dk, dv, pad):
    x = inputs(kind, batch * length, hk, hv, dk, dv, pad=pad)
    h0 = torch.randn(batch, hv, dk, dv, device="cuda")
    hT = torch.empty_like(h0)
    o = forward(*x, batch, h0=h0, hT=hT)
    spans = [(b * length, (b + 1) * length) for b in range(batch)]
    ref = reference(*x, spans, h0=h0.double())
    assert ref.close("o", o, KINDS[kind])[0], ref.close("o", o, KINDS[kind])
    assert ref.close("hT", hT, torch.float32)[0], ref.close("hT", hT, torch.float32)
    # without a state in, and with the state updated in place
    again = forward(*x, batch, scale=0.7)
    ref = reference(*x, spans, scale=0.7)
    assert ref.close("o", again, KINDS[kind])[0]
    state = h0.clone()
    assert torch.equal(forward(*x, batch, h0=state, hT=state), o) and torch.equal(state, hT)


@pytest.mark.parametrize("kind, hk, hv, dk, dv", [("bf16", 2, 4, 128, 128), ("f16", 1, 3, 64, 72),
                                                  ("f32", 2, 2, 51, 33)])
def test_packed(kind, hk, hv, dk, dv):
    """Uneven sequences, empty ones, rows in front of the first and behind the last: those keep what
    was there, and what is read is not theirs."""
    cuts = [5, 5, 6, 70, 134, 134, 400, 463, 591]
    x = inputs(kind, 600, hk, hv, dk, dv, seed=1)
    for t in x:
        t[:5], t[591:] = float("nan"), float("nan")
    offsets = torch.tensor(cuts, device="cuda")
    h0 = torch.randn(len(cuts) - 1, hv, dk, dv, device="cuda")
    hT = torch.empty_like(h0)
    o = forward(*x, len(cuts) - 1, offsets, h0=h0, hT=hT)
    spans = list(zip(cuts[:-1], cuts[1:]))
    ref = reference(*x, spans, h0=h0.double())
    assert bool((o[:5] == 7).all()) and bool((o[591:] == 7).all())
    o[:5], o[591:] = 0, 0
    assert ref.close("o", o, KINDS[kind])[0], ref.close("o", o, KINDS[kind])
    assert ref.close("hT", hT, torch.float32)[0], ref.close("hT", hT, torch.float32)
    assert torch.equal(hT[0], h0[0]) and torch.equal(hT[4], h0[4])


@pytest.mark.parametrize("batch", [1, 33, 100, 300])
def test_many_packed(batch):
    """Places of chunks are looked up among many sequences; longest first up to a block's threads."""
    gen = torch.Generator().manual_seed(batch)
    lens = torch.randint(0, 140, (batch,), generator=gen)
    cuts = [0, *torch.cumsum(lens, 0).tolist()]
    x = inputs("bf16", cuts[-1], 1, 1, 64, 64, seed=2)
    hT = torch.empty(batch, 1, 64, 64, device="cuda")
    o = forward(*x, batch, torch.tensor(cuts, device="cuda"), hT=hT)
    ref = reference(*x, list(zip(cuts[:-1], cuts[1:])))
    assert ref.close("o", o, torch.bfloat16)[0]
    assert ref.close("hT", hT, torch.float32)[0]


def test_strong_decays_and_resets():
    """Decays far below one lose nothing of the rows behind them; g = -infinity forgets the state."""
    q, k, v, g, beta = inputs("f32", 256, 1, 2, 64, 32, seed=3)
    g[::7] *= 400
    g[40, 0] = -3e4
    g[100, 1] = float("-inf")
    g[101:130] = -1e-5
    o = forward(q, k, v, g, beta, 1)
    ref = reference(q, k, v, g, beta, [(0, 256)])
    ok, worst = ref.close("o", o, torch.float32)
    assert ok, worst
    fresh = forward(q[100:], k[100:], v[100:], g[100:], beta[100:], 1)
    ref = reference(q[100:], k[100:], v[100:], g[100:], beta[100:], [(0, 156)])
    assert ref.close("o", torch.cat([fresh[:, :1] * 0 + ref.o[:, :1].float(), o[100:, 1:]], 1),
                     torch.float32)[0]


def test_equal_keys():
    """The worst system: every key of a chunk the same, beta 1. Each row replaces what the last wrote."""
    q, k, v, g, beta = inputs("f32", 200, 1, 1, 64, 64, seed=4)
    k[:], g[:], beta[:] = k[:1].clone(), 0.0, 1.0
    o = forward(q, k, v, g, beta, 1)
    ref = reference(q, k, v, g, beta, [(0, 200)])
    assert ref.close("o", o, torch.float32)[0], ref.close("o", o, torch.float32)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_what_is_not_finite_stays_in_its_head(bad):
    x = inputs("bf16", 3 * 130, 2, 4, 64, 64, seed=5)
    want = forward(*x, 3)
    x[2][130 + 70, 1, 3] = bad
    o = forward(*x, 3)
    other = torch.ones(390, 4, dtype=torch.bool, device="cuda")
    other[130 + 64:260, 1] = False
    assert torch.equal(o[other], want[other])
    assert not bool(o[130 + 70, 1].isfinite().all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch, slots, hk, hv, dk, dv", [
    (1, 1, 1, 1, 128, 128), (3, 7, 2, 4, 128, 128), (40, 41, 4, 16, 64, 72), (5, 5, 1, 2, 93, 77),
    (2, 3, 1, 1, 1, 1), (2, 2, 1, 2, 100, 1024), (1, 2, 3, 6, 16, 30)])
def test_step(kind, batch, slots, hk, hv, dk, dv):
    q, k, v, g, beta = inputs(kind, batch, hk, hv, dk, dv, seed=6, pad=5 if dk == 93 else 0)
    pool = torch.randn(slots, hv, dk, dv, device="cuda")
    at = torch.randperm(slots, generator=torch.Generator().manual_seed(1))[:batch].to("cuda", torch.int32)
    state, o = pool.clone(), torch.empty(batch, hv, dv, device="cuda").to(KINDS[kind])
    bs.bs_gdelta_step_batched(q, k, v, g, beta, state, o, slots=at)
    ref = reference(q, k, v, g, beta, [(b, b + 1) for b in range(batch)], h0=pool[at.long()].double())
    assert ref.close("o", o, KINDS[kind])[0], ref.close("o", o, KINDS[kind])
    assert ref.close("hT", state[at.long()], torch.float32)[0]
    kept = torch.ones(slots, dtype=torch.bool, device="cuda")
    kept[at.long()] = False
    assert torch.equal(state[kept], pool[kept])
    # row j with entry j
    state = pool[at.long()].clone()
    again = torch.empty_like(o)
    bs.bs_gdelta_step_batched(q, k, v, g, beta, state, again)
    assert torch.equal(again, o)
    # entries outside the pool
    at[0] = slots if batch % 2 else -1
    state = pool.clone()
    bs.bs_gdelta_step_batched(q, k, v, g, beta, state, again, slots=at)
    assert bool((again[0] == 0).all()) and torch.equal(again[1:], o[1:])


def test_steps_continue_a_sequence():
    """A prompt, then its next rows one by one, against the whole sequence."""
    x = inputs("f32", 2 * 150, 2, 4, 64, 96, seed=7)
    parts = [t.unflatten(0, (2, 150)) for t in x]
    state = torch.empty(2, 4, 64, 96, device="cuda")
    whole = torch.empty_like(state)
    o = forward(*x, 2, hT=whole).unflatten(0, (2, 150))
    forward(*(t[:, :100].flatten(0, 1) for t in parts), 2, hT=state)
    spans = [(0, 150), (150, 300)]
    ref = reference(*x, spans)
    got = o.clone()
    for t in range(100, 150):
        y = torch.empty(2, 4, 96, device="cuda")
        bs.bs_gdelta_step_batched(*(p[:, t] for p in parts), state, y)
        got[:, t] = y
    assert ref.close("o", got.flatten(0, 1), torch.float32)[0]
    assert ref.close("hT", state, torch.float32)[0]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("batch, length, hk, hv, dk, dv, pad", [
    (1, 1, 1, 1, 64, 64, 0), (2, 64, 1, 2, 64, 64, 16), (1, 65, 1, 1, 128, 128, 0),
    (2, 130, 2, 4, 93, 77, 0), (1, 200, 1, 3, 128, 24, 3), (2, 70, 1, 1, 1, 1, 0),
    (1, 100, 1, 2, 40, 300, 0), (3, 191, 2, 2, 64, 48, 8)])
def test_gradients(kind, batch, length, hk, hv, dk, dv, pad):
    x = inputs(kind, batch * length, hk, hv, dk, dv, seed=8, pad=pad)
    do = torch.randn(batch * length, hv, dv, device="cuda").to(KINDS[kind])
    h0, dhT = (torch.randn(batch, hv, dk, dv, device="cuda") for _ in range(2))
    tape, dh0 = tape_of(x, batch), torch.empty_like(h0)
    o = forward(*x, batch, h0=h0, tape=tape)
    assert torch.equal(o, forward(*x, batch, h0=h0))
    got = backward(x, tape, do, batch, dhT=dhT, dh0=dh0)
    spans = [(b * length, (b + 1) * length) for b in range(batch)]
    ref = reference(*x, spans, h0=h0.double()).backward(do.double(), dhT.double())
    check_gradients(ref, dict(got, dh0=dh0), KINDS[kind])
    # the same bits again; the final states' gradient overwritten in place; none given
    state = dhT.clone()
    again = backward(x, tape, do, batch, dhT=state, dh0=state)
    assert all(torch.equal(again[n], got[n]) for n in got) and torch.equal(state, dh0)
    none = backward(x, tape, do, batch)
    check_gradients(reference(*x, spans, h0=h0.double()).backward(do.double()), none, KINDS[kind])


@pytest.mark.parametrize("kind, hk, hv, dk, dv", [("bf16", 2, 4, 128, 128), ("f16", 1, 3, 64, 72),
                                                  ("f32", 1, 2, 51, 33)])
def test_packed_gradients(kind, hk, hv, dk, dv):
    """Into column windows of one matrix; rows of no sequence keep what was there."""
    cuts = [5, 5, 6, 70, 134, 134, 400, 463]
    x = inputs(kind, 470, hk, hv, dk, dv, seed=9)
    for t in x:
        t[:5], t[463:] = float("nan"), float("nan")
    batch, offsets = len(cuts) - 1, torch.tensor(cuts, device="cuda")
    do = torch.randn(470, hv, dv, device="cuda").to(KINDS[kind])
    do[:5], do[463:] = float("nan"), float("nan")
    tape = tape_of(x, batch)
    forward(*x, batch, offsets, tape=tape)
    wide = torch.full((470, 2 * hk * dk + hv * dv), 7.0, device="cuda").to(KINDS[kind])
    parts = [p.unflatten(1, t.shape[1:]) for p, t in zip(wide.split([hk * dk, hk * dk, hv * dv], 1), x)]
    parts += [torch.full((470, hv), 7.0, device="cuda") for _ in range(2)]
    dhT, dh0 = torch.randn(batch, hv, dk, dv, device="cuda"), torch.empty(batch, hv, dk, dv, device="cuda")
    got = backward(x, tape, do, batch, offsets, dhT=dhT, dh0=dh0, into=parts)
    ref = reference(*x, list(zip(cuts[:-1], cuts[1:]))).backward(do.double(), dhT.double())
    for t in parts:
        assert bool((t[:5] == 7).all()) and bool((t[463:] == 7).all())
        t[:5], t[463:] = 0, 0
    check_gradients(ref, dict(got, dh0=dh0), KINDS[kind])
    assert torch.equal(dh0[0], dhT[0]) and torch.equal(dh0[4], dhT[4])


def test_gradients_of_strong_decays_and_idle_rows():
    """Resets, rows that write nothing (beta = 0: dbeta is what they would have written) and rates of 2."""
    x = inputs("f32", 200, 1, 2, 64, 32, seed=10)
    x[3][50, 0], x[3][90, 1], x[3][::9] = float("-inf"), -500.0, -3.0
    x[4][30:40], x[4][120:125] = 0.0, 2.0
    do = torch.randn(200, 2, 32, device="cuda")
    tape = tape_of(x, 1)
    forward(*x, 1, tape=tape)
    got = backward(x, tape, do, 1)
    check_gradients(reference(*x, [(0, 200)]).backward(do.double()), got, torch.float32)


def test_gradients_against_differences():
    """Central differences of the 64-bit forward pass, to which the 64-bit gradients are held too."""
    x = inputs("f32", 67, 1, 2, 8, 5, seed=11)
    do = torch.randn(67, 2, 5, device="cuda")
    tape = tape_of(x, 1)
    forward(*x, 1, tape=tape)
    got = backward(x, tape, do, 1)
    gen = torch.Generator("cuda").manual_seed(1)
    wide = [t.double() for t in x]
    for n, name in enumerate(("dq", "dk", "dv", "dg", "dbeta")):
        way = torch.randn(x[n].shape, generator=gen, device="cuda", dtype=torch.float64)
        step, ends = 1e-5, []
        for sign in (1, -1):
            moved = [t + sign * step * way if m == n else t for m, t in enumerate(wide)]
            ends.append((Delta(*moved, [(0, 67)]).o * do.double()).sum())
        slope = (ends[0] - ends[1]) / (2 * step)
        ref = (got[name].double() * way).sum()
        # the quotient is good to step^2; the gradients to 2^-18 of their terms
        assert abs(float(ref - slope)) <= 1e-4 * float((got[name].double().abs() * way.abs()).sum())
