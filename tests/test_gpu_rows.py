"""The row operators on the GPU against their 64-bit references: types, head and tail sizes, strides,
packed sequences, masked rows, infinities, slots, streams and graphs. Tolerances are the
references' running error bounds (tests/rows_ref.py)."""
import itertools

import numpy as np
import pytest
import torch

import dense_linear_solvers_gb300 as bs
from tests.rows_ref import Norms, Recurrence, rounded

pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
MARK = 77.0  # what stands in every element that no call may write


def window(rows, width, kind, values=None, pad=(0, 0), tail=3):
    """A (rows, width) column window of a wider marked tensor with `tail` rows behind it; pad: the
    columns before and after. Returns (window, whole)."""
    whole = torch.full((rows + tail, pad[0] + width + pad[1]), MARK, dtype=DT[kind], device="cuda")
    w = whole[:rows, pad[0]:pad[0] + width]
    if values is not None:
        w.copy_(torch.from_numpy(np.ascontiguousarray(values)))
    return w, whole


def untouched(w, whole):
    """Whether everything of whole outside the window still holds the mark."""
    keep = whole.clone()
    keep[:w.shape[0], w.storage_offset():w.storage_offset() + w.shape[1]] = MARK
    return bool((keep == MARK).all())


def values(rng, shape, kind, scale=1.0):
    """float64 values that the type holds exactly."""
    v = torch.from_numpy(rng.standard_normal(shape) * scale).to(DT[kind])
    return v.double().numpy()


def f32(v):
    return torch.from_numpy(np.asarray(v, dtype=np.float64)).float().cuda()


def near(got, ref, bound, kind, what, rows=slice(None)):
    g = got.double().cpu().numpy()[rows]
    off, most = np.abs(g - ref[rows]), rounded(ref, bound, kind)[rows]
    bad = ~(off <= most)
    assert not bad.any(), (what, int(bad.sum()), bad.size, np.argwhere(bad)[:3].tolist(),
                           float((off / most).max()))


def run_recurrence(rng, kind, c, spans, rows, *, kappa=8.0, packed=True, h0=True, train=True,
                   pads=((0, 0),) * 4, r=None, lam=None, i=None, inplace=False):
    """Every call of the recurrence on random inputs against the reference."""
    batch = len(spans)
    x, ra, ia = (values(rng, (rows, c), kind) for _ in range(3))
    ra, ia = ra if r is None else r, ia if i is None else i
    la = (rng.uniform(-7, 0, c) if lam is None else lam).astype(np.float32).astype(np.float64)
    start = rng.standard_normal((batch, c)).astype(np.float32).astype(np.float64) if h0 else None
    ref = Recurrence(x, ra, ia, la, kappa, spans, start)
    tx, tr, ti = (window(rows, c, kind, v, p)[0] for v, p in zip((x, ra, ia), pads))
    th, whole = window(rows, c, kind, None, pads[3])
    offsets = torch.tensor([p for p, _ in spans] + [spans[-1][1]], device="cuda") if packed else None

    def shape(t):
        return t if packed else t.unflatten(0, (batch, -1))

    s0 = f32(start) if h0 else None
    hT = s0 if inplace else torch.full((batch, c), MARK, device="cuda")
    tape = torch.full((bs.bs_grec_tape_rows(batch, rows), c), MARK, device="cuda")
    # an operand's window starts at row 0 of its tensor: the rows behind stay out of the call
    bs.bs_grec_batched(shape(tx), shape(tr), shape(ti), f32(la), shape(th), h0=s0, hT=hT,
                       offsets=offsets, tape=tape, kappa=kappa)
    live = np.zeros(rows, bool)
    for p, q in spans:
        live[p:q] = True
    near(th, ref.h, ref.err["h"], kind, "h", live)
    near(hT, ref.hT, ref.err["hT"], "f32", "hT")
    assert untouched(th, whole)
    assert bool((th[torch.from_numpy(~live).cuda()] == MARK).all())
    for b, (p, q) in enumerate(spans):
        for k, t in enumerate(range(p, q, 32)):
            near(tape[p // 32 + b + k], ref.before[t], ref.err_before[t], "f32", "tape")
    if not train:
        return
    dh = values(rng, (rows, c), kind)
    dT = rng.standard_normal((batch, c)).astype(np.float32).astype(np.float64) if h0 else None
    ref.backward(np.where(live[:, None], dh, 0), dT)
    tdh = window(rows, c, kind, dh, pads[1])[0]
    outs = [window(rows, c, kind, None, p) for p in pads[:3]]
    dlam, dh0 = torch.full((c,), MARK, device="cuda"), torch.full((batch, c), MARK, device="cuda")
    work = torch.empty(bs.bs_grec_backward_workspace(c, batch, rows), dtype=torch.uint8,
                       device="cuda")
    bs.bs_grec_backward_batched(
        shape(tx), shape(tr), shape(ti), f32(la), tape, shape(tdh),
        *(shape(w) for w, _ in outs), dlam, work, dhT=None if dT is None else f32(dT),
        dh0=dh0 if h0 else None, offsets=offsets, kappa=kappa)
    for (w, whole), name in zip(outs, ("dx", "dr", "di")):
        near(w, getattr(ref, name), ref.err[name], kind, name, live)
        assert untouched(w, whole) and bool((w[torch.from_numpy(~live).cuda()] == MARK).all())
    near(dlam, ref.dlam, ref.err["dlam"], "f32", "dlam")
    if h0:
        near(dh0, ref.dh0, ref.err["dh0"], "f32", "dh0")


def uniform(batch, length):
    return [(b * length, (b + 1) * length) for b in range(batch)]


# one row, around the tape's 32 rows, several tiles, more than one pass of the largest split
LENGTHS = [1, 2, 15, 16, 17, 63, 64, 65, 127, 130, 257, 700]


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("length", LENGTHS)
def test_recurrence_lengths(kind, length):
    rng = np.random.default_rng(length)
    run_recurrence(rng, kind, 72, uniform(2, length), 2 * length, packed=False)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("channels", [1, 2, 3, 31, 33, 63, 64, 65, 127, 200, 258])
def test_recurrence_channels(kind, channels):
    rng = np.random.default_rng(channels)
    run_recurrence(rng, kind, channels, uniform(3, 70), 210, packed=False)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("pads", [((0, 8), (8, 0), (16, 8), (0, 0)), ((1, 0), (0, 1), (3, 2), (2, 1)),
                                  ((2, 0), (4, 2), (0, 2), (0, 4)), ((0, 0), (0, 0), (1, 0), (0, 0))])
def test_recurrence_strides_and_alignment(kind, pads):
    rng = np.random.default_rng(5)
    run_recurrence(rng, kind, 96, uniform(2, 150), 300, packed=False, pads=pads)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_recurrence_packed(kind):
    """Empty sequences first, last and between, single rows, sequences over several tiles, and
    rows before and behind all sequences that are not touched."""
    rng = np.random.default_rng(6)
    cuts = [3, 3, 4, 90, 90, 90, 91, 300, 364, 1000, 1000]
    run_recurrence(rng, kind, 65, list(zip(cuts[:-1], cuts[1:])), 1011)


@pytest.mark.parametrize("channels,length,batch", [(64, 9000, 1), (40, 4097, 3), (1500, 2500, 1)])
def test_recurrence_long(channels, length, batch):
    """Few channels and a long sequence: the sequence itself is what is split."""
    rng = np.random.default_rng(7)
    run_recurrence(rng, "bf16", channels, uniform(batch, length), batch * length, packed=False)


def test_recurrence_many_sequences():
    rng = np.random.default_rng(8)
    run_recurrence(rng, "bf16", 10, uniform(1500, 5), 7500, packed=False)


@pytest.mark.parametrize("kind,channels", [("bf16", 104), ("bf16", 99), ("f16", 128), ("f32", 100)])
def test_recurrence_many_sequences_of_several_steps(kind, channels):
    """Enough pairs of a sequence and a tile that blocks of four warps take each alone."""
    rng = np.random.default_rng(18)
    run_recurrence(rng, kind, channels, uniform(230, 133), 230 * 133, packed=False)


def test_recurrence_more_sequences_than_a_grid_has_rows():
    rng = np.random.default_rng(19)
    cuts = np.concatenate([[0, 1], np.arange(2, 70001), [70300]])
    run_recurrence(rng, "bf16", 5, list(zip(cuts[:-1].tolist(), cuts[1:].tolist())), 70300)


def test_recurrence_without_states():
    rng = np.random.default_rng(9)
    run_recurrence(rng, "bf16", 64, uniform(2, 100), 200, packed=False, h0=False)


def test_recurrence_state_in_place():
    rng = np.random.default_rng(10)
    run_recurrence(rng, "bf16", 128, uniform(4, 300), 1200, packed=False, inplace=True, train=False)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_recurrence_extreme_gates(kind):
    """Rows whose gates are closed (-inf, the type's lowest value) hand the state on; open gates;
    channels with no decay and with full decay."""
    rng = np.random.default_rng(11)
    rows, c = 200, 64
    lowest = float(torch.finfo(DT[kind]).min)
    r, i = values(rng, (rows, c), kind, 3.0), values(rng, (rows, c), kind, 3.0)
    for k, v in enumerate((-np.inf, lowest, -90.0, -45.0, 90.0, np.inf, -lowest)):
        r[10 + 7 * k], i[11 + 7 * k] = v, v
        r[100 + k, ::2], i[100 + k, 1::3] = v, v
    lam = rng.uniform(-8, 2, c)
    lam[:6] = [-100.0, -30.0, 30.0, 100.0, -15.5, 0.0]
    run_recurrence(rng, kind, c, uniform(1, rows), rows, packed=False, r=r, i=i, lam=lam)


def test_recurrence_closed_rows_hand_the_state_on():
    rng = np.random.default_rng(12)
    c = 70
    x = f32(rng.standard_normal((1, 200, c)))
    shut = torch.full_like(x, -float("inf"))
    h0, h, hT = f32(rng.standard_normal((1, c))), torch.empty_like(x), torch.empty(1, c, device="cuda")
    bs.bs_grec_batched(x, shut, shut, f32(rng.uniform(-5, 0, c)), h, h0=h0, hT=hT)
    assert torch.equal(hT, h0) and torch.equal(h, h0.expand(200, c)[None])


def test_recurrence_nonfinite_values_stay_in_their_channel():
    rng = np.random.default_rng(13)
    rows, c = 600, 66
    base = [values(rng, (rows, c), "bf16") for _ in range(3)]
    la = f32(rng.uniform(-7, 0, c))
    outs = []
    for spoil in (False, True):
        t = [torch.from_numpy(v).to(torch.bfloat16).cuda() for v in base]
        if spoil:
            t[0][250, 5], t[1][260, 9], t[2][270, 33] = float("inf"), float("nan"), float("nan")
        off = torch.tensor([0, 200, 400, 600], device="cuda")
        h, tape = torch.empty_like(t[0]), torch.empty(bs.bs_grec_tape_rows(3, rows), c, device="cuda")
        bs.bs_grec_batched(*t, la, h, offsets=off, tape=tape)
        g = [torch.empty_like(h) for _ in range(3)]
        dlam = torch.empty(c, device="cuda")
        work = torch.empty(bs.bs_grec_backward_workspace(c, 3, rows), dtype=torch.uint8, device="cuda")
        bs.bs_grec_backward_batched(*t, la, tape, torch.ones_like(h), *g, dlam, work, offsets=off)
        outs.append((h, *g))
    for clean, bad in zip(*outs):
        hit = torch.zeros(rows, c, dtype=torch.bool, device="cuda")
        for ch in (5, 9, 33):
            hit[200:400, ch] = True
        assert torch.equal(clean[~hit], bad[~hit])
    h = outs[1][0]
    assert bool(torch.isnan(h[260:400, 9]).all()) and bool(torch.isnan(h[270:400, 33]).all())
    assert not bool(torch.isfinite(h[250:400, 5]).any())
    assert bool(torch.isfinite(h[200:250, 5]).all())


def test_recurrence_offsets_past_32_bits():
    """Rows whose element offsets pass 2^32: windows of one 9 GB tensor."""
    rows, ld, c = 66000, 70000, 3
    need = 2 * rows * ld * 2
    if torch.cuda.mem_get_info()[0] < need + (2 << 30):
        pytest.skip("not enough device memory")
    rng = np.random.default_rng(14)
    whole = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    out = torch.empty(rows, ld, dtype=torch.bfloat16, device="cuda")
    x, r, i = (values(rng, (rows, c), "bf16") for _ in range(3))
    la = rng.uniform(-7, 0, c).astype(np.float32).astype(np.float64)
    w = [whole[:, k:k + c] for k in (8, 40000, 69990)]
    for t, v in zip(w, (x, r, i)):
        t.copy_(torch.from_numpy(v))
    h = out[:, 69000:69000 + c]
    hT = torch.empty(1, c, device="cuda")
    bs.bs_grec_batched(*(t[None] for t in w), f32(la), h[None], hT=hT)
    ref = Recurrence(x, r, i, la, 8.0, [(0, rows)])
    near(h, ref.h, ref.err["h"], "bf16", "h")
    near(hT, ref.hT, ref.err["hT"], "f32", "hT")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("batch,c,pad", [(1, 1, 0), (1, 2048, 0), (3, 65, 0), (17, 200, 3),
                                         (300, 128, 8), (5, 1000, 1),
                                         (6000, 66, 0)])
@pytest.mark.parametrize("slots", [False, True])
def test_step(kind, batch, c, pad, slots):
    rng = np.random.default_rng(batch + c)
    x, r, i = (values(rng, (batch, c), kind) for _ in range(3))
    la = rng.uniform(-7, 0, c).astype(np.float32).astype(np.float64)
    pool = batch + 5 if slots else batch
    st = rng.standard_normal((pool, c)).astype(np.float32).astype(np.float64)
    at = rng.permutation(pool)[:batch].astype(np.int32) if slots else np.arange(batch, dtype=np.int32)
    dead = np.zeros(batch, bool)
    if slots and batch >= 3:
        at[1], at[2] = -1, pool            # outside the pool: skipped
        dead[1:3] = True
    state = f32(st)
    y, whole = window(batch, c, kind, None, (pad, 0))
    ins = [window(batch, c, kind, v, (0, pad))[0] for v in (x, r, i)]
    bs.bs_grec_step_batched(*ins, f32(la), state, y,
                            slots=torch.from_numpy(at).cuda() if slots else None)
    want, bound = st.copy(), np.zeros_like(st)
    live = np.flatnonzero(~dead)
    ref = Recurrence(x, r, i, la, 8.0, [(j, j + 1) for j in range(batch)],
                     st[np.where(dead, 0, at)])
    want[at[live]], bound[at[live]] = ref.hT[live], ref.err["hT"][live]
    near(state, want, bound, "f32", "state")
    near(y, ref.h, ref.err["h"], kind, "y", live)
    assert bool((y[torch.from_numpy(dead).cuda()] == 0).all())
    assert untouched(y, whole)


def test_steps_equal_the_sequence():
    """Token by token from the prompt's final state gives what one call over all rows gives."""
    rng = np.random.default_rng(15)
    c, n = 96, 140
    x, r, i = (torch.from_numpy(values(rng, (1, n, c), "f32")).float().cuda() for _ in range(3))
    la = f32(rng.uniform(-7, 0, c))
    full, hT = torch.empty_like(x), torch.empty(1, c, device="cuda")
    bs.bs_grec_batched(x, r, i, la, full, hT=hT)
    state, part = torch.empty(1, c, device="cuda"), torch.empty(1, 100, c, device="cuda")
    bs.bs_grec_batched(x[:, :100], r[:, :100], i[:, :100], la, part, hT=state)
    y = torch.empty(1, c, device="cuda")
    for t in range(100, n):
        bs.bs_grec_step_batched(x[:, t], r[:, t], i[:, t], la, state, y)
    ref = Recurrence(*(v[0].double().cpu().numpy() for v in (x, r, i)), la.double().cpu().numpy(),
                     8.0, [(0, n)])
    near(state, ref.hT, ref.err["hT"], "f32", "state")
    near(hT, ref.hT, ref.err["hT"], "f32", "hT")


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_recurrence_norm_of_the_error(kind):
    """The worst-case bounds above grow with the memory; the errors themselves are independent roundings.
    A 32-bit result sums up to 1000 rows' errors of 2^-22, which add like their root to 2^-17 of the
    result's norm at most; a stored 16-bit row has its own rounding, uniform in half a unit, of
    at most 2^-8 (2^-11) / sqrt(3), besides."""
    rng = np.random.default_rng(20)
    rows, c = 2000, 256
    x, r, i, dh = (values(rng, (rows, c), kind) for _ in range(4))
    la = rng.uniform(-7, 0, c).astype(np.float32).astype(np.float64)
    start, dT = (rng.standard_normal((2, c)).astype(np.float32).astype(np.float64) for _ in range(2))
    ref = Recurrence(x, r, i, la, 8.0, uniform(2, 1000), start).backward(dh, dT)
    t = [torch.from_numpy(v).to(DT[kind]).cuda().view(2, 1000, c) for v in (x, r, i, dh)]
    out = {k: torch.empty_like(t[0]) for k in ("h", "dx", "dr", "di")}
    out.update({k: torch.empty(2, c, device="cuda") for k in ("hT", "dh0")}, dlam=torch.empty(c, device="cuda"))
    tape = torch.empty(bs.bs_grec_tape_rows(2, rows), c, device="cuda")
    work = torch.empty(bs.bs_grec_backward_workspace(c, 2, rows), dtype=torch.uint8, device="cuda")
    bs.bs_grec_batched(*t[:3], f32(la), out["h"], h0=f32(start), hT=out["hT"], tape=tape)
    bs.bs_grec_backward_batched(*t[:3], f32(la), tape, t[3], out["dx"], out["dr"], out["di"],
                                out["dlam"], work, dhT=f32(dT), dh0=out["dh0"])
    for k, v in out.items():
        want = getattr(ref, k)
        own = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kind] / np.sqrt(3) if v.dim() == 3 else 0.0
        off = np.linalg.norm(v.double().cpu().numpy().reshape(want.shape) - want)
        assert off <= (2.0 ** -17 + own) * np.linalg.norm(want), (k, off / np.linalg.norm(want))


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_norms_norm_of_the_error(kind):
    """As above: 32-bit results sum the rows' or the elements' errors of 2^-22 like their root."""
    rng = np.random.default_rng(21)
    rows, w = 500, 1024
    f, z, x, dy, du = (values(rng, (rows, w), kind) for _ in range(5))
    ws = [(1 + 0.3 * rng.standard_normal(w)).astype(np.float32).astype(np.float64) for _ in range(3)]
    ref = Norms(f, z, x, *ws).backward(dy, du)
    tf, tz, tx, tdy, tdu = (torch.from_numpy(v).to(DT[kind]).cuda() for v in (f, z, x, dy, du))
    vec = [f32(v) for v in ws]
    out = {k: torch.empty_like(tf) for k in ("y", "u", "df", "dz", "dx")}
    out.update({k: torch.empty(w, device="cuda") for k in ("dw_post", "dscale", "dw_pre")})
    bs.bs_gnorm_batched(tf, out["y"], z=tz, x=tx, w_post=vec[0], scale=vec[1], w_pre=vec[2], u=out["u"])
    work = torch.empty(bs.bs_gnorm_backward_workspace(w, rows), dtype=torch.uint8, device="cuda")
    bs.bs_gnorm_backward_batched(
        tf, tdy, out["df"], work, z=tz, x=tx, w_post=vec[0], scale=vec[1], w_pre=vec[2], du=tdu,
        **{k: out[k] for k in ("dz", "dx", "dw_post", "dscale", "dw_pre")})
    for k, v in out.items():
        want = getattr(ref, k)
        own = {"f32": 0.0, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}[kind] / np.sqrt(3) if v.dim() == 2 else 0.0
        off = np.linalg.norm(v.double().cpu().numpy() - want)
        assert off <= (2.0 ** -17 + own) * np.linalg.norm(want), (k, off / np.linalg.norm(want))


def test_recurrence_is_the_same_every_time():
    rng = np.random.default_rng(16)
    c, rows = 520, 5000
    t = [torch.from_numpy(values(rng, (1, rows, c), "bf16")).to(torch.bfloat16).cuda()
         for _ in range(4)]
    la = f32(rng.uniform(-7, 0, c))
    seen = []
    for _ in range(3):
        h, tape = torch.empty_like(t[0]), torch.empty(bs.bs_grec_tape_rows(1, rows), c, device="cuda")
        g, dlam = [torch.empty_like(h) for _ in range(3)], torch.empty(c, device="cuda")
        work = torch.empty(bs.bs_grec_backward_workspace(c, 1, rows), dtype=torch.uint8, device="cuda")
        bs.bs_grec_batched(*t[:3], la, h, tape=tape)
        bs.bs_grec_backward_batched(*t[:3], la, tape, t[3], *g, dlam, work)
        seen.append([h, *g, dlam])
    for other in seen[1:]:
        assert all(torch.equal(a, b) for a, b in zip(seen[0], other))


# ------------------------------------------------------------------------------ norms
def run_norms(rng, kind, rows, width, *, parts="zxwcpy", gate=0, pads=(0, 0), eps=1e-6, f=None):
    has = {k: k in parts for k in "zxwcpy"}
    fv = values(rng, (rows, width), kind) if f is None else f
    zv = values(rng, (rows, width), kind, 2.0) if has["z"] else None
    xv = values(rng, (rows, width), kind, 2.0) if has["x"] else None
    w, c, p = ((1 + 0.3 * rng.standard_normal(width)).astype(np.float32).astype(np.float64)
               if has[k] else None for k in "wcp")
    ref = Norms(fv, zv, xv, w, c, p, eps, gate)

    def put(v):
        return None if v is None else window(rows, width, kind, v, pads)[0]

    def new(flag=True):
        return window(rows, width, kind, None, pads) if flag else (None, None)

    vec = {k: None if v is None else f32(v) for k, v in zip("wcp", (w, c, p))}
    tf, tz, tx = put(fv), put(zv), put(xv)
    (y, wy), (u, wu) = new(has["y"]), new(has["p"])
    bs.bs_gnorm_batched(tf, y, z=tz, x=tx, w_post=vec["w"], scale=vec["c"], w_pre=vec["p"], u=u,
                        eps=eps, gate=gate)
    for t, whole, name in ((y, wy, "y"), (u, wu, "u")):
        if t is not None:
            near(t, getattr(ref, name), ref.err[name], kind, name)
            assert untouched(t, whole)
    dy = values(rng, (rows, width), kind) if has["y"] else None
    du = values(rng, (rows, width), kind) if has["p"] else None
    ref.backward(dy, du)
    outs = {"df": new(), "dz": new(has["z"]), "dx": new(has["x"])}
    sums = {n: torch.full((width,), MARK, device="cuda") if has[k] else None
            for n, k in (("dw_post", "w"), ("dscale", "c"), ("dw_pre", "p"))}
    work = torch.empty(bs.bs_gnorm_backward_workspace(width, rows), dtype=torch.uint8, device="cuda")
    bs.bs_gnorm_backward_batched(
        tf, put(dy), outs["df"][0], work, z=tz, x=tx, w_post=vec["w"], scale=vec["c"],
        w_pre=vec["p"], du=put(du), dz=outs["dz"][0], dx=outs["dx"][0], **sums, eps=eps, gate=gate)
    for name, (t, whole) in outs.items():
        if t is not None:
            near(t, getattr(ref, name), ref.err[name], kind, name)
            assert untouched(t, whole)
    for name, t in sums.items():
        if t is not None:
            near(t, getattr(ref, name), ref.err[name], "f32", name)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("width", [1, 2, 7, 8, 31, 32, 63, 64, 72, 256, 257, 1000, 1024, 2048, 2056,
                                   4096, 5001, 8192, 16384, 20000])
def test_norms_widths(kind, width):
    run_norms(np.random.default_rng(width), kind, 5, width)


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("rows,width", [(1, 64), (1, 4096), (1237, 96), (700, 1024), (3000, 40)])
def test_norms_rows(kind, rows, width):
    run_norms(np.random.default_rng(rows), kind, rows, width)


@pytest.mark.parametrize("kind,rows,width,pads", [
    ("bf16", 5000, 1024, (0, 0)), ("f16", 1500, 4096, (0, 8)), ("f32", 1300, 4096, (0, 0)),
    ("bf16", 700, 8192, (0, 0)), ("bf16", 1400, 4000, (1, 0)), ("f32", 2600, 1001, (0, 0)),
    ("f16", 40001, 64, (0, 0)), ("bf16", 30011, 100, (0, 4)), ("bf16", 400, 17000, (0, 0))])
def test_norms_more_rows_than_blocks_hold(kind, rows, width, pads):
    """Blocks walk several turns of rows, the last of them short."""
    run_norms(np.random.default_rng(rows), kind, rows, width, pads=pads)


@pytest.mark.parametrize("parts", ["".join(p) for n in range(7)
                                   for p in itertools.combinations("zxwcpy", n)
                                   if "y" in p or "p" in p])
def test_norms_parts(parts):
    run_norms(np.random.default_rng(1), "f32", 9, 136, parts=parts)


@pytest.mark.parametrize("gate", [bs.BS_GATE_SILU, bs.BS_GATE_SIGMOID, bs.BS_GATE_LINEAR])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_norms_gates(kind, gate):
    run_norms(np.random.default_rng(2), kind, 33, 384, gate=gate)


@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("pads", [(0, 8), (8, 8), (1, 0), (2, 2), (4, 0), (0, 1)])
def test_norms_strides_and_alignment(kind, pads):
    run_norms(np.random.default_rng(3), kind, 21, 520, pads=pads)


def test_norms_zero_rows_and_open_gates():
    """Rows of zeros have a finite norm (eps), rows of large values do not overflow it, gates at
    the ends of their range are 0, 1 or z."""
    rng = np.random.default_rng(4)
    f = values(rng, (6, 200), "f32")
    f[0], f[1], f[2] = 0.0, f[1] * 1e15, f[2] * 1e-18
    run_norms(rng, "f32", 6, 200, f=f, parts="xwcpy")
    z = torch.tensor([[-100.0, -1e30, 0.0, 100.0, 1e30, 88.0, -88.0, 1.0]], device="cuda")
    one, y = torch.ones_like(z), torch.empty_like(z)
    bs.bs_gnorm_batched(one, y, z=z)
    assert bool((y[0, :3].abs() < 1e-30).all()) and bool((y[0, 3:6] == z[0, 3:6]).all())
    assert abs(float(y[0, 7]) - 0.7310585786300049) < 1e-6


def test_norms_nonfinite_rows_stay_apart():
    rng = np.random.default_rng(5)
    f, z, x = (torch.from_numpy(values(rng, (40, 300), "bf16")).to(torch.bfloat16).cuda()
               for _ in range(3))
    w = f32(1 + 0.1 * rng.standard_normal(300))
    got = []
    for bad in (False, True):
        g = f.clone()
        if bad:
            g[7, 3], g[30, 299] = float("inf"), float("nan")
        y, u = torch.empty_like(f), torch.empty_like(f)
        bs.bs_gnorm_batched(g, y, z=z, x=x, w_post=w, w_pre=w, u=u)
        got.append((y, u))
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[[7, 30]] = False
    for a, b in zip(*got):
        assert torch.equal(a[keep], b[keep])
    assert bool(torch.isnan(got[1][0][30]).all())


# ----------------------------------------------------------------- streams, graphs, windows
def test_streams_and_graphs():
    """A captured pass replays on new inputs, on a stream of its own."""
    rng = np.random.default_rng(17)
    c, rows = 128, 500
    p = torch.empty(1, rows, 3 * c, dtype=torch.bfloat16, device="cuda")
    x, r, i = p[..., :c], p[..., c:2 * c], p[..., 2 * c:]
    la, w = f32(rng.uniform(-7, 0, c)), torch.ones(c, device="cuda")
    h, y, u = (torch.empty(1, rows, c, dtype=torch.bfloat16, device="cuda") for _ in range(3))
    tape = torch.empty(bs.bs_grec_tape_rows(1, rows), c, device="cuda")
    dp, dlam = torch.empty_like(p), torch.empty(c, device="cuda")
    d = dp[..., :c], dp[..., c:2 * c], dp[..., 2 * c:]
    work = torch.empty(bs.bs_grec_backward_workspace(c, 1, rows), dtype=torch.uint8, device="cuda")

    def calls():
        bs.bs_grec_batched(x, r, i, la, h, tape=tape)
        bs.bs_gnorm_batched(h, y, z=x, w_post=w, w_pre=w, u=u)
        bs.bs_grec_backward_batched(x, r, i, la, tape, u, *d, dlam, work)

    def once(v):
        p.copy_(v)
        calls()
        torch.cuda.synchronize()
        return [t.clone() for t in (h, y, u, dp, dlam)]

    inputs = [torch.from_numpy(values(rng, p.shape, "bf16")).to(torch.bfloat16).cuda()
              for _ in range(2)]
    want = [once(v) for v in inputs]
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph, stream=stream):
        calls()
    for v, ws in zip(inputs, want):
        p.copy_(v)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip((h, y, u, dp, dlam), ws))
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        p.copy_(inputs[0])
        calls()
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((h, y, u, dp, dlam), want[0]))


def test_empty_calls():
    c = 64
    la = torch.zeros(c, device="cuda")
    e = torch.empty(0, c, device="cuda")
    h0, hT = torch.randn(3, c, device="cuda"), torch.empty(3, c, device="cuda")
    off = torch.zeros(4, dtype=torch.int64, device="cuda")
    tape = torch.empty(3, c, device="cuda")
    bs.bs_grec_batched(e, e, e, la, e, h0=h0, hT=hT, offsets=off, tape=tape)
    assert torch.equal(h0, hT)
    dlam, dh0 = torch.full((c,), MARK, device="cuda"), torch.empty(3, c, device="cuda")
    work = torch.empty(max(16, bs.bs_grec_backward_workspace(c, 3, 0)), dtype=torch.uint8,
                       device="cuda")
    bs.bs_grec_backward_batched(e, e, e, la, tape, e, e, e, e, dlam, work, dhT=h0, dh0=dh0,
                                offsets=off)
    assert torch.equal(dh0, h0) and bool((dlam == 0).all())
    bs.bs_gnorm_batched(e, e)
    s = [torch.full((c,), MARK, device="cuda") for _ in range(3)]
    bs.bs_gnorm_backward_batched(e, e, e, work, w_post=la, scale=la, w_pre=la, du=e, dw_post=s[0],
                                 dscale=s[1], dw_pre=s[2])
    assert all(bool((t == 0).all()) for t in s)
    bs.bs_grec_step_batched(e, e, e, la, h0, e)


def test_binding_refuses():
    """Operands of another type, shape, device or layout than the first one's."""
    x = torch.zeros(2, 10, 8, device="cuda")
    lam = torch.zeros(8, device="cuda")
    h = torch.empty_like(x)
    bad = [
        (TypeError, "dtype", dict(r=x.half())), (ValueError, "shape", dict(r=x[:, :9])),
        (ValueError, "device", dict(i=x.cpu())), (ValueError, "contiguous", dict(h=x.mT.contiguous().mT)),
        (ValueError, "one distance", dict(x=x[:, :9], r=x[:, :9], i=x[:, :9], h=x[:, :9])),
        (ValueError, "one distance", dict(i=x[:, :1].expand(2, 10, 8))),
        (TypeError, "dtype", dict(lam=lam.double())), (ValueError, "elements", dict(lam=lam[:7])),
        (ValueError, "elements", dict(h0=torch.zeros(3, 8, device="cuda"))),
        (ValueError, "device", dict(hT=torch.zeros(2, 8))),
        (ValueError, "contiguous", dict(hT=torch.zeros(8, 2, device="cuda").T)),
        (ValueError, "elements", dict(tape=torch.zeros(1, 8, device="cuda"))),
        (ValueError, "expected", dict(offsets=torch.zeros(3, dtype=torch.int64, device="cuda"))),
        (TypeError, "tensor", dict(lam=3.0)),
    ]
    for error, text, change in bad:
        with pytest.raises(error, match=text):
            bs.bs_grec_batched(**{**dict(x=x, r=x, i=x, lam=lam, h=h), **change})
    with pytest.raises(ValueError, match="rows overlap"):
        bs.bs_gnorm_batched(x[0, :1].expand(10, 8), h[0])
    with pytest.raises(TypeError, match="dtype"):
        bs.bs_grec_batched(x[0], x[0], x[0], lam, h[0],
                           offsets=torch.zeros(3, dtype=torch.int32, device="cuda"))
    with pytest.raises(ValueError, match="state"):
        bs.bs_grec_step_batched(x[0], x[0], x[0], lam, torch.zeros(3, 9, device="cuda"), h[0])
    with pytest.raises(TypeError, match="dtype"):
        bs.bs_grec_step_batched(x[0], x[0], x[0], lam, torch.zeros(10, 8, device="cuda"), h[0],
                                slots=torch.zeros(10, device="cuda"))
    with pytest.raises(bs.BsolveError, match="INVALID_ARG"):
        bs.bs_grec_batched(x, x, x, lam, x)  # the output over its inputs
    with pytest.raises(TypeError, match="dtype"):
        bs.bs_gnorm_backward_batched(x, x, h, work=lam)
