"""Cases of the recurrent-block operators: the gated linear recurrence (forward over long and packed
sequences, training pass, one-token step) and the norms around a block fused with its gate and
residual scale (forward, training pass).

`own` false: elementary torch operations in 32 bits, rounded once at the end. `own` true: the library's
calls, as a user makes them."""
import math

import torch

own = False

KAPPA = 8.0
EPS = 1e-6
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token: a single row, launch latency is all there is
        {"name": "grec_step_1", "op": "grec_step", "dtype": "bf16", "batch": 1, "slots": 1,
         "channels": 2048},
        # a full serving batch, the rows' states in a larger pool by slot
        {"name": "grec_step_256", "op": "grec_step", "dtype": "bf16", "batch": 256, "slots": 320,
         "channels": 4096},
        # prompts of uneven lengths packed without padding, some empty or one token long,
        # some continued from a kept state
        {"name": "grec_prompts", "op": "grec_forward", "dtype": "bf16", "batch": 24, "rows": 12011,
         "packed": True, "channels": 2048},
        # one very long document: parallelism has to come from the sequence itself
        {"name": "grec_long", "op": "grec_forward", "dtype": "bf16", "batch": 1, "rows": 65536,
         "packed": False, "channels": 4096},
        # 32-bit data with an odd channel count: no row but the first is aligned
        {"name": "grec_f32_odd", "op": "grec_forward", "dtype": "f32", "batch": 3, "rows": 3 * 1023,
         "packed": False, "channels": 1001},
        # an ordinary training pass of a layer: forward, then every gradient
        {"name": "grec_train", "op": "grec_train", "dtype": "bf16", "batch": 8, "rows": 8 * 4096,
         "packed": False, "channels": 2048},
        # a small training pass in 16 bits at odd sizes, sequences packed
        {"name": "grec_train_f16_odd", "op": "grec_train", "dtype": "f16", "batch": 5, "rows": 3885,
         "packed": True, "channels": 523},
        # the norms around a block for one token
        {"name": "gnorm_1", "op": "gnorm_forward", "dtype": "bf16", "rows": 1, "width": 2048},
        # and over a long prompt or a training batch
        {"name": "gnorm_16k", "op": "gnorm_forward", "dtype": "bf16", "rows": 16384, "width": 4096},
        # 32-bit data at an odd width
        {"name": "gnorm_f32_odd", "op": "gnorm_forward", "dtype": "f32", "rows": 4099, "width": 1001},
        # an ordinary training pass
        {"name": "gnorm_train", "op": "gnorm_train", "dtype": "bf16", "rows": 16384, "width": 4096},
        # a small one in 16 bits
        {"name": "gnorm_train_f16", "op": "gnorm_train", "dtype": "f16", "rows": 515, "width": 1536},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["grec_step", "grec_forward", "grec_forward", "grec_train", "gnorm_forward",
                     "gnorm_train"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    width = _log(rng, 64, 8192)
    if rng.random() < 0.6:  # most widths in use are multiples of 64
        width = max(64, width // 64 * 64)
    if op == "grec_step":
        batch = _log(rng, 1, 512)
        return {"op": op, "dtype": dtype, "batch": batch, "slots": batch + rng.randrange(64),
                "channels": width}
    if op in ("grec_forward", "grec_train"):
        most = (1 << 27 if op == "grec_forward" else 1 << 26) // width
        rows = _log(rng, 16, min(most, 65536))
        batch = _log(rng, 1, min(64, rows))
        packed = rng.random() < 0.5
        if not packed:
            rows = max(1, rows // batch) * batch
        return {"op": op, "dtype": dtype, "batch": batch, "rows": rows, "packed": packed,
                "channels": width}
    return {"op": op, "dtype": dtype, "rows": _log(rng, 1, min((1 << 26) // width, 65536)),
            "width": width}


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "grec_step":
        n = case["batch"] * case["channels"]
        return {"bytes": n * (4 * b + 8) + 4 * case["channels"], "flops": 30 * n}
    if case["op"].startswith("grec"):
        n, s = case["rows"] * case["channels"], case["batch"] * case["channels"] * 4
        if case["op"] == "grec_forward":  # x, r, i in, h out, states in and out
            return {"bytes": n * 4 * b + 2 * s, "flops": 30 * n}
        # x, r, i, dh in, h, dx, dr, di out; the state and its gradient on both sides
        return {"bytes": n * 8 * b + 4 * s + 8 * case["channels"], "flops": 80 * n}
    n, w = case["rows"] * case["width"], case["width"] * 4
    if case["op"] == "gnorm_forward":  # f, z, x in, y, u out
        return {"bytes": n * 5 * b + 3 * w, "flops": 20 * n}
    # f, z, x, dy, du in, y, u, df, dz, dx out
    return {"bytes": n * 10 * b + 6 * w, "flops": 60 * n}


# -------------------------------------------------------------------------------- inputs
def _lengths(case, seed):
    """Lengths of the sequences: equal, or uneven where they are packed, with one of no row and one
    of a single row among four or more."""
    batch, rows = case["batch"], case["rows"]
    if not case["packed"]:
        return [rows // batch] * batch
    g = torch.Generator().manual_seed(1000003 + seed)
    cut = torch.sort(torch.randint(0, rows + 1, (batch - 1,), generator=g)).values.tolist()
    lens = [q - p for p, q in zip([0] + cut, cut + [rows])]
    if batch >= 4:
        lens[0], lens[1] = lens[0] + lens[1], 0
        both = lens[2] + lens[3]
        lens[2], lens[3] = both - min(1, both), min(1, both)
    return lens


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed))
    dt = DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt, scale=1.0):
        return (torch.randn(*shape, generator=g, device=DEVICE) * scale).to(dtype)

    s = dict(case)
    if case["op"].startswith("grec"):
        c = case["channels"]
        # decay of each channel at an open gate between 0.9 and 0.999
        keep = 0.9 + 0.099 * torch.rand(c, generator=g, device=DEVICE)
        s["lam"] = torch.log(torch.expm1(-2.0 * torch.log(keep) / KAPPA)).contiguous()
        rows = case["batch"] if case["op"] == "grec_step" else case["rows"]
        # x, r, i are column windows of one product's output, as a layer's projection leaves them
        p = normal(rows, 3 * c)
        s["x"], s["r"], s["i"] = p[:, :c], p[:, c:2 * c], p[:, 2 * c:]
        if case["op"] == "grec_step":
            s["state"] = normal(case["slots"], c, dtype=torch.float32)
            s["slot"] = torch.randperm(case["slots"], generator=g,
                                       device=DEVICE)[:case["batch"]].to(torch.int32)
            return s
        lens = _lengths(case, int(seed))
        at = [0]
        for n in lens:
            at.append(at[-1] + n)
        s["longest"] = max(lens)
        s["offsets"] = torch.tensor(at, dtype=torch.int64, device=DEVICE)
        live = [b for b, n in enumerate(lens) if n]
        s["live"] = torch.tensor(live, dtype=torch.int64, device=DEVICE)
        s["first"] = torch.tensor([at[b] for b in live], dtype=torch.int64, device=DEVICE)
        s["last"] = torch.tensor([at[b + 1] - 1 for b in live], dtype=torch.int64, device=DEVICE)
        s["h0"] = normal(case["batch"], c, dtype=torch.float32)
        if case["op"] == "grec_train":
            s["dh"] = normal(rows, c)
            s["dhT"] = normal(case["batch"], c, dtype=torch.float32)
        return s
    rows, w = case["rows"], case["width"]
    s["f"], s["z"], s["x"] = normal(rows, w, scale=0.7), normal(rows, w), normal(rows, w, scale=2.0)
    s["w_post"] = 1.0 + normal(w, dtype=torch.float32, scale=0.1)
    s["scale"] = 0.5 + normal(w, dtype=torch.float32, scale=0.1)
    s["w_pre"] = 1.0 + normal(w, dtype=torch.float32, scale=0.1)
    if case["op"] == "gnorm_train":
        s["dy"], s["du"] = normal(rows, w), normal(rows, w)
    return s


# ---------------------------------------------------------------------------- plain forms
def _gates(s):
    x, r, i = s["x"].float(), s["r"].float(), s["i"].float()
    sp = KAPPA * (torch.clamp(s["lam"], min=0) + torch.log1p(torch.exp(-torch.abs(s["lam"]))))
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    l = -sp * sr
    return x, sr, si, sp, l, torch.exp(l), torch.sqrt(-torch.expm1(2 * l))


def _solve(a, u, longest):
    """h_t = a_t h_{t-1} + u_t down the rows by doubling; a is 0 where a sequence starts."""
    d = 1
    while d < longest:
        u = torch.cat([u[:d], u[d:] + a[d:] * u[:-d]])
        a = torch.cat([a[:d], a[d:] * a[:-d]])
        d *= 2
    return u


def _plain_recurrence(s):
    x, sr, si, sp, l, a, root = _gates(s)
    u = root * si * x
    u[s["first"]] += a[s["first"]] * s["h0"][s["live"]]
    start = a.clone()
    start[s["first"]] = 0
    h = _solve(start, u, s["longest"])
    hT = s["h0"].clone()
    hT[s["live"]] = h[s["last"]]
    return x, sr, si, sp, l, a, root, h, hT


def _plain_train(s):
    dt = s["x"].dtype
    x, sr, si, sp, l, a, root, h, hT = _plain_recurrence(s)
    out = {"h": h.to(dt), "hT": hT}
    before = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    before[s["first"]] = s["h0"][s["live"]]
    dh = s["dh"].float()
    dh[s["last"]] += s["dhT"][s["live"]]
    after = torch.cat([a[1:], torch.zeros_like(a[:1])])
    after[s["last"]] = 0
    g = _solve(after.flip(0), dh.flip(0), s["longest"]).flip(0)
    ratio = torch.where(root > 0, l / root, torch.zeros_like(l))
    d = g * (l * a * before - si * x * a * a * ratio)
    out["dx"] = (g * root * si).to(dt)
    out["dr"] = (d * (1 - sr)).to(dt)
    out["di"] = (g * root * x * si * (1 - si)).to(dt)
    out["dlam"] = d.sum(0) * KAPPA * torch.sigmoid(s["lam"]) / sp
    dh0 = s["dhT"].clone()
    dh0[s["live"]] = a[s["first"]] * g[s["first"]]
    out["dh0"] = dh0
    return out


def _plain_step(s):
    x, sr, si, sp, l, a, root = _gates(s)
    at = s["slot"].long()
    h = a * s["state"][at] + root * si * x
    s["state"][at] = h
    return {"y": h.to(s["x"].dtype), "state": s["state"]}


def _plain_norms(s):
    f, z, x = s["f"].float(), s["z"].float(), s["x"].float()
    r1 = torch.rsqrt((f * f).mean(1, keepdim=True) + EPS)
    n = f * r1
    t = n * s["w_post"] * (z * torch.sigmoid(z))
    y = x + s["scale"] * t
    r2 = torch.rsqrt((y * y).mean(1, keepdim=True) + EPS)
    return f, z, x, r1, n, t, y, r2


def _plain_norms_train(s):
    dt = s["f"].dtype
    f, z, x, r1, n, t, y, r2 = _plain_norms(s)
    out = {"y": y.to(dt), "u": (y * r2 * s["w_pre"]).to(dt)}
    dy, du = s["dy"].float(), s["du"].float()
    out["dw_pre"] = (du * y * r2).sum(0)
    m = du * s["w_pre"] * r2
    d = dy + m - y * r2 * r2 * (m * y).mean(1, keepdim=True)
    out["dx"] = d.to(dt)
    out["dscale"] = (d * t).sum(0)
    d = d * s["scale"]
    sz = torch.sigmoid(z)
    out["dz"] = (d * n * s["w_post"] * sz * (1 + z * (1 - sz))).to(dt)
    d = d * z * sz
    out["dw_post"] = (d * n).sum(0)
    d = d * s["w_post"]
    out["df"] = (r1 * (d - n * (d * n).mean(1, keepdim=True))).to(dt)
    return out


# ------------------------------------------------------------------------ the library's calls
def _own_step(bs, s):
    y = torch.empty(s["batch"], s["channels"], dtype=s["x"].dtype, device=DEVICE)
    bs.bs_grec_step_batched(s["x"], s["r"], s["i"], s["lam"], s["state"], y, slots=s["slot"],
                            kappa=KAPPA)
    return {"y": y, "state": s["state"]}


def _sequences(s, t):
    """How the call takes the rows: packed with offsets, or as (batch, length, channels)."""
    return t if s["packed"] else t.view(s["batch"], -1, s["channels"])


def _own_forward(bs, s, tape=None):
    h = torch.empty(s["rows"], s["channels"], dtype=s["x"].dtype, device=DEVICE)
    hT = torch.empty_like(s["h0"])
    bs.bs_grec_batched(_sequences(s, s["x"]), _sequences(s, s["r"]), _sequences(s, s["i"]),
                       s["lam"], _sequences(s, h), h0=s["h0"], hT=hT,
                       offsets=s["offsets"] if s["packed"] else None, tape=tape, kappa=KAPPA)
    return {"h": h, "hT": hT}


def _own_train(bs, s):
    c = s["channels"]
    tape = torch.empty(bs.bs_grec_tape_rows(s["batch"], s["rows"]), c, device=DEVICE)
    out = _own_forward(bs, s, tape)
    out["dx"], out["dr"], out["di"] = (torch.empty_like(out["h"]) for _ in range(3))
    out["dlam"], out["dh0"] = torch.empty_like(s["lam"]), torch.empty_like(s["h0"])
    work = torch.empty(bs.bs_grec_backward_workspace(c, s["batch"], s["rows"]),
                       dtype=torch.uint8, device=DEVICE)
    bs.bs_grec_backward_batched(
        *(_sequences(s, s[k]) for k in ("x", "r", "i")), s["lam"], tape, _sequences(s, s["dh"]),
        *(_sequences(s, out[k]) for k in ("dx", "dr", "di")), out["dlam"], work, dhT=s["dhT"],
        dh0=out["dh0"], offsets=s["offsets"] if s["packed"] else None, kappa=KAPPA)
    return out


def _own_norms(bs, s):
    y, u = torch.empty_like(s["f"]), torch.empty_like(s["f"])
    bs.bs_gnorm_batched(s["f"], y, z=s["z"], x=s["x"], w_post=s["w_post"], scale=s["scale"],
                        w_pre=s["w_pre"], u=u, eps=EPS, gate=bs.BS_GATE_SILU)
    return {"y": y, "u": u}


def _own_norms_train(bs, s):
    out = _own_norms(bs, s)
    out["df"], out["dz"], out["dx"] = (torch.empty_like(s["f"]) for _ in range(3))
    out["dw_post"], out["dscale"], out["dw_pre"] = (torch.empty_like(s["scale"]) for _ in range(3))
    work = torch.empty(bs.bs_gnorm_backward_workspace(s["width"], s["rows"]), dtype=torch.uint8,
                       device=DEVICE)
    bs.bs_gnorm_backward_batched(
        s["f"], s["dy"], out["df"], work, z=s["z"], x=s["x"], w_post=s["w_post"],
        scale=s["scale"], w_pre=s["w_pre"], du=s["du"], dz=out["dz"], dx=out["dx"],
        dw_post=out["dw_post"], dscale=out["dscale"], dw_pre=out["dw_pre"], eps=EPS,
        gate=bs.BS_GATE_SILU)
    return out


def run(s):
    if own:
        import dense_linear_solvers_gb300 as bs
        return {"grec_step": _own_step, "grec_forward": _own_forward, "grec_train": _own_train,
                "gnorm_forward": _own_norms, "gnorm_train": _own_norms_train}[s["op"]](bs, s)
    dt = s["x"].dtype
    if s["op"] == "grec_step":
        return _plain_step(s)
    if s["op"] == "grec_forward":
        h, hT = _plain_recurrence(s)[-2:]
        return {"h": h.to(dt), "hT": hT}
    if s["op"] == "grec_train":
        return _plain_train(s)
    if s["op"] == "gnorm_forward":
        y, r2 = _plain_norms(s)[-2:]
        return {"y": y.to(dt), "u": (y * r2 * s["w_pre"]).to(dt)}
    return _plain_norms_train(s)


# ------------------------------------------------------------------------ 64-bit definition
def exact(case, seed):
    """The definition in 64 bits: the recurrence row by row, every gradient by the chain rule
    through that loop, the norms by their formulas."""
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v
         for k, v in prepare(case, seed).items()}
    if case["op"].startswith("gnorm"):
        return _exact_norms(s, case["op"] == "gnorm_train")
    rate = KAPPA * torch.nn.functional.softplus(s["lam"], threshold=100.0)
    sr, si = 1 / (1 + torch.exp(-s["r"])), 1 / (1 + torch.exp(-s["i"]))
    decay = torch.exp(-rate * sr)
    room = -torch.expm1(-2 * rate * sr)
    if case["op"] == "grec_step":
        h = decay * s["state"][s["slot"].long()] + torch.sqrt(room) * si * s["x"]
        s["state"][s["slot"].long()] = h
        return {"y": h, "state": s["state"]}
    rows, ends = case["rows"], s["offsets"].tolist()
    begins = {}
    for b in range(case["batch"]):
        if ends[b] < ends[b + 1]:
            begins[ends[b]] = b
    add = torch.sqrt(room) * si * s["x"]
    # all sequences advance together, padded to the longest
    longest, batch, c = s["longest"], case["batch"], case["channels"]
    if longest * batch * c > 3 << 28:
        return None
    length = s["offsets"][1:] - s["offsets"][:-1]
    t = torch.arange(longest, device=DEVICE)[:, None]
    valid = t < length[None]
    source = torch.where(valid, s["offsets"][:-1][None] + t, torch.zeros_like(t))

    def spread(v):  # (rows, c) -> (longest, batch, c), zeros past a sequence's end
        return v[source.reshape(-1)].view(longest, batch, c) * valid[..., None]

    def gather(v):
        return v.reshape(longest * batch, c)[
            torch.zeros(rows, dtype=torch.int64, device=DEVICE).index_put_(
                (source[valid],), torch.arange(longest * batch,
                                               device=DEVICE).view(longest, batch)[valid])]

    a, u = spread(decay), spread(add)
    a = a + (~valid)[..., None].double()         # past its end a sequence keeps its state
    h, states = s["h0"], torch.empty_like(u)
    for k in range(longest):
        h = torch.addcmul(u[k], a[k], h, out=states[k])
    out = {"h": gather(states), "hT": h.clone()}
    if case["op"] == "grec_forward":
        return out
    up, grad, g = spread(s["dh"]), torch.empty_like(u), s["dhT"]
    for k in range(longest - 1, -1, -1):         # g: the gradient of the state after row k
        grad[k] = g + up[k]
        g = a[k] * grad[k]
    out["dh0"] = g
    g = gather(grad)
    prev = gather(torch.cat([s["h0"][None], states[:-1]]))
    root = torch.sqrt(room)
    out["dx"] = g * root * si
    out["di"] = g * root * s["x"] * (si - si * si)
    da = g * (prev - decay / root * si * s["x"])
    out["dr"] = da * decay * -rate * sr * (1 - sr)
    out["dlam"] = (da * decay * -sr).sum(0) * KAPPA / (1 + torch.exp(-s["lam"]))
    return out


def _exact_norms(s, train):
    f, z, x, w, c, p = (s[k] for k in ("f", "z", "x", "w_post", "scale", "w_pre"))
    width = f.shape[1]
    q1 = 1 / torch.sqrt(torch.einsum("ij,ij->i", f, f) / width + EPS)[:, None]
    sz = 1 / (1 + torch.exp(-z))
    y = x + c * (f * q1 * w) * (z * sz)
    q2 = 1 / torch.sqrt(torch.einsum("ij,ij->i", y, y) / width + EPS)[:, None]
    out = {"y": y, "u": y * q2 * p}
    if not train:
        return out
    du, dy = s["du"], s["dy"]
    out["dw_pre"] = torch.einsum("ij,ij->j", du, y * q2)
    e = du * p
    dx = dy + q2 * e - y * q2 ** 3 * (torch.einsum("ij,ij->i", e, y) / width)[:, None]
    out["dx"] = dx
    out["dscale"] = torch.einsum("ij,ij->j", dx, f * q1 * w * z * sz)
    out["dz"] = dx * c * f * q1 * w * (sz + z * sz * (1 - sz))
    dn = dx * c * z * sz
    out["dw_post"] = torch.einsum("ij,ij->j", dn, f * q1)
    e = dn * w
    out["df"] = q1 * e - f * q1 ** 3 * (torch.einsum("ij,ij->i", e, f) / width)[:, None]
    return out
