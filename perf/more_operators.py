"""Cases of the gated delta rule (forward over long and packed sequences, training pass, one-token
step), of the norms around a block with an output in 8 bits, and of the product that reads it.

`own` false: elementary torch operations in 32 bits, rounded once at the end. `own` true: the library's
calls, as a user makes them."""
import math

import torch

own = False

EPS = 1e-6
CHUNK = 64          # rows that the plain form solves together
BLOCK = 128         # elements of a row under one scale
TOP = 448.0         # largest number of the 8-bit type
DTYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
BYTES = {"bf16": 2, "f16": 2, "f32": 4}
DEVICE = "cuda" if torch.cuda.is_available() else "cpu"


# ------------------------------------------------------------------------------- cases
def listed():
    return [
        # one user's next token: the heads' states are read and written, little else
        {"name": "gdelta_step_1", "op": "gdelta_step", "dtype": "bf16", "batch": 1, "slots": 1,
         "heads_k": 16, "heads_v": 32, "dk": 128, "dv": 128},
        # a serving batch, the rows' states in a larger pool by slot
        {"name": "gdelta_step_200", "op": "gdelta_step", "dtype": "bf16", "batch": 200, "slots": 256,
         "heads_k": 16, "heads_v": 32, "dk": 128, "dv": 128},
        # prompts of uneven lengths packed without padding, some empty or one token long, all
        # continued from a kept state
        {"name": "gdelta_prompts", "op": "gdelta_forward", "dtype": "bf16", "batch": 24,
         "rows": 12011, "packed": True, "heads_k": 16, "heads_v": 32, "dk": 128, "dv": 128},
        # one very long document in few heads: the chain of states is all that bounds it
        {"name": "gdelta_long", "op": "gdelta_forward", "dtype": "bf16", "batch": 1, "rows": 32768,
         "packed": False, "heads_k": 8, "heads_v": 16, "dk": 128, "dv": 128},
        # 32-bit data with odd head sizes: no row but the first is aligned
        {"name": "gdelta_f32_odd", "op": "gdelta_forward", "dtype": "f32", "batch": 3,
         "rows": 3 * 1023, "packed": False, "heads_k": 5, "heads_v": 5, "dk": 93, "dv": 77},
        # an ordinary training pass of a layer: forward, then every gradient
        {"name": "gdelta_train", "op": "gdelta_train", "dtype": "bf16", "batch": 8, "rows": 8 * 2048,
         "packed": False, "heads_k": 8, "heads_v": 16, "dk": 128, "dv": 128},
        # a small training pass in 16 bits, three value heads a key head, sequences packed
        {"name": "gdelta_train_f16_odd", "op": "gdelta_train", "dtype": "f16", "batch": 5,
         "rows": 3885, "packed": True, "heads_k": 2, "heads_v": 6, "dk": 64, "dv": 72},
        # the norms around a block for one token, the next product's input in 8 bits
        {"name": "gnorm_q8_1", "op": "gnorm_q8", "dtype": "bf16", "rows": 1, "width": 2048},
        # and over a long prompt
        {"name": "gnorm_q8_16k", "op": "gnorm_q8", "dtype": "bf16", "rows": 16384, "width": 4096},
        # a block's products for one token: the weights are read once
        {"name": "gemm_q8_1", "op": "gemm_q8", "dtype": "bf16", "m": 1, "n": 8192, "k": 2048},
        # ragged sizes at a batch of a few hundred rows
        {"name": "gemm_q8_ragged", "op": "gemm_q8", "dtype": "f16", "m": 515, "n": 2000, "k": 1552},
        # and over a long prompt: arithmetic alone
        {"name": "gemm_q8_16k", "op": "gemm_q8", "dtype": "bf16", "m": 16384, "n": 8192, "k": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["gdelta_step", "gdelta_forward", "gdelta_forward", "gdelta_train", "gnorm_q8",
                     "gemm_q8"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op == "gemm_q8":
        m, n, k = _log(rng, 1, 16384), _log(rng, 64, 16384), 16 * _log(rng, 4, 1024)
        if rng.random() < 0.6:
            n, k = max(64, n // 64 * 64), max(64, k // 64 * 64)
        while m * n * k > 1 << 39:
            m = m // 2
        return {"op": op, "dtype": dtype, "m": m, "n": n, "k": k}
    if op == "gnorm_q8":
        width = _log(rng, 64, 8192)
        if rng.random() < 0.6:
            width = max(64, width // 64 * 64)
        return {"op": op, "dtype": dtype, "rows": _log(rng, 1, min((1 << 26) // width, 65536)),
                "width": width}
    heads_k, dk, dv = _log(rng, 1, 16), rng.choice([64, 128, 128]), rng.choice([64, 128, 128, 256])
    if rng.random() < 0.3:
        dk, dv = rng.randint(16, 128), rng.randint(16, 256)
    heads_v = heads_k * rng.choice([1, 1, 2, 2, 3, 4])
    case = {"op": op, "dtype": dtype, "heads_k": heads_k, "heads_v": heads_v, "dk": dk, "dv": dv}
    state = heads_v * dk * dv
    if op == "gdelta_step":
        batch = _log(rng, 1, max(2, min(512, (100 << 20) // state)))
        return dict(case, batch=batch, slots=batch + rng.randrange(64))
    most = (1 << (28 if op == "gdelta_forward" else 27)) // (heads_v * (dk + dv) // 2)
    rows = _log(rng, 16, max(17, min(most, 32768 if op == "gdelta_forward" else 16384)))
    batch = _log(rng, 1, min(32, rows))
    packed = rng.random() < 0.5
    if not packed:
        rows = max(1, rows // batch) * batch
    return dict(case, batch=batch, rows=rows, packed=packed)


def work(case):
    b = BYTES[case["dtype"]]
    if case["op"] == "gemm_q8":
        m, n, k = case["m"], case["n"], case["k"]
        blocks = -(-k // BLOCK)
        return {"bytes": m * k + n * k + m * n * b + 4 * blocks * (m + -(-n // BLOCK)),
                "flops": 2 * m * n * k}
    if case["op"] == "gnorm_q8":  # f, z, x in, y, the 8-bit output and its scales out
        n, w = case["rows"] * case["width"], case["width"]
        return {"bytes": n * (4 * b + 1) + 4 * case["rows"] * -(-w // BLOCK) + 12 * w,
                "flops": 24 * n}
    qk, v = case["heads_k"] * case["dk"], case["heads_v"] * case["dv"]
    state = case["heads_v"] * case["dk"] * case["dv"]
    if case["op"] == "gdelta_step":
        n = case["batch"]
        return {"bytes": n * (b * (2 * qk + 2 * v) + 8 * case["heads_v"] + 8 * state),
                "flops": 8 * n * state}
    rows, n = case["rows"], case["batch"]
    # the recurrence row by row: k S, the update, q S
    flops = 6 * rows * state
    if case["op"] == "gdelta_forward":
        return {"bytes": rows * (b * (2 * qk + 2 * v) + 8 * case["heads_v"]) + 8 * n * state,
                "flops": flops}
    # q, k, v, g, beta, do in, o and five gradients out; the state and its gradient on both sides
    return {"bytes": rows * (b * (4 * qk + 4 * v) + 16 * case["heads_v"]) + 16 * n * state,
            "flops": 3 * flops}


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
    if case["op"] == "gemm_q8":
        m, n, k = case["m"], case["n"], case["k"]
        s["a"], s["sa"] = _quantised(normal(m, k, dtype=torch.float32))
        # weights under one scale a 128 x 128 block, laid out once
        w = normal(n, k, dtype=torch.float32, scale=k ** -0.5)
        nb, kb = -(-n // BLOCK), -(-k // BLOCK)
        full = torch.zeros(nb * BLOCK, kb * BLOCK, device=DEVICE)
        full[:n, :k] = w
        full = full.view(nb, BLOCK, kb, BLOCK)
        s["sw"] = full.abs().amax((1, 3)).clamp_min(2.0 ** -100) / TOP
        full = full / s["sw"][:, None, :, None]
        s["w"] = full.view(nb * BLOCK, kb * BLOCK)[:n, :k].contiguous().to(torch.float8_e4m3fn)
        return s
    if case["op"] == "gnorm_q8":
        rows, w = case["rows"], case["width"]
        s["f"], s["z"] = normal(rows, w, scale=0.7), normal(rows, w)
        s["x"] = normal(rows, w, scale=2.0)
        s["w_post"] = 1.0 + normal(w, dtype=torch.float32, scale=0.1)
        s["scale"] = 0.5 + normal(w, dtype=torch.float32, scale=0.1)
        s["w_pre"] = 1.0 + normal(w, dtype=torch.float32, scale=0.1)
        return s
    hk, hv, dk, dv = (case[n] for n in ("heads_k", "heads_v", "dk", "dv"))
    rows = case["batch"] if case["op"] == "gdelta_step" else case["rows"]
    # q, k of length one, a head's keys with a part in common; v; all three column windows of one
    # matrix, as a layer's projection leaves them
    p = torch.empty(rows, 2 * hk * dk + hv * dv, dtype=dt, device=DEVICE)
    for j, common in ((0, 0.2), (1, 0.5)):
        t = torch.randn(rows, hk, dk, generator=g, device=DEVICE) + common * torch.randn(
            hk, dk, generator=g, device=DEVICE)
        t = t / t.norm(dim=-1, keepdim=True)
        p[:, j * hk * dk:(j + 1) * hk * dk] = t.view(rows, hk * dk).to(dt)
    p[:, 2 * hk * dk:] = normal(rows, hv * dv)
    s["q"] = p[:, :hk * dk].unflatten(1, (hk, dk))
    s["k"] = p[:, hk * dk:2 * hk * dk].unflatten(1, (hk, dk))
    s["v"] = p[:, 2 * hk * dk:].unflatten(1, (hv, dv))
    # log decays of rates 1 to 16 and steps 0.001 to 0.1; the rate of writing
    rate = 1 + 15 * torch.rand(hv, generator=g, device=DEVICE)
    step = torch.exp(math.log(1e-3) + math.log(100) * torch.rand(rows, hv, generator=g, device=DEVICE))
    s["g"] = -rate * step
    s["beta"] = torch.sigmoid(normal(rows, hv, dtype=torch.float32))
    if case["op"] == "gdelta_step":
        s["state"] = normal(case["slots"], hv, dk, dv, dtype=torch.float32, scale=0.3)
        s["slot"] = torch.randperm(case["slots"], generator=g,
                                   device=DEVICE)[:case["batch"]].to(torch.int32)
        return s
    lens = _lengths(case, int(seed))
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    s["longest"] = max(lens)
    s["offsets"] = torch.tensor(at, dtype=torch.int64, device=DEVICE)
    s["h0"] = normal(case["batch"], hv, dk, dv, dtype=torch.float32, scale=0.3)
    if case["op"] == "gdelta_train":
        s["do"] = normal(rows, hv, dv)
        s["dhT"] = normal(case["batch"], hv, dk, dv, dtype=torch.float32, scale=0.3)
    return s


# ---------------------------------------------------------------------------- plain forms
def _quantised(u):
    """(rows, width) values in 8 bits with one scale for each 128 of a row."""
    rows, width = u.shape
    blocks = -(-width // BLOCK)
    full = torch.zeros(rows, blocks * BLOCK, dtype=u.dtype, device=u.device)
    full[:, :width] = u
    full = full.view(rows, blocks, BLOCK)
    scales = full.abs().amax(2).clamp_min(2.0 ** -100) / TOP
    full = (full / scales[..., None]).view(rows, blocks * BLOCK)
    return full[:, :width].to(torch.float8_e4m3fn), scales


class _Chunks:
    """Rows of all sequences as (batch, heads, chunks, 64, ...), zeros behind a sequence's end."""

    def __init__(self, s):
        self.s = s
        self.count = max(1, -(-s["longest"] // CHUNK))
        t = torch.arange(self.count * CHUNK, device=DEVICE)[None]
        lens = (s["offsets"][1:] - s["offsets"][:-1])[:, None]
        self.valid = t < lens
        self.at = torch.where(self.valid, s["offsets"][:-1, None] + t, torch.zeros_like(t))
        self.group = s["heads_v"] // s["heads_k"]

    def spread(self, t):
        """(rows, heads, ...) in 32 bits; key heads once for each of their value heads."""
        if t.shape[1] != self.s["heads_v"]:
            t = t.repeat_interleave(self.group, 1)
        t = t.float()[self.at]
        t = t * self.valid.view(*self.valid.shape, *[1] * (t.dim() - 2))
        return t.unflatten(1, (self.count, CHUNK)).movedim(3, 1)

    def gather(self, t):
        """The rows of a (batch, heads, chunks, 64, ...) tensor."""
        t = t.movedim(1, 3).flatten(1, 2)
        out = torch.empty(self.s["rows"], *t.shape[2:], device=DEVICE)
        out[self.at[self.valid]] = t[self.valid]
        return out

    def keys(self, t):
        """Gradients of value heads summed over a key head's group."""
        return self.gather(t).unflatten(1, (self.s["heads_k"], self.group)).sum(2)


def _inverse(low):
    """(I + low)^-1 of strictly lower triangular matrices, row by row."""
    t = torch.eye(CHUNK, device=DEVICE).expand(low.shape).clone()
    for j in range(1, CHUNK):
        t[..., j, :j] = -(low[..., j, :j, None] * t[..., :j, :j]).sum(-2)
    return t


def _plain_chunks(s):
    """The quantities of every chunk, and the states in front of it."""
    c = _Chunks(s)
    q, k, v, g, beta = (c.spread(s[n]) for n in ("q", "k", "v", "g", "beta"))
    b = g.double().cumsum(-1)
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEVICE).tril()
    decay = torch.exp(torch.where(low, b[..., :, None] - b[..., None, :], -math.inf)).float()
    kk = (k @ k.mT) * decay
    inverse = _inverse(beta[..., None] * kk.tril(-1))
    scale = s["dk"] ** -0.5
    mixed = scale * (q @ k.mT) * decay
    front, back = torch.exp(b).float()[..., None], torch.exp(b[..., -1:] - b).float()[..., None]
    state, states, news = s["h0"], [], []
    for n in range(c.count):
        states.append(state)
        r = beta[:, :, n, :, None] * (v[:, :, n] - front[:, :, n] * (k[:, :, n] @ state))
        u = inverse[:, :, n] @ r
        news.append(u)
        state = front[:, :, n, -1:] * state + (back[:, :, n] * k[:, :, n]).mT @ u
    states, u = torch.stack(states, 2), torch.stack(news, 2)
    o = scale * front * (q @ states) + mixed @ u
    return c, q, k, v, beta, kk, inverse, mixed, front, back, scale, states, u, o, state


def _plain_forward(s):
    out = _plain_chunks(s)
    return {"o": out[0].gather(out[-2]).to(s["q"].dtype), "hT": out[-1]}


def _plain_train(s):
    c, q, k, v, beta, kk, inverse, mixed, front, back, scale, states, u, o, last = _plain_chunks(s)
    dt = s["q"].dtype
    out = {"o": c.gather(o).to(dt), "hT": last}
    do = c.spread(s["do"])
    grad, grads, dr = s["dhT"], [None] * c.count, [None] * c.count
    for n in range(c.count - 1, -1, -1):
        grads[n] = grad                          # the gradient of the state behind the chunk
        du = mixed[:, :, n].mT @ do[:, :, n] + (back[:, :, n] * k[:, :, n]) @ grad
        dr[n] = inverse[:, :, n].mT @ du
        grad = (front[:, :, n, -1:] * grad + (scale * front[:, :, n] * q[:, :, n]).mT @ do[:, :, n]
                - (beta[:, :, n, :, None] * front[:, :, n] * k[:, :, n]).mT @ dr[n])
    grads, dr = torch.stack(grads, 2), torch.stack(dr, 2)
    out["dh0"] = grad
    low = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=DEVICE).tril()
    b = torch.cumsum(c.spread(s["g"]).double(), -1)
    decay = torch.exp(torch.where(low, b[..., :, None] - b[..., None, :], -math.inf)).float()
    dlow = -(dr @ u.mT).tril(-1)
    dmix = (do @ u.mT).tril()
    w = dlow * beta[..., None] * decay
    x = scale * dmix * decay
    kept = k @ states                                            # k S in front of the chunk
    qs, ds, rs = do @ states.mT, u @ grads.mT, dr @ states.mT
    dq = x @ k + scale * front * qs
    dk = x.mT @ q + w @ k + w.mT @ k + back * ds - beta[..., None] * front * rs
    out["dq"], out["dk"] = c.keys(dq).to(dt), c.keys(dk).to(dt)
    out["dv"] = c.gather(beta[..., None] * dr).to(dt)
    dbeta = (dr * (v - front * kept)).sum(-1) + (dlow * kk).sum(-1)
    own_low, own_mix = dlow * beta[..., None] * kk, dmix * mixed
    db = (own_low + own_mix).sum(-1) - (own_low + own_mix).sum(-2)
    db = db + scale * (front * q * qs).sum(-1) - beta * (front * k * rs).sum(-1)
    tail = (back * k * ds).sum(-1)
    db = db - tail
    db[..., -1] += tail.sum(-1) + front[..., -1, 0] * (grads * states).sum((-1, -2))
    dg = db.flip(-1).cumsum(-1).flip(-1)
    out["dg"], out["dbeta"] = c.gather(dg), c.gather(dbeta)
    return out


def _plain_step(s):
    group, at = s["heads_v"] // s["heads_k"], s["slot"].long()
    q, k = (s[n].float().repeat_interleave(group, 1)[..., None] for n in ("q", "k"))
    state = torch.exp(s["g"])[..., None, None] * s["state"][at]
    delta = s["beta"][..., None] * (s["v"].float() - (k * state).sum(2))
    state = state + k * delta[:, :, None]
    s["state"][at] = state
    o = s["dk"] ** -0.5 * (q * state).sum(2)
    return {"o": o.to(s["q"].dtype), "state": s["state"]}


def _plain_norms(s):
    f, z, x = s["f"].float(), s["z"].float(), s["x"].float()
    n = f * torch.rsqrt((f * f).mean(1, keepdim=True) + EPS) * s["w_post"]
    y = x + s["scale"] * n * (z * torch.sigmoid(z))
    q, scales = _quantised(y * torch.rsqrt((y * y).mean(1, keepdim=True) + EPS) * s["w_pre"])
    return {"y": y.to(s["f"].dtype), "q": q, "scales": scales}


def _spread_scales(q, scales):
    return q.float() * scales.repeat_interleave(BLOCK, 1)[:, :q.shape[1]]


def _plain_gemm(s):
    sw = s["sw"].repeat_interleave(BLOCK, 0)[:s["n"]]
    a, w = _spread_scales(s["a"], s["sa"]), _spread_scales(s["w"], sw)
    return {"y": (a @ w.mT).to(DTYPES[s["dtype"]])}


# ------------------------------------------------------------------------ the library's calls
def _sequences(s, t):
    """How the calls take the rows: packed with offsets, or as (batch, length, ...)."""
    return t if s["packed"] else t.unflatten(0, (s["batch"], -1))


def _own_step(bs, s):
    o = torch.empty(s["batch"], s["heads_v"], s["dv"], dtype=s["q"].dtype, device=DEVICE)
    bs.bs_gdelta_step_batched(s["q"], s["k"], s["v"], s["g"], s["beta"], s["state"], o,
                              slots=s["slot"])
    return {"o": o, "state": s["state"]}


def _own_forward(bs, s, tape=None):
    o = torch.empty(s["rows"], s["heads_v"], s["dv"], dtype=s["q"].dtype, device=DEVICE)
    hT = torch.empty_like(s["h0"])
    work = torch.empty(bs.bs_gdelta_workspace(s["heads_v"], s["batch"], s["rows"]),
                       dtype=torch.uint8, device=DEVICE)
    bs.bs_gdelta_batched(*(_sequences(s, s[n]) for n in ("q", "k", "v", "g", "beta")),
                         _sequences(s, o), work, h0=s["h0"], hT=hT,
                         offsets=s["offsets"] if s["packed"] else None, tape=tape)
    return {"o": o, "hT": hT}


def _own_train(bs, s):
    hk, hv, dk, dv, batch, rows = (s[n] for n in ("heads_k", "heads_v", "dk", "dv", "batch", "rows"))
    tape = torch.empty(bs.bs_gdelta_tape(hv, dk, dv, batch, rows), dtype=torch.uint8, device=DEVICE)
    out = _own_forward(bs, s, tape)
    for n, like in (("dq", "q"), ("dk", "k"), ("dv", "v"), ("dg", "g"), ("dbeta", "beta")):
        out[n] = torch.empty(s[like].shape, dtype=s[like].dtype, device=DEVICE)
    out["dh0"] = torch.empty_like(s["h0"])
    work = torch.empty(bs.bs_gdelta_backward_workspace(hv, dk, dv, batch, rows),
                       dtype=torch.uint8, device=DEVICE)
    bs.bs_gdelta_backward_batched(
        *(_sequences(s, s[n]) for n in ("q", "k", "v", "g", "beta")), tape, _sequences(s, s["do"]),
        *(_sequences(s, out[n]) for n in ("dq", "dk", "dv", "dg", "dbeta")), work, dhT=s["dhT"],
        dh0=out["dh0"], offsets=s["offsets"] if s["packed"] else None)
    return out


def _own_norms(bs, s):
    y = torch.empty_like(s["f"])
    q = torch.empty(s["f"].shape, dtype=torch.float8_e4m3fn, device=DEVICE)
    scales = torch.empty(s["rows"], -(-s["width"] // BLOCK), device=DEVICE)
    bs.bs_gnorm_q8_batched(s["f"], q, scales, y=y, z=s["z"], x=s["x"], w_post=s["w_post"],
                           scale=s["scale"], w_pre=s["w_pre"], eps=EPS, gate=bs.BS_GATE_SILU)
    return {"y": y, "q": q, "scales": scales}


def _own_gemm(bs, s):
    y = torch.empty(s["m"], s["n"], dtype=DTYPES[s["dtype"]], device=DEVICE)
    bs.bs_gemm_q8(s["a"], s["sa"], s["w"], s["sw"], y)
    return {"y": y}


def run(s):
    if own:
        import dense_linear_solvers_gb300 as bs
        return {"gdelta_step": _own_step, "gdelta_forward": _own_forward, "gdelta_train": _own_train,
                "gnorm_q8": _own_norms, "gemm_q8": _own_gemm}[s["op"]](bs, s)
    return {"gdelta_step": _plain_step, "gdelta_forward": _plain_forward,
            "gdelta_train": _plain_train, "gnorm_q8": _plain_norms,
            "gemm_q8": _plain_gemm}[s["op"]](s)


# ------------------------------------------------------------------------ 64-bit definition
def exact(case, seed):
    """The definition in 64 bits: the delta rule row by row and its gradients by the chain rule
    through that loop, the norms and the product by their formulas."""
    raw = prepare(case, seed)
    s = {k: v.double() if torch.is_tensor(v) and v.is_floating_point() else v for k, v in raw.items()}
    if case["op"] == "gemm_q8":
        n, k = case["n"], case["k"]
        col = torch.arange(k, device=DEVICE) // BLOCK
        a = s["a"] * s["sa"][:, col]
        w = s["w"] * s["sw"][torch.arange(n, device=DEVICE) // BLOCK][:, col]
        return {"y": torch.einsum("mk,nk->mn", a, w)}
    if case["op"] == "gnorm_q8":
        return _exact_norms(s)
    group = case["heads_v"] // case["heads_k"]
    own_key = torch.arange(case["heads_v"], device=DEVICE) // group
    q, k = s["q"][:, own_key] * s["dk"] ** -0.5, s["k"][:, own_key]
    v, beta, alpha = s["v"], s["beta"], torch.exp(s["g"])
    if case["op"] == "gdelta_step":
        at = s["slot"].long()
        state = _advance(s["state"][at], k, v, beta, alpha)
        s["state"][at] = state
        return {"o": torch.einsum("bhk,bhkv->bhv", q, state), "state": s["state"]}
    longest, batch = s["longest"], case["batch"]
    if longest * (4 if case["op"] == "gdelta_train" else 1) > 150000:
        return None
    ends = s["offsets"]
    size = ends[1:] - ends[:-1]
    order = torch.arange(longest, device=DEVICE)[:, None]
    valid = order < size[None]
    at = torch.where(valid, ends[:-1][None] + order, torch.zeros_like(order))

    def row(t, n):  # row n of every sequence; past its end a row that changes nothing
        live = valid[n].view(batch, *[1] * (t.dim() - 1))
        return torch.where(live, t[at[n]], torch.zeros_like(t[:1]))

    alpha_of = lambda n: torch.where(valid[n][:, None], alpha[at[n]], torch.ones_like(alpha[:1]))  # noqa: E731
    step = lambda state, n: _advance(state, row(k, n), row(v, n), row(beta, n), alpha_of(n))       # noqa: E731
    state, o, kept, span = s["h0"], torch.empty_like(v), [], 64

    def put(out, n, value):
        out[at[n][valid[n]]] = value[valid[n]]

    for n in range(longest):
        if n % span == 0 and case["op"] == "gdelta_train":
            kept.append(state)
        state = step(state, n)
        put(o, n, torch.einsum("bhk,bhkv->bhv", row(q, n), state))
    out = {"o": o, "hT": state}
    if case["op"] == "gdelta_forward":
        return out
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dg, dbeta, grad = torch.zeros_like(beta), torch.zeros_like(beta), s["dhT"]
    for part in range(len(kept) - 1, -1, -1):
        first = part * span
        states = [kept[part]]
        for n in range(first, min(first + span, longest)):
            states.append(step(states[-1], n))
        for n in range(min(first + span, longest) - 1, first - 1, -1):
            before, after = states[n - first], states[n - first + 1]
            kn, bn, an, don = row(k, n), row(beta, n), alpha_of(n), row(s["do"], n)
            put(dq, n, torch.einsum("bhkv,bhv->bhk", after, don) * s["dk"] ** -0.5)
            grad = grad + row(q, n)[..., None] * don[:, :, None]
            faded = an[..., None, None] * before
            miss = row(v, n) - torch.einsum("bhk,bhkv->bhv", kn, faded)
            ddelta = torch.einsum("bhk,bhkv->bhv", kn, grad)
            put(dv, n, bn[..., None] * ddelta)
            put(dbeta, n, (ddelta * miss).sum(-1))
            dmiss = bn[..., None] * ddelta
            put(dk, n, torch.einsum("bhkv,bhv->bhk", grad, bn[..., None] * miss)
                - torch.einsum("bhkv,bhv->bhk", faded, dmiss))
            grad = grad - kn[..., None] * dmiss[:, :, None]
            put(dg, n, (grad * faded).sum((-1, -2)))
            grad = an[..., None, None] * grad
    add = lambda t: t.unflatten(1, (case["heads_k"], group)).sum(2)  # noqa: E731
    return dict(out, dq=add(dq), dk=add(dk), dv=dv, dg=dg, dbeta=dbeta, dh0=grad)


def _advance(state, k, v, beta, alpha):
    state = alpha[..., None, None] * state
    miss = v - torch.einsum("bhk,bhkv->bhv", k, state)
    return state + k[..., None] * (beta[..., None] * miss)[:, :, None]


def _exact_norms(s):
    f, z, x, w, c, p = (s[k] for k in ("f", "z", "x", "w_post", "scale", "w_pre"))
    rows, width = f.shape
    q1 = 1 / torch.sqrt(torch.einsum("ij,ij->i", f, f) / width + EPS)[:, None]
    y = x + c * (f * q1 * w) * z / (1 + torch.exp(-z))
    u = y / torch.sqrt(torch.einsum("ij,ij->i", y, y) / width + EPS)[:, None] * p
    q, scales = torch.empty_like(u), []
    for at in range(0, width, BLOCK):
        block = u[:, at:at + BLOCK]
        scales.append(torch.clamp(block.abs().max(1).values, min=2.0 ** -100) / TOP)
        t = block / scales[-1][:, None]
        # the nearest number of four significant bits, of the type's subnormal spacing below 2^-6
        unit = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6))) - 3)
        q[:, at:at + BLOCK] = torch.round(t / unit) * unit
    return {"y": y, "q": q, "scales": torch.stack(scales, 1)}
