"""Plain 64-bit reference of the gated delta rule, row by row, with bounds in the Frobenius norm of a
sequence's and head's results.

Every operand of a matrix product in the kernels is within 2^-18 of itself (two BF16 terms; the product
leaves out their last one, 2^-18 too) and every sum is FP32. A row adds its term k d^T, d = beta (v - a S^T k),
to the state, off by a small multiple of 2^-18 of |k| beta (|v| + a |k| |S|): a few products of two split
operands, and the solution's 64 terms, whose independent errors add to sqrt(64) = 8 of one: ROW = 16 of
2^-18, doubled for the sums. A chunk takes the state itself as split operand: 4 of 2^-18 of its norm.
The map from one state to the next does not stretch errors (|k| <= 1, 0 <= beta <= 2, a <= 1), so that
they add up with the decays alone. The same holds for the state's gradient on the way back."""
import torch

UNIT = 2.0 ** -18
ROW = 32
STATE = 4
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def norm(t, dims=1):
    return t.flatten(-dims).norm(dim=-1)


class Delta:
    """o, hT and, after backward(), dq, dk, dv, dg, dbeta, dh0, from float64 tensors of rows:
    q, k (rows, heads_k, dk), v (rows, heads_v, dv), g, beta (rows, heads_v), h0 (batch, heads_v, dk, dv);
    spans: (start, end) of each sequence. size[name]: what errors of `name` are multiples of UNIT of, by
    row and head (by sequence and head for states)."""

    def __init__(self, q, k, v, g, beta, spans, scale=None, h0=None):
        heads_k, heads_v = q.shape[1], v.shape[1]
        self.group, self.spans = heads_v // heads_k, spans
        self.scale = q.shape[2] ** -0.5 if scale is None else scale
        wide = lambda t: t.repeat_interleave(self.group, 1)  # noqa: E731
        self.q, self.k, self.v, self.beta, self.a = wide(q), wide(k), v, beta, torch.exp(g)
        batch, (rows, _, dv), dk = len(spans), v.shape, q.shape[2]
        self.h0 = v.new_zeros(batch, heads_v, dk, dv) if h0 is None else h0
        self.o, self.hT = torch.zeros_like(v), self.h0.clone()
        self.size = {"o": v.new_zeros(rows, heads_v), "hT": v.new_zeros(batch, heads_v)}
        self.before, self.off, self.miss = {}, {}, torch.zeros_like(v)
        for b, (first, end) in enumerate(spans):
            S, off = self.h0[b], v.new_zeros(heads_v)
            for t in range(first, end):
                if (t - first) % 64 == 0:
                    off = off + STATE * norm(S, 2)
                self.before[t], self.off[t] = S, off
                a, kn = self.a[t], norm(self.k[t])
                size = norm(self.v[t]) + kn * a * norm(S, 2)
                S = a[:, None, None] * S
                self.miss[t] = v[t] - torch.einsum("hk,hkv->hv", self.k[t], S)
                S = S + self.k[t][..., None] * (beta[t][:, None] * self.miss[t])[:, None]
                off = a * off + ROW * self.beta[t].abs() * kn * size
                self.o[t] = self.scale * torch.einsum("hk,hkv->hv", self.q[t], S)
                self.size["o"][t] = abs(self.scale) * norm(self.q[t]) * (
                    off + ROW * (a * norm(self.before[t], 2) + beta[t].abs() * kn * size))
            self.hT[b], self.size["hT"][b] = S, off + norm(S, 2)
            self.last = S

    def backward(self, do, dhT=None):
        rows, heads, dv = self.v.shape
        like = {"dq": self.q, "dk": self.k, "dv": self.v, "dg": self.beta, "dbeta": self.beta}
        out = {n: torch.zeros_like(t) for n, t in like.items()}
        size = {n: self.v.new_zeros(rows, heads) for n in like}
        self.dh0 = torch.zeros_like(self.h0) if dhT is None else dhT.clone()
        size["dh0"] = self.v.new_zeros(len(self.spans), heads)
        for b, (first, end) in enumerate(self.spans):
            G, off = self.dh0[b], self.v.new_zeros(heads)
            for t in range(end - 1, first - 1, -1):
                if (t - first) % 64 == 63 or t == end - 1:
                    off = off + STATE * norm(G, 2)
                q, k, a, beta, S = self.q[t], self.k[t], self.a[t], self.beta[t], self.before[t]
                qn, kn, dn, bn, sn = norm(q), norm(k), norm(do[t]), beta.abs(), a * norm(S, 2)
                far = a * self.off[t]                    # of the faded state
                after = a[:, None, None] * S + k[..., None] * (beta[:, None] * self.miss[t])[:, None]
                s = abs(self.scale)
                out["dq"][t] = self.scale * torch.einsum("hkv,hv->hk", after, do[t])
                vn = norm(self.v[t]) + kn * sn           # the terms of what is missed
                size["dq"][t] = s * dn * (far + ROW * (sn + bn * kn * vn))
                gn = norm(G, 2) + s * qn * dn            # the terms of the gradient behind the row
                goff = off + ROW * s * qn * dn
                G = G + self.scale * q[..., None] * do[t][:, None]
                dd = torch.einsum("hk,hkv->hv", k, G)
                e_dd, e_miss = kn * goff + ROW * kn * gn, kn * far + ROW * vn
                out["dv"][t], size["dv"][t] = beta[:, None] * dd, bn * e_dd
                out["dbeta"][t] = (dd * self.miss[t]).sum(-1)
                size["dbeta"][t] = e_dd * vn + kn * gn * e_miss
                out["dk"][t] = torch.einsum("hkv,hv->hk", G, beta[:, None] * self.miss[t]) \
                    - torch.einsum("hkv,hv->hk", a[:, None, None] * S, beta[:, None] * dd)
                size["dk"][t] = bn * (goff * vn + gn * e_miss + far * kn * gn + sn * e_dd
                                      + ROW * gn * (vn + kn * sn))
                G = G - k[..., None] * (beta[:, None] * dd)[:, None]
                out["dg"][t] = (G * a[:, None, None] * S).sum((-1, -2))
                # summed from the chunk's end: 64 terms of this size
                size["dg"][t] = 8 * ROW * gn * (1 + bn * kn ** 2) * (sn + bn * kn * vn) \
                    + goff * sn + gn * far
                G = a[:, None, None] * G
                off = a * (goff + ROW * bn * kn ** 2 * gn)
            self.dh0[b], size["dh0"][b] = G, off + norm(G, 2)
        # a chunk's sums reach all of its rows
        for first, end in self.spans:
            for c in range(first, end, 64):
                part = size["dg"][c:min(c + 64, end)]
                part[:] = part.amax(0)
        add = lambda t: t.unflatten(1, (-1, self.group)).sum(2)  # noqa: E731
        self.dq, self.dk = add(out["dq"]), add(out["dk"])
        size["dq"], size["dk"] = add(size["dq"]), add(size["dk"])
        self.dv, self.dg, self.dbeta = out["dv"], out["dg"], out["dbeta"]
        self.size.update(size)
        return self

    def close(self, name, got, kind):
        """Whether `got` is within the bound, and how much of it it takes; kind: its type."""
        got, want = got.double(), getattr(self, name)
        dims = 2 if name in ("hT", "dh0") else 1 if want.dim() == 3 else 0
        far = norm(got - want, dims) if dims else (got - want).abs()
        size = norm(want, dims) if dims else want.abs()
        allowed = UNIT * self.size[name] * (1 + HALF_STEP[kind]) + HALF_STEP[kind] * size \
            + 1e-30 + (2.0 ** -25 * want.shape[-1] ** 0.5 if kind == torch.float16 else 0)
        return bool((far <= allowed).all()), float((far / allowed).max()) if far.numel() else 0.0
