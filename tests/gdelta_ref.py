"""Plain 64-bit reference of the gated delta rule, row by row, with bounds in the Frobenius norm of a
sequence's and head's results.

Every operand of a matrix product in the kernels is within 2^-18 of itself (two BF16 terms; the product
leaves out their last one, 2^-18 too) and every sum is FP32, so that a state made of terms k d^T is
off by a small multiple of 2^-18 of the terms' norms. m_t = a m_(t-1) + |k_t| |d_t| bounds the norm of
the state's terms without their cancellation; the map from one state to the next does not stretch
errors (|k| <= 1, 0 <= beta <= 2, a <= 1), nor does the solution of a chunk's system: its inverse's
entries are products of such maps. What a row adds is a few products of two split operands and the
solution's 64 terms, whose independent errors add to sqrt(64) = 8 of one: ROW = 32 of 2^-18, doubled
for the sums."""
import torch

UNIT = 2.0 ** -18
ROW = 64
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
        self.before, self.m_before, self.d = {}, {}, torch.zeros_like(v)
        for b, (first, end) in enumerate(spans):
            S, m = self.h0[b], norm(self.h0[b], 2)
            for t in range(first, end):
                self.before[t], self.m_before[t] = S, m
                S, m = self._row(t, S, m)
                self.o[t] = self.scale * torch.einsum("hk,hkv->hv", self.q[t], S)
                self.size["o"][t] = abs(self.scale) * norm(self.q[t]) * m * ROW
            self.hT[b], self.size["hT"][b] = S, m * ROW

    def _row(self, t, S, m):
        S = self.a[t][:, None, None] * S
        miss = self.v[t] - torch.einsum("hk,hkv->hv", self.k[t], S)
        self.d[t] = self.beta[t][:, None] * miss
        kn = norm(self.k[t])
        # the terms of d: v and k S, without their cancellation
        add = self.beta[t].abs() * kn * (norm(self.v[t]) + kn * self.a[t] * m)
        return S + self.k[t][..., None] * self.d[t][:, None], self.a[t] * m + add

    def close(self, name, got, kind):
        """Whether `got` is within the bound; kind: its type."""
        got, want = got.double(), getattr(self, name)
        dims = 2 if name in ("hT", "dh0") else 1 if want.dim() == 3 else 0
        far = norm(got - want, dims) if dims else (got - want).abs()
        size = norm(want, dims) if dims else want.abs()
        allowed = UNIT * self.size[name] * (1 + HALF_STEP[kind]) + HALF_STEP[kind] * size \
            + 1e-30 + (2.0 ** -24 * want.shape[-1] ** 0.5 if kind == torch.float16 else 0)
        return bool((far <= allowed).all()), float((far / allowed).max()) if far.numel() else 0.0
