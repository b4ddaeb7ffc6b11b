"""How near the gated delta rule's FP32 results have to be tells two BF16 terms an operand from one: a restatement
of the chunk form on the CPU, whose operands are cut as the kernels' are, against the definition in 64 bits."""
import pytest
import torch

from tests.delta_forms import allowed
from tests.gdelta_ref import Delta

CHUNK = 64


def cut(x, terms):
    hi = x.bfloat16().float()
    return hi if terms == 1 else hi + (x - hi).bfloat16().float()


def chunk_form(q, k, v, g, beta, h0, state=2, prepared=2, solution=2):
    """o and the last state of one sequence, (rows, heads, ...) in FP32; the operands' terms by what they are."""
    q, k, v, g, beta = (t.transpose(0, 1) for t in (q, k, v, g, beta))
    scale, S, out = q.shape[2] ** -0.5, h0, []
    for first in range(0, q.shape[1], CHUNK):
        Q, K, V, b = (t[:, first:first + CHUNK] for t in (q, k, v, beta))
        s = g[:, first:first + CHUNK].double().cumsum(1)
        n = s.shape[1]
        low = torch.ones(n, n, dtype=torch.bool).tril()
        D = torch.exp(torch.where(low, s[:, :, None] - s[:, None], -torch.inf)).float()
        front, back = torch.exp(s).float()[..., None], torch.exp(s[:, -1:] - s).float()[..., None]
        Q2, K2 = cut(Q, 2), cut(K, 2)
        N = (K2 @ K2.mT * D).tril(-1)
        inverse = cut(torch.linalg.inv(torch.eye(n) + N * b[:, None]), prepared)
        mixing = cut(scale * (Q2 @ K2.mT) * D, prepared)
        S2 = cut(S, state)
        M = inverse @ cut(cut(V, 2) - front * (K2 @ S2), solution)
        U = b[..., None] * M
        out.append(scale * front * (Q2 @ S2) + mixing @ cut(U, solution))
        S = front[:, -1:] * S + K2.mT @ cut(back * U, solution)
    return torch.cat(out, 1).transpose(0, 1), S


@pytest.mark.parametrize("length, heads, dk, dv", [(64, 2, 64, 64), (150, 4, 128, 128), (190, 3, 93, 77), (65, 2, 104, 120)])
def test_one_term_is_seen(length, heads, dk, dv):
    gen = torch.Generator().manual_seed(length)
    new = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    unit = lambda t: t / t.norm(dim=-1, keepdim=True)  # noqa: E731
    q, k = unit(new(length, heads, dk)), unit(new(length, heads, dk) + new(heads, dk))
    v, h0 = new(length, heads, dv), new(1, heads, dk, dv)
    g, beta = -torch.rand(length, heads, generator=gen) ** 3, torch.sigmoid(new(length, heads))
    ref = Delta(*(t.double() for t in (q, k, v, g, beta)), [(0, length)], h0=h0.double())

    def far(**terms):
        o, S = chunk_form(q, k, v, g, beta, h0[0], **terms)
        return (float((a.double() - b).norm() / b.norm()) / allowed(length) for a, b in ((o, ref.o), (S, ref.hT[0])))

    assert max(far()) <= 0.5
    for terms in (dict(state=1), dict(prepared=1), dict(solution=1)):
        assert max(far(**terms)) > 1.5, terms
