"""A small recurrent sequence model on the row operators: training, then generation token by token.

Each block is a product that gives the recurrence's input, its two gates and the block's gate; the
gated linear recurrence over the sequence; and the norm of its output, fused with the gate, the residual
scale and the norm in front of the next block. Training runs whole sequences through the forward and
backward calls; generation starts from the prompt's final states and advances them by
bs_grec_step_batched, one token at a time.

    python examples/recurrent_block.py [--dtype bf16] [--steps 60]
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import dense_linear_solvers_gb300 as bs  # noqa: E402


class Recurrence(torch.autograd.Function):
    """h of a (batch, length, 3 * width) product: x, r, i as column windows, no copies."""

    @staticmethod
    def forward(ctx, p, lam):
        batch, length, width = p.shape[0], p.shape[1], p.shape[2] // 3
        h = torch.empty(batch, length, width, dtype=p.dtype, device=p.device)
        tape = torch.empty(bs.bs_grec_tape_rows(batch, batch * length), width, device=p.device)
        bs.bs_grec_batched(*p.split(width, -1), lam, h, tape=tape)
        ctx.save_for_backward(p, lam, tape)
        return h

    @staticmethod
    def backward(ctx, dh):
        p, lam, tape = ctx.saved_tensors
        batch, length, width = p.shape[0], p.shape[1], p.shape[2] // 3
        dp, dlam = torch.empty_like(p), torch.empty_like(lam)
        work = torch.empty(bs.bs_grec_backward_workspace(width, batch, batch * length),
                           dtype=torch.uint8, device=p.device)
        bs.bs_grec_backward_batched(*p.split(width, -1), lam, tape, dh.contiguous(),
                                    *dp.split(width, -1), dlam, work)
        return dp, dlam


class BlockNorms(torch.autograd.Function):
    """(y, u): the new residual and the next block's input."""

    @staticmethod
    def forward(ctx, f, z, x, w_post, scale, w_pre):
        y, u = torch.empty_like(x), torch.empty_like(x)
        bs.bs_gnorm_batched(f, y, z=z, x=x, w_post=w_post, scale=scale, w_pre=w_pre, u=u)
        ctx.save_for_backward(f, z, x, w_post, scale, w_pre)
        return y, u

    @staticmethod
    def backward(ctx, dy, du):
        f, z, x, w_post, scale, w_pre = ctx.saved_tensors
        df, dz, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        sums = [torch.empty_like(w) for w in (w_post, scale, w_pre)]
        work = torch.empty(bs.bs_gnorm_backward_workspace(f.shape[-1], f.numel() // f.shape[-1]),
                           dtype=torch.uint8, device=f.device)
        bs.bs_gnorm_backward_batched(
            f, dy.contiguous(), df, work, z=z, x=x, w_post=w_post, scale=scale, w_pre=w_pre,
            du=du.contiguous(), dz=dz, dx=dx, dw_post=sums[0], dscale=sums[1], dw_pre=sums[2])
        return (df, dz, dx, *sums)


class Model(torch.nn.Module):
    def __init__(self, vocabulary, width, blocks, dtype):
        super().__init__()
        self.width, self.dtype = width, dtype
        new = lambda *shape: torch.nn.Parameter(torch.randn(*shape) * shape[0] ** -0.5)  # noqa: E731
        vec = lambda v: torch.nn.Parameter(torch.full((width,), v))                      # noqa: E731
        self.embed = torch.nn.Parameter(torch.randn(vocabulary, width))
        self.out = new(width, vocabulary)
        self.products = torch.nn.ParameterList([new(width, 4 * width) for _ in range(blocks)])
        # decays of the channels between 0.9 and 0.999 at an open gate
        keep = torch.linspace(0.9, 0.999, width)
        self.lam = torch.nn.ParameterList(
            [torch.nn.Parameter(torch.log(torch.expm1(-torch.log(keep) / 8))) for _ in range(blocks)])
        self.w_post = torch.nn.ParameterList([vec(1.0) for _ in range(blocks)])
        self.scale = torch.nn.ParameterList([vec(0.5) for _ in range(blocks)])
        self.w_pre = torch.nn.ParameterList([vec(1.0) for _ in range(blocks + 1)])

    def _first(self, tokens):
        """The embedded tokens and the first block's input: the norm alone."""
        x = self.embed[tokens].to(self.dtype)
        if torch.is_grad_enabled():
            zero = torch.zeros_like(x)
            one = torch.ones(self.width, device=x.device)
            return BlockNorms.apply(zero, zero, x, one, one, self.w_pre[0])
        u = torch.empty_like(x)
        bs.bs_gnorm_batched(x, w_pre=self.w_pre[0].detach(), u=u)
        return x, u

    def forward(self, tokens):
        """Logits of every position of (batch, length) tokens."""
        x, u = self._first(tokens)
        for k, product in enumerate(self.products):
            p = u @ product.to(self.dtype)
            h = Recurrence.apply(p[..., :3 * self.width], self.lam[k])
            x, u = BlockNorms.apply(h, p[..., 3 * self.width:], x, self.w_post[k], self.scale[k],
                                    self.w_pre[k + 1])
        return u.float() @ self.out

    @torch.no_grad()
    def prompt(self, tokens):
        """Logits behind a prompt, and every block's state there."""
        x, u = self._first(tokens)
        batch, states = tokens.shape[0], []
        for k, product in enumerate(self.products):
            p = u @ product.to(self.dtype)
            a, r, i, z = p.split(self.width, -1)
            h, state = torch.empty_like(x), torch.empty(batch, self.width, device=x.device)
            bs.bs_grec_batched(a, r, i, self.lam[k].detach(), h, hT=state)
            states.append(state)
            x, u = BlockNorms.apply(h, z, x, self.w_post[k], self.scale[k], self.w_pre[k + 1])
        return u[:, -1].float() @ self.out, states

    @torch.no_grad()
    def step(self, tokens, states):
        """Logits behind one more token of each sequence; the states advance in place."""
        x, u = self._first(tokens)
        for k, product in enumerate(self.products):
            p = u @ product.to(self.dtype)
            a, r, i, z = p.split(self.width, -1)
            h = torch.empty_like(x)
            bs.bs_grec_step_batched(a, r, i, self.lam[k].detach(), states[k], h)
            x, u = BlockNorms.apply(h, z, x, self.w_post[k], self.scale[k], self.w_pre[k + 1])
        return u.float() @ self.out


def sequences(batch, length, vocabulary, device):
    """Sequences in which a token is followed by its fixed successor or, in two of three sequences, by
    that token's successor: what came before tells which."""
    jump = 1 + (torch.rand(batch, 1, device=device) < 2 / 3).long()
    start = torch.randint(vocabulary, (batch, 1), device=device)
    place = (start + jump * torch.arange(length + 1, device=device)) % vocabulary
    order = torch.randperm(vocabulary, generator=torch.Generator().manual_seed(1)).to(device)
    return order[place]


def main(argv=None):
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--dtype", choices=("f32", "bf16", "f16"), default="f32")
    ap.add_argument("--steps", type=int, default=60)
    ap.add_argument("--width", type=int, default=128)
    ap.add_argument("--seed", type=int, default=0)
    a = ap.parse_args(argv)
    dtype = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}[a.dtype]
    torch.manual_seed(a.seed)
    vocabulary, batch, length = 32, 32, 64
    model = Model(vocabulary, a.width, 2, dtype).cuda()
    optimizer = torch.optim.Adam(model.parameters(), 3e-3)
    losses = []
    for step in range(a.steps):
        data = sequences(batch, length, vocabulary, "cuda")
        logits = model(data[:, :-1])
        loss = torch.nn.functional.cross_entropy(logits.flatten(0, 1), data[:, 1:].flatten())
        optimizer.zero_grad()
        loss.backward()
        optimizer.step()
        losses.append(loss.item())
        if step % 10 == 0 or step + 1 == a.steps:
            print(f"step {step:4d}  loss {losses[-1]:.4f}")
    # generation: the states behind a prompt, then single tokens; the whole sequence at once has to
    # give the same logits
    data = sequences(4, 40, vocabulary, "cuda")
    logits, states = model.prompt(data[:, :24])
    with torch.no_grad():
        whole = model(data[:, :40])
    far = [(logits - whole[:, 23]).abs().max().item()]
    for t in range(24, 40):
        logits = model.step(data[:, t], states)
        far.append((logits - whole[:, t]).abs().max().item())
    print(f"single tokens against the whole sequence: logits differ by at most {max(far):.2e}")
    return losses, max(far), whole.abs().max().item()


if __name__ == "__main__":
    main()
