"""A small language model of gated delta-rule blocks: trained on associative recall, then answering token by token.

Each block reads the normed stream h, projects it to q, k, v, a gate z, a log decay g and a write strength beta, runs the
gated delta rule, and hands its output to the block norm, which adds it to the residual stream and norms the stream for
the next block in the same pass:

    o = gated_delta_rule(q, k, v, g, beta) W_o;   x = x + scale rms_norm(o) w_post silu(z);   h = rms_norm(x) w_pre

Training takes gdr_forward and norm_forward, whose gradients (gdr_backward, norm_backward) torch's graph calls; answering
takes a prompt with gdr_forward, whose last states fill a pool, and goes on with gdr_step on that pool.

    python examples/delta_block.py [--steps 100] [--dtype bf16|f16|f32]
"""

import argparse
import os
import sys

import torch
import torch.nn.functional as F

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import deterministic_fp32_gemm_amd as sdm  # noqa: E402

TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


class Block(torch.nn.Module):
    def __init__(self, D, Hk, Hv, dk, dv):
        super().__init__()
        self.heads = Hk, Hv, dk, dv
        self.parts = [Hk * dk, Hk * dk, Hv * dv, D, Hv, Hv]
        self.w_in = torch.nn.Parameter(torch.randn(sum(self.parts), D) * D ** -0.5)
        self.w_out = torch.nn.Parameter(torch.randn(D, Hv * dv) * (Hv * dv) ** -0.5)
        self.w_post = torch.nn.Parameter(torch.ones(D))
        self.w_pre = torch.nn.Parameter(torch.ones(D))
        self.scale = torch.nn.Parameter(torch.full((D,), 0.5))

    def operands(self, h):
        Hk, Hv, dk, dv = self.heads
        B, T, _ = h.shape
        q, k, v, z, g, beta = F.linear(h, self.w_in.to(h.dtype)).split(self.parts, -1)
        q, k = (F.normalize(t.float().view(B, T, Hk, dk), dim=-1).to(h.dtype) for t in (q, k))
        return q, k, v.unflatten(-1, (Hv, dv)), -F.softplus(g.float() - 4), torch.sigmoid(beta.float()), z

    def forward(self, x, h):
        """Whole sequences: the stream, the next block's input and the states after the last token."""
        q, k, v, g, beta, z = self.operands(h)
        o, state = sdm.gdr_forward(q, k, v, g, beta)
        x, h, _ = sdm.norm_forward(x, F.linear(o.flatten(2), self.w_out.to(h.dtype)), z, self.w_post, self.w_pre,
                                   self.scale)
        return x, h, state

    def step(self, x, h, pool, slots):
        """One token of each stream, its state at pool[slots] updated in place."""
        q, k, v, g, beta, z = self.operands(h)
        o = sdm.gdr_step(q, k, v, g, beta, pool, slots=slots)
        x, h, _ = sdm.norm_forward(x, F.linear(o.flatten(2), self.w_out.to(h.dtype)), z, self.w_post, self.w_pre,
                                   self.scale)
        return x, h


class Model(torch.nn.Module):
    def __init__(self, vocab=64, D=256, Hk=2, Hv=4, dk=64, dv=64, layers=2, dtype=torch.bfloat16):
        super().__init__()
        self.dtype = dtype
        self.embed = torch.nn.Parameter(torch.randn(vocab, D))
        self.near = torch.nn.Parameter(torch.randn(2, D) * 0.5 + 0.5)     # each token also sees the one before it
        self.w_first = torch.nn.Parameter(torch.ones(D))
        self.blocks = torch.nn.ModuleList(Block(D, Hk, Hv, dk, dv) for _ in range(layers))
        self.head = torch.nn.Parameter(torch.randn(vocab, D) * D ** -0.5)

    def begin(self, tokens, before):
        x = (self.embed[tokens] * self.near[0] + self.embed[before] * self.near[1]).to(self.dtype)
        return x, sdm.norm_forward(x, None, None, None, self.w_first, None, act="none")[1]

    def forward(self, tokens):
        x, h = self.begin(tokens, F.pad(tokens[:, :-1], (1, 0)))
        states = []
        for block in self.blocks:
            x, h, s = block(x, h)
            states.append(s)
        return F.linear(h, self.head.to(h.dtype)).float(), states

    @torch.no_grad()
    def step(self, tokens, before, pools, slots):
        x, h = self.begin(tokens[:, None], before[:, None])
        for block, pool in zip(self.blocks, pools):
            x, h = block.step(x, h, pool, slots)
        return F.linear(h, self.head.to(h.dtype)).float()[:, 0]


def recall(batch, pairs, gen, vocab=64):
    """Sequences of key, value, key, value ..., and then the keys again, in another order, each with its value."""
    half = vocab // 2
    keys = torch.stack([torch.randperm(half, generator=gen)[:pairs] for _ in range(batch)])
    values = torch.randint(half, vocab, (batch, pairs), generator=gen)
    order = torch.stack([torch.randperm(pairs, generator=gen) for _ in range(batch)])
    first = torch.stack([keys, values], -1).flatten(1)
    again = torch.stack([keys.gather(1, order), values.gather(1, order)], -1).flatten(1)
    return torch.cat([first, again], 1).cuda()


def train(model, steps, pairs=16, batch=64, lr=3e-3, seed=0, log=None):
    """The loss of every step, on the values of the second half."""
    gen = torch.Generator().manual_seed(seed)
    opt = torch.optim.AdamW(model.parameters(), lr=lr, weight_decay=0.0)
    losses = []
    for i in range(steps):
        tokens = recall(batch, pairs, gen)
        logits, _ = model(tokens)
        loss = F.cross_entropy(logits[:, 2 * pairs::2].flatten(0, 1), tokens[:, 2 * pairs + 1::2].flatten())
        opt.zero_grad()
        loss.backward()
        opt.step()
        losses.append(loss.detach())
        if log is not None and (i % 20 == 0 or i == steps - 1):
            log(f"step {i}: loss {float(losses[-1]):.3f}")
    return [float(x) for x in losses]


@torch.no_grad()
def answer(model, tokens, prompt):
    """Logits of the tokens from `prompt` on, one token at a time from the states that the prompt leaves."""
    _, states = model(tokens[:, :prompt])
    B = tokens.shape[0]
    slots = torch.arange(B, dtype=torch.int32, device=tokens.device).flip(0).contiguous()
    pools = [s[slots.long()].contiguous() for s in states]          # stream b's state lies at pool[slots[b]]
    return torch.stack([model.step(tokens[:, t], tokens[:, t - 1], pools, slots)
                        for t in range(prompt, tokens.shape[1])], 1)


def main():
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--steps", type=int, default=100)
    ap.add_argument("--dtype", choices=TYPES, default="bf16")
    args = ap.parse_args()
    torch.manual_seed(0)
    model = Model(dtype=TYPES[args.dtype]).cuda()
    train(model, args.steps, log=print)
    tokens = recall(64, 16, torch.Generator().manual_seed(1))
    logits = answer(model, tokens, 32)[:, ::2]
    right = (logits.argmax(-1) == tokens[:, 33::2]).float().mean()
    print(f"recalled token by token: {100 * float(right):.1f}% of {logits.shape[0] * logits.shape[1]} values")


if __name__ == "__main__":
    main()
