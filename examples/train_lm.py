"""A small language model trained with Muon, every operator of the library in
its place: the token embedding, layer norms, the output head's cross entropy
with a tied table, and the Muon step on the hidden matrices.

    python examples/train_lm.py [steps]

The model predicts the next token from the present one: embedding, two blocks
x + W2 relu(W1 norm(x)), norm, head.  The data are sequences of a noisy
permutation of the vocabulary, so the loss falls from log(vocab) to about the
noise's entropy.  Hidden matrices are fp32 masters updated by muon_step; the
table and the norms' weights take Adam, which torch computes here.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import newton_schulz_07_gb300 as ns  # noqa: E402

VOCAB, DIM, HIDDEN, BLOCKS, TOKENS = 1000, 256, 512, 2, 2048
NOISE = 0.1  # share of tokens drawn at random
IGNORE = -100


class Adam:
    def __init__(self, params, lr, betas=(0.9, 0.99), eps=1e-8):
        self.params, self.lr, self.betas, self.eps, self.t = params, lr, betas, eps, 0
        self.m = [torch.zeros_like(p) for p in params]
        self.v = [torch.zeros_like(p) for p in params]

    def step(self, grads):
        self.t += 1
        b1, b2 = self.betas
        for p, g, m, v in zip(self.params, grads, self.m, self.v):
            m.lerp_(g, 1 - b1)
            v.lerp_(g * g, 1 - b2)
            p.addcdiv_(m / (1 - b1 ** self.t), (v / (1 - b2 ** self.t)).sqrt_().add_(self.eps), value=-self.lr)


class Model:
    def __init__(self, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, scale):
            return torch.randn(shape, generator=g, device="cuda") * scale

        self.table = normal(VOCAB, DIM, scale=0.02)
        self.w1 = [normal(HIDDEN, DIM, scale=DIM ** -0.5) for _ in range(BLOCKS)]
        self.w2 = [normal(DIM, HIDDEN, scale=HIDDEN ** -0.5) for _ in range(BLOCKS)]
        self.gain = [torch.ones(DIM, device="cuda") for _ in range(BLOCKS + 1)]
        self.bias = [torch.zeros(DIM, device="cuda") for _ in range(BLOCKS + 1)]
        self.momentum = [torch.zeros_like(w) for w in self.w1 + self.w2]
        self.adam = Adam([self.table] + self.gain + self.bias, lr=3e-3)

    def step(self, tokens, targets, lr=0.02):
        """One training step; returns the mean loss (on the device)."""
        table = self.table.bfloat16()
        w1, w2 = [w.bfloat16() for w in self.w1], [w.bfloat16() for w in self.w2]
        # Forward.
        x = ns.muon_embed(table, tokens, scale=math.sqrt(DIM))
        kept = []
        for i in range(BLOCKS):
            n, mean, rstd = ns.muon_layer_norm(x, self.gain[i], self.bias[i])
            a = torch.relu(n @ w1[i].t())
            kept.append((x, n, mean, rstd, a))
            x = x + a @ w2[i].t()
        n, mean, rstd = ns.muon_layer_norm(x, self.gain[-1], self.bias[-1])
        # The head's loss, its gradient, and the tied table's in fp32.
        dtable = torch.empty_like(self.table)
        loss, dn, _ = ns.muon_head_loss_grad(n, table, targets, ignore_index=IGNORE, dtable=dtable)
        # Backward.
        dgain, dbias, dw1, dw2 = [None] * (BLOCKS + 1), [None] * (BLOCKS + 1), [None] * BLOCKS, [None] * BLOCKS
        dx, dgain[-1], dbias[-1] = ns.muon_layer_norm_grad(dn, x, self.gain[-1], mean, rstd)
        for i in reversed(range(BLOCKS)):
            x, n, mean, rstd, a = kept[i]
            da = (dx @ w2[i]) * (a > 0)
            dw2[i], dw1[i] = (dx.t() @ a).float(), (da.t() @ n).float()
            dxn, dgain[i], dbias[i] = ns.muon_layer_norm_grad(da @ w1[i], x, self.gain[i], mean, rstd)
            dx = dx + dxn
        ns.muon_embed_grad(dx, tokens, VOCAB, scale=math.sqrt(DIM), dtable=dtable, accumulate=True)
        # Update: Muon for the hidden matrices, Adam for the rest.
        for w, m, g in zip(self.w1 + self.w2, self.momentum, dw1 + dw2):
            ns.muon_step(w, m, g, lr=lr)
        self.adam.step([dtable] + dgain + dbias)
        return loss.sum() / (targets != IGNORE).sum()

    def evaluate(self, tokens, targets):
        table = self.table.bfloat16()
        x = ns.muon_embed(table, tokens, scale=math.sqrt(DIM))
        for i in range(BLOCKS):
            n, _, _ = ns.muon_layer_norm(x, self.gain[i], self.bias[i])
            x = x + torch.relu(n @ self.w1[i].bfloat16().t()) @ self.w2[i].bfloat16().t()
        n, _, _ = ns.muon_layer_norm(x, self.gain[-1], self.bias[-1])
        return ns.muon_head_loss(n, table, targets, ignore_index=IGNORE).sum() / (targets != IGNORE).sum()


def batches(seed=1):
    """Endless (tokens, targets): targets a fixed permutation of tokens but for
    the noise; one target in sixteen carries no loss."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    follow = torch.randperm(VOCAB, generator=g, device="cuda")
    while True:
        tokens = torch.randint(0, VOCAB, (TOKENS,), generator=g, device="cuda")
        noise = torch.rand(TOKENS, generator=g, device="cuda") < NOISE
        targets = torch.where(noise, torch.randint(0, VOCAB, (TOKENS,), generator=g, device="cuda"), follow[tokens])
        targets[::16] = IGNORE
        yield tokens, targets


def main(steps=150, report=25):
    model, data = Model(), batches()
    losses = []
    for i in range(steps):
        losses.append(model.step(*next(data)))
        if report and i % report == 0:
            print(f"step {i:4d}  loss {float(losses[-1]):.4f}", flush=True)
    final = float(model.evaluate(*next(data)))
    if report:
        print(f"after {steps} steps: loss {final:.4f} on new data (log vocab {math.log(VOCAB):.4f})")
    return [float(v) for v in losses], final


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 150)
