"""A feed-forward language model trained and sampled with the layer operators.

    python examples/ffn_lm.py [--steps 200] [--dtype bf16]

Each token predicts the next one: an embedding (which is the output head too),
and per layer a linear layer and a gated feed-forward block, both with their
input as residual.  The tokens follow a noisy permutation of the vocabulary,
so the loss falls from log(vocabulary) towards the noise's entropy.  Every
product, activation, loss, gradient and the clipping run in libpgemm; torch
looks up embeddings and updates the fp32 copies of the weights.
"""
import argparse
import math
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
if ROOT not in sys.path:
    sys.path.insert(0, ROOT)

import torch  # noqa: E402

import software_pipelined_tiled_pgemm_amd as pg  # noqa: E402

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}
NAMES = ("w", "b", "w_in", "w_out")


class Model:
    """fp32 weights (`master`) and the 16-bit copies that the operators take
    (`weights`): the embedding, then NAMES for each layer."""

    def __init__(self, vocab=1000, width=256, hidden=512, layers=2, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std
        self.layers, self.dtype = layers, dtype
        self.master = {"embed": normal(vocab, width, std=1.0)}
        for i in range(layers):
            self.master["w%d" % i] = normal(width, width, std=0.5 * width ** -0.5)
            self.master["b%d" % i] = torch.zeros(width, device="cuda")
            self.master["w_in%d" % i] = normal(width, 2 * hidden, std=width ** -0.5)
            self.master["w_out%d" % i] = normal(hidden, width, std=0.5 * hidden ** -0.5)
        self.scale = width ** -0.5  # of the head, applied to its input
        self.momentum = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.refresh()

    def refresh(self):
        self.weights = {k: v.to(self.dtype) for k, v in self.master.items()}

    def body(self, tokens, keep=None):
        """Activations of the last layer; `keep` receives what the backward
        pass needs."""
        p = self.weights
        x = p["embed"][tokens]
        for i in range(self.layers):
            w, b, w_in, w_out = (p[n + str(i)] for n in NAMES)
            z = gate_up = None
            if keep is not None:
                z = torch.empty(len(x), w.shape[1], dtype=x.dtype, device=x.device)
                # bf16's kept form is no bf16: 16 bits that only pffn_bwd reads
                form = torch.int16 if x.dtype is torch.bfloat16 else x.dtype
                gate_up = torch.empty(len(x), w_in.shape[1], dtype=form, device=x.device)
            y = pg.plinear(x, w, bias=b, residual=x, act="gelu", preact=z)
            out = pg.pffn(y, w_in, w_out, residual=y, act="silu", gate_up=gate_up)
            if keep is not None:
                keep.append((x, z, y, gate_up))
            x = out
        return x

    def loss_and_grads(self, tokens, targets):
        p, keep, grads = self.weights, [], {}
        x = self.body(tokens, keep)
        h = x * self.scale
        loss, lse = pg.pxent(h, p["embed"], targets)
        dh, grads["embed"] = pg.pxent_bwd(h, p["embed"], targets, lse)
        dx = dh * self.scale
        for i in reversed(range(self.layers)):
            w, _, w_in, w_out = (p[n + str(i)] for n in NAMES)
            x, z, y, gate_up = keep[i]
            # each input was also the residual, so dy goes to dx directly too
            dy, grads["w_in%d" % i], grads["w_out%d" % i] = pg.pffn_bwd(
                dx, y, w_in, w_out, gate_up, act="silu", dx_residual=dx)
            dx, grads["w%d" % i], grads["b%d" % i] = pg.plinear_bwd(
                dy, x, w, preact=z, act="gelu", dx_residual=dy)
        total = grads["embed"].float().index_add_(0, tokens, dx.float())
        grads["embed"] = total.to(self.dtype)
        return loss, grads

    def step(self, tokens, targets, lr, max_norm=1.0, momentum=0.9):
        loss, grads = self.loss_and_grads(tokens, targets)
        norm = pg.pclip_grad_norm(list(grads.values()), max_norm)
        for k, g in grads.items():
            m = self.momentum[k].mul_(momentum).add_(g.float())
            self.master[k].sub_(m, alpha=lr)
        self.refresh()
        return loss, norm

    def generate(self, token, count):
        """Greedy continuation, one token at a time."""
        head = self.weights["embed"].t().contiguous()
        out = [int(token)]
        for _ in range(count):
            x = self.body(torch.tensor([out[-1]], device="cuda"))
            logits = pg.plinear(x * self.scale, head)
            out.append(int(logits.argmax()))
        return out


def batches(vocab, tokens, noise=0.1, seed=1):
    """(tokens, targets, permutation): the target is the permutation of the
    token, or any token with probability `noise`."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    permutation = torch.randperm(vocab, generator=g, device="cuda")
    while True:
        t = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        other = torch.randint(0, vocab, (tokens,), generator=g, device="cuda")
        noisy = torch.rand(tokens, generator=g, device="cuda") < noise
        yield t, torch.where(noisy, other, permutation[t]), permutation


def train(steps=200, tokens=4096, vocab=1000, dtype="bf16", lr=0.3, report=0):
    model = Model(vocab=vocab, dtype=DTYPES[dtype])
    data = batches(vocab, tokens)
    losses = []
    for i in range(steps):
        t, target, permutation = next(data)
        loss, norm = model.step(t, target, lr)
        losses.append(loss)
        if report and (i % report == 0 or i == steps - 1):
            print("step %4d  loss %.4f  gradient norm %.3f" % (i, float(loss), float(norm)),
                  flush=True)
    return model, [float(v) for v in losses], permutation


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--steps", type=int, default=200)
    ap.add_argument("--tokens", type=int, default=4096)
    ap.add_argument("--vocab", type=int, default=1000)
    ap.add_argument("--dtype", choices=sorted(DTYPES), default="bf16")
    ap.add_argument("--lr", type=float, default=0.3)
    a = ap.parse_args()
    print("log(vocabulary) = %.4f" % math.log(a.vocab))
    model, _, permutation = train(a.steps, a.tokens, a.vocab, a.dtype, a.lr, report=20)
    text = model.generate(7, 12)
    right = sum(int(permutation[u]) == v for u, v in zip(text, text[1:]))
    print("greedy continuation of 7:", text[1:], "(%d of 12 follow the permutation)" % right)


if __name__ == "__main__":
    main()
