"""A pre-norm feed-forward language model trained in 16 bits and served with
4-bit weights.

    python examples/served_lm.py [--steps 200] [--dtype bf16]

Per layer the residual stream is normed and goes through a gated feed-forward
block, whose output the next norm adds to the stream; the last norm's result meets
the embedding again as the output head.  Trained as in ffn_lm.py, on the same noisy
permutation.  Served, the norms write 8-bit microscaled operands, the weights are
4-bit ones, and tokens are sampled from the logits.
"""
import argparse
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
for path in (ROOT, os.path.join(ROOT, "examples")):
    if path not in sys.path:
        sys.path.insert(0, path)

import torch  # noqa: E402

import software_pipelined_tiled_pgemm_amd as pg  # noqa: E402
from ffn_lm import DTYPES, batches  # noqa: E402

EPS = 1e-5


class Model:
    """fp32 weights (`master`) and their 16-bit copies (`weights`): the embedding,
    and per layer the norm's weight and the block's two matrices; the last norm's
    weight."""

    def __init__(self, vocab=1000, width=256, hidden=512, layers=2, dtype=torch.bfloat16, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def normal(*shape, std):
            return torch.randn(*shape, generator=g, device="cuda") * std
        self.layers, self.dtype = layers, dtype
        self.master = {"embed": normal(vocab, width, std=0.5 * width ** -0.25)}
        for i in range(layers):
            self.master["norm%d" % i] = torch.ones(width, device="cuda")
            self.master["w_in%d" % i] = normal(width, 2 * hidden, std=width ** -0.5)
            self.master["w_out%d" % i] = normal(hidden, width, std=0.5 * hidden ** -0.5)
        self.master["norm%d" % layers] = torch.ones(width, device="cuda")
        self.momentum = {k: torch.zeros_like(v) for k, v in self.master.items()}
        self.refresh()

    def refresh(self):
        self.weights = {k: v.to(self.dtype) for k, v in self.master.items()}

    def loss_and_grads(self, tokens, targets):
        p, kept, grads = self.weights, [], {}
        h = p["embed"][tokens]
        n = pg.prmsnorm(h, p["norm0"], eps=EPS)
        for i in range(self.layers):
            form = torch.int16 if self.dtype is torch.bfloat16 else self.dtype
            w_in, w_out = p["w_in%d" % i], p["w_out%d" % i]
            gate_up = torch.empty(len(h), w_in.shape[1], dtype=form, device=h.device)
            out = pg.pffn(n, w_in, w_out, gate_up=gate_up)
            kept.append((h, n, gate_up))
            stream = torch.empty_like(h)
            n = pg.prmsnorm(out, p["norm%d" % (i + 1)], residual=h, eps=EPS, h=stream)
            h = stream
        loss, lse = pg.pxent(n, p["embed"], targets)
        dn, grads["embed"] = pg.pxent_bwd(n, p["embed"], targets, lse)
        # the gradient of the stream, and of the block that was added to it
        dh, grads["norm%d" % self.layers] = pg.prmsnorm_bwd(dn, h, p["norm%d" % self.layers], eps=EPS)
        for i in reversed(range(self.layers)):
            h, n, gate_up = kept[i]
            dn, grads["w_in%d" % i], grads["w_out%d" % i] = pg.pffn_bwd(
                dh, n, p["w_in%d" % i], p["w_out%d" % i], gate_up)
            dh, grads["norm%d" % i] = pg.prmsnorm_bwd(dn, h, p["norm%d" % i], eps=EPS, dh=dh)
        total = grads["embed"].float().index_add_(0, tokens, dh.float())
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


class Served:
    """A model's weights in 4 bits, one row per output, and its next tokens."""

    def __init__(self, model):
        self.layers, self.dtype = model.layers, model.dtype
        self.embed = model.weights["embed"]
        self.norms = [model.weights["norm%d" % i] for i in range(model.layers + 1)]
        self.w_in, self.w_out = ([pg.pmx_quantize(model.weights[n + str(i)].t().contiguous(), "e2m1")
                                  for i in range(model.layers)] for n in ("w_in", "w_out"))
        self.head = pg.pmx_quantize(self.embed, "e2m1")

    def logits(self, tokens):
        h = self.embed[tokens]
        n = pg.prmsnorm(h, self.norms[0], eps=EPS, format="e4m3")
        for i in range(self.layers):
            gate, up = pg.pmx_linear(n, self.w_in[i], dtype=self.dtype).chunk(2, dim=1)
            out = pg.pmx_linear(torch.nn.functional.silu(gate) * up, self.w_out[i])
            n = pg.prmsnorm(out, self.norms[i + 1], residual=h, eps=EPS, h=h, format="e4m3")
        return pg.pmx_linear(n, self.head, dtype=self.dtype)

    def next(self, tokens, u, **settings):
        """(tokens, logprobs) that follow each of `tokens`, drawn with u."""
        return pg.psample(self.logits(tokens), u, **settings)

    def generate(self, token, count, seed=0, **settings):
        g = torch.Generator(device="cuda").manual_seed(seed)
        tokens = torch.tensor([int(token)], device="cuda")
        out = [tokens]
        for _ in range(count):
            tokens, _ = self.next(tokens, torch.rand(1, generator=g, device="cuda"), **settings)
            out.append(tokens)
        return torch.cat(out).tolist()


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
    model, _, permutation = train(a.steps, a.tokens, a.vocab, a.dtype, a.lr, report=20)
    text = Served(model).generate(7, 12, temperature=0.7, top_k=20, top_p=0.95)
    right = sum(int(permutation[u]) == v for u, v in zip(text, text[1:]))
    print("sampled continuation of 7:", text[1:], "(%d of 12 follow the permutation)" % right)


if __name__ == "__main__":
    main()
